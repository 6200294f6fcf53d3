"""Calls on one stream take effect in order. Kernels launched as programmatic dependents may begin before
the kernel ahead of them has ended, so every such launch needs a wait: seen in the edges of a captured graph
(nothing runs there), and in chains of dependent calls whose results must equal those of the same calls
with the device idle between them."""

from __future__ import annotations

import ctypes

import pytest
import torch

import exact_attention_116_b200 as fa
from chunk_cases import Batch

pytestmark = pytest.mark.gpu

FULL, PROGRAMMATIC = 0, 1


class EdgeData(ctypes.Structure):
    _fields_ = [("from_port", ctypes.c_ubyte), ("to_port", ctypes.c_ubyte), ("type", ctypes.c_ubyte),
                ("reserved", ctypes.c_ubyte * 5)]


def edge_kinds(call):
    """The kinds of the edges between the kernels that `call` launches, in launch order (captured, not run)."""
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph):
        call()
    handle, count = ctypes.c_void_p(graph.raw_cuda_graph()), ctypes.c_size_t(0)
    get = ctypes.CDLL("libcuda.so.1").cuGraphGetEdges_v2
    assert get(handle, None, None, None, ctypes.byref(count)) == 0
    n = count.value
    ends, data = [(ctypes.c_void_p * n)() for _ in range(2)], (EdgeData * n)()
    assert get(handle, ends[0], ends[1], data, ctypes.byref(count)) == 0
    after = {ends[0][i]: (ends[1][i], data[i].type) for i in range(n)}
    assert len(after) == n  # one chain
    node = (set(after) - {to for to, _ in after.values()}).pop()
    kinds = []
    while node in after:
        node, kind = after[node]
        kinds.append(kind)
    return kinds


def batch(new, keys, H=2, f8=False, page=64, d=128):
    return Batch(new, keys, H, H, d, page, f8, seed=sum(keys) + len(new), stray=0)


def write(t, k, v):
    fa.cache_write_paged(k, v, t["k"], t["v"], t["table"], t["lens"], t["cu"], t["ks"], t["vs"])


def test_a_decode_of_several_pieces_begins_early_only_behind_its_own_counters():
    b = batch([1, 1], [100, 70])
    t = b.gpu()
    k, v = (torch.zeros_like(t["q"]) for _ in range(2))
    q = t["q"].view(2, 1, 2, 128)
    o, lse = torch.zeros_like(q), torch.zeros(2, 2, 1, device="cuda")
    ws = torch.zeros(fa.decode_workspace_bytes(2, 1, 2, 128, 2), dtype=torch.uint8, device="cuda")
    fa.decode_splits(2, 1, 2, 128, 128)  # the device's set-up, outside the capture
    torch.cuda.synchronize()

    def step():
        write(t, k, v)
        fa.decode_paged_into(q, t["k"], t["v"], t["table"], t["lens"], o, lse, causal=True, splits=2, workspace=ws)

    assert edge_kinds(step) == [FULL, PROGRAMMATIC]


CHAINS = {  # new rows, keys: a cache of one key tile (no join), a long chunk ahead, several sequences
    "one tile": ([4], [60]), "long chunk": ([900], [6000]), "several": ([4, 300, 9], [90, 2500, 700]),
}


@pytest.mark.parametrize("splits", [1, 3])
@pytest.mark.parametrize("append", [False, True])
@pytest.mark.parametrize("case", list(CHAINS))
def test_paged_calls_and_decodes_in_turn(case, append, splits):
    """write -> chunk -> decode of the chunk's output (appending rows the chunk reads) -> write -> decode ->
    read, with nothing else on the stream."""
    new, keys = CHAINS[case]
    b = batch(new, keys)
    B, total, H, d = len(new), sum(new), 2, 128
    g = torch.Generator().manual_seed(5)
    rows = [[torch.randn(total, H, d, generator=g).bfloat16().cuda() for _ in range(4)] for _ in range(3)]
    last = torch.randn(2, B, 4, H, d, generator=g).bfloat16().cuda()
    ws = torch.empty(fa.chunk_workspace_bytes(B, total, H, H, d), dtype=torch.uint8, device="cuda")
    dws = torch.empty(max(256, fa.decode_workspace_bytes(B, 4, H, d, splits)), dtype=torch.uint8, device="cuda")

    def run(pause):
        t, out = b.gpu(), []
        o, lse = torch.zeros(total, H, d, dtype=torch.bfloat16, device="cuda"), torch.zeros(H, total, device="cuda")
        o2 = [torch.zeros(B, 4, H, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        lse2 = [torch.zeros(B, H, 4, device="cuda") for _ in range(2)]
        back = [torch.zeros(total, H, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        torch.cuda.synchronize()

        def then(call):
            call()
            if pause:
                torch.cuda.synchronize()

        def decode(i):  # its queries: the first rows of the chunk's output
            fa.decode_paged_into(o.view(-1)[:B * 4 * H * d].view(B, 4, H, d), t["k"], t["v"], t["table"], t["lens"],
                                 o2[i], lse2[i], causal=True, splits=splits, workspace=dws,
                                 k_new=last[0] if append else None, v_new=last[1] if append else None)

        for k, v, k2, v2 in rows:
            then(lambda: write(t, k, v))
            then(lambda: fa.chunk_paged_into(t["q"], t["k"], t["v"], t["table"], t["lens"], t["cu"], o, lse, None, True,
                                             workspace=ws))
            then(lambda: decode(0))
            then(lambda: write(t, k2, v2))
            then(lambda: decode(1))
            then(lambda: fa.cache_read_paged_into(t["k"], t["v"], t["table"], t["lens"], t["cu"], *back))
            torch.cuda.synchronize()
            out += [x.clone() for x in (o, lse, *o2, *lse2, *back, t["k"], t["v"])]
        fa.check()
        return out

    slow = run(True)
    for _ in range(4):
        for got, ref in zip(run(False), slow):
            assert torch.equal(got, ref)
