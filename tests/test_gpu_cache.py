"""Writing rows into a paged cache and reading them back on the GPU, against the float64 oracle: the
codes, scales and rows are defined exactly (power-of-two scales, one rounding), so they are compared
bit for bit."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import exact_attention_116_b200 as fa
from chunk_cases import Batch
from oracle import chunk_paged_fp64 as oracle

pytestmark = pytest.mark.gpu

SHAPES = [  # new rows, keys, heads, d, page size
    ([1], [1], 1, 64, 16),
    ([1, 1, 1], [5, 64, 65], 8, 128, 64),
    ([3, 0, 17, 1], [3, 9, 40, 100], 5, 128, 16),
    ([130, 7], [200, 7], 16, 64, 48),
    ([33, 64], [33, 300], 9, 128, 32),
    ([5, 4], [3, 4], 2, 64, 16),   # more new rows than positions: the first ones have no place
]


def rows(total, H, d, seed, wide=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(total, H, d + wide, generator=g) * torch.exp2(torch.randint(-20, 20, (total, H, 1), generator=g))
    return x.to(torch.bfloat16)


@pytest.mark.parametrize("new,keys,H,d,page", SHAPES)
@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("pad", [0, 3])
def test_write_then_read(new, keys, H, d, page, f8, pad):
    b = Batch(new, keys, H, H, d, page, f8, pad=pad, seed=len(new) + H)
    t = b.gpu()
    kn, vn = rows(b.total, H, d, 1), rows(b.total, H, d, 2)
    want = [x.clone() for x in (b.k, b.v)], [None if x is None else x.clone() for x in (b.ks, b.vs)]
    back = [torch.full((b.total, H, d), 7.0) for _ in range(2)]
    for s in range(len(new)):
        for i in range(new[s]):
            row = int(b.cu[s]) + i
            at = oracle.place(b.table.numpy(), b.lens.numpy(), b.cu.numpy(), page, s, i)
            for kv, x in enumerate((kn, vn)):
                if at is None:
                    back[kv][row] = 0.0
                elif f8:
                    codes, scale = oracle.quantise_rows(x[row].double().numpy())
                    want[0][kv].view(torch.uint8)[at] = torch.from_numpy(codes)
                    want[1][kv][at[0], :, at[1]] = torch.from_numpy(scale)
                    back[kv][row] = torch.from_numpy(oracle.row_values(codes, scale))
                else:
                    want[0][kv][at] = x[row]
                    back[kv][row] = x[row].float()
    fa.cache_write_paged(kn.cuda(), vn.cuda(), t["k"], t["v"], t["table"], t["lens"], t["cu"], t["ks"], t["vs"])
    out = [torch.full((b.total, H, d), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    fa.cache_read_paged_into(t["k"], t["v"], t["table"], t["lens"], t["cu"], *out, t["ks"], t["vs"])
    fa.check()
    for got, ref in zip((t["k"], t["v"]), want[0]):
        assert torch.equal(got.cpu().view(torch.uint8), ref.view(torch.uint8))
    if f8:
        for got, ref in zip((t["ks"], t["vs"]), want[1]):
            assert torch.equal(got.cpu(), ref)
    for got, ref in zip(out, back):
        assert torch.equal(got.cpu().float(), ref)


def test_every_code_every_scale_reads_back_exactly():
    """All finite codes under all written scales: code * 2^e, subnormal codes included. A code above 240
    under the scale 2^120 (never written) is 2^128 or more, which bf16 rounds to infinity."""
    scales = np.arange(17, 248)
    H, d, page = 1, 128, 16
    n = 2 * len(scales)
    b = Batch([n], [n], H, H, d, page, True)
    at = [oracle.place(b.table.numpy(), [n], [0, n], page, 0, i) for i in range(n)]
    codes = np.arange(256, dtype=np.uint8).reshape(2, 128)
    codes[codes % 128 == 127] = 0
    ref = np.zeros((n, 1, d))
    for i, (pg, r) in enumerate(at):
        b.k.view(torch.uint8)[pg, r, 0] = torch.from_numpy(codes[i % 2])
        b.ks[pg, 0, r] = int(scales[i // 2])
        ref[i, 0] = oracle.row_values(codes[i % 2], scales[i // 2])
    t = b.gpu()
    k, _ = fa.cache_read_paged(t["k"], t["k"].clone(), t["table"], t["lens"], t["cu"], n, t["ks"], t["ks"].clone())
    fa.check()
    ref = np.where(np.abs(ref) >= 2.0 ** 128, np.copysign(np.inf, ref), ref)
    assert np.array_equal(k.double().cpu().numpy(), ref)


@pytest.mark.parametrize("d", [64, 128])
def test_values_at_the_borders(d):
    """Zero rows, the largest and least bf16 values, ties, subnormals; rows with NaN or an infinity."""
    x = torch.zeros(8, 1, d, dtype=torch.bfloat16)
    x[1, 0, 3] = 3.3895e38
    x[2, 0, 0] = 1e-40            # a bf16 subnormal
    x[3, 0, :4] = torch.tensor([448.0, 1.0625, 1.1875, -17.0])
    x[4, 0, 5] = float("nan")
    x[5, 0, d - 1] = float("-inf")
    x[6, 0] = -0.0
    x[7, 0, :3] = torch.tensor([1.7578125, 0.001, -1.75])
    b = Batch([8], [8], 1, 1, d, 16, True)
    t = b.gpu()
    fa.cache_write_paged(x.cuda(), x.cuda(), t["k"], t["v"], t["table"], t["lens"], t["cu"], t["ks"], t["vs"])
    k, v = fa.cache_read_paged(t["k"], t["v"], t["table"], t["lens"], t["cu"], 8, t["ks"], t["vs"])
    fa.check()
    codes, scale = oracle.quantise_rows(x.double().numpy())
    ref = oracle.row_values(codes, scale)
    assert np.array_equal(k.double().cpu().numpy(), ref, equal_nan=True)
    assert torch.equal(k.view(torch.int16), v.view(torch.int16)) and np.isnan(ref[4:6]).all()


@pytest.mark.parametrize("f8", [False, True])
def test_rows_sliced_from_a_projection_and_another_stream(f8):
    H, d, page = 4, 128, 32
    b = Batch([40, 3], [50, 70], H, H, d, page, f8, seed=5)
    qkv = torch.randn(43, 3 * H * d).to(torch.bfloat16).cuda()
    kn, vn = (qkv[:, i * H * d:(i + 1) * H * d].view(43, H, d) for i in (1, 2))
    t, u = b.gpu(), b.gpu()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    fa.cache_write_paged(kn, vn, t["k"], t["v"], t["table"], t["lens"], t["cu"], t["ks"], t["vs"], stream=side)
    k, v = fa.cache_read_paged(t["k"], t["v"], t["table"], t["lens"], t["cu"], 43, t["ks"], t["vs"], stream=side)
    torch.cuda.current_stream().wait_stream(side)
    fa.cache_write_paged(kn.contiguous(), vn.contiguous(), u["k"], u["v"], u["table"], u["lens"], u["cu"], u["ks"],
                         u["vs"])
    fa.check()
    assert torch.equal(t["k"].view(torch.uint8), u["k"].view(torch.uint8))
    assert torch.equal(t["v"].view(torch.uint8), u["v"].view(torch.uint8))
    kv = torch.empty(43, 2, H, d, dtype=torch.bfloat16, device="cuda")  # read into slices of one tensor
    fa.cache_read_paged_into(t["k"], t["v"], t["table"], t["lens"], t["cu"], kv[:, 0], kv[:, 1], t["ks"], t["vs"])
    assert torch.equal(kv[:, 0], k) and torch.equal(kv[:, 1], v)
    if not f8:
        assert torch.equal(k, kn) and torch.equal(v, vn)


def test_bad_pages_and_lengths_are_reported_and_not_followed():
    H, d, page = 2, 64, 16
    b = Batch([20, 4, 6], [20, 4, 6], H, H, d, page, True, seed=3)
    kn = rows(30, H, d, 4)
    for what in ("page", "length", "offsets"):
        t = b.gpu()
        before = t["k"].clone(), t["ks"].clone()
        if what == "page":
            t["table"][0, 1] = t["k"].shape[0]
        elif what == "length":
            t["lens"][2] = t["table"].shape[1] * page + 1
        else:
            t["cu"][3] = 31
        fa.cache_write_paged(kn.cuda(), kn.cuda(), t["k"], t["v"], t["table"], t["lens"], t["cu"], t["ks"], t["vs"])
        with pytest.raises(fa.FaError):
            fa.check()
        k, _ = fa.cache_read_paged(t["k"], t["v"], t["table"], t["lens"], t["cu"], 30, t["ks"], t["vs"])
        with pytest.raises(fa.FaError):
            fa.check()
        bad = slice(16, 20) if what == "page" else slice(24, 30)
        ref = oracle.row_values(*oracle.quantise_rows(kn.double().numpy()))
        good = [i for i in range(30) if not bad.start <= i < bad.stop]
        assert np.array_equal(k.double().cpu().numpy()[good], ref[good])
        if what != "offsets":  # (rows of bad offsets belong to no sequence)
            assert (k[bad] == 0).all()
        changed = (t["k"].view(torch.uint8) != before[0].view(torch.uint8)).any(-1).any(-1).sum()
        assert int(changed) <= len(good)


def test_places_past_2_31_elements():
    H, d, page, num_pages = 8, 128, 256, 9000   # 2.36e9 elements
    k = torch.empty(num_pages, page, H, d, dtype=torch.float8_e4m3fn, device="cuda")
    ks = torch.empty(num_pages, H, page, dtype=torch.uint8, device="cuda")
    v, vs = torch.empty_like(k), torch.empty_like(ks)
    table = torch.tensor([[num_pages - 1, 0]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([300], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 300], dtype=torch.int32, device="cuda")
    kn, vn = rows(300, H, d, 8).cuda(), rows(300, H, d, 9).cuda()
    fa.cache_write_paged(kn, vn, k, v, table, lens, cu, ks, vs)
    rk, rv = fa.cache_read_paged(k, v, table, lens, cu, 300, ks, vs)
    fa.check()
    for got, x in ((rk, kn), (rv, vn)):
        ref = oracle.row_values(*oracle.quantise_rows(x[::37].double().cpu().numpy()))
        assert np.array_equal(got[::37].double().cpu().numpy(), ref)


def test_nothing_to_do():
    b = Batch([2], [2], 1, 1, 64, 16, True)
    t = b.gpu()
    none = torch.empty(0, 1, 64, dtype=torch.bfloat16, device="cuda")
    t["cu"].zero_()
    before = t["k"].clone()
    fa.cache_write_paged(none, none, t["k"], t["v"], t["table"], t["lens"], t["cu"], t["ks"], t["vs"])
    k, v = fa.cache_read_paged(t["k"], t["v"], t["table"], t["lens"], t["cu"], 0, t["ks"], t["vs"])
    fa.check()
    assert k.shape == (0, 1, 64) and torch.equal(before.view(torch.uint8), t["k"].view(torch.uint8))
