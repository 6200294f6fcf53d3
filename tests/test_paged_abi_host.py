"""Host-side checks of the paged-cache calls: they refuse invalid arguments before anything is launched
(fake pointers are never dereferenced), the argument structures have the layout the binding packs, and the
set-up's arithmetic (fast division, pieces) covers every tile once. No GPU is touched."""

from __future__ import annotations

import ctypes
import os
import re

import numpy as np
import pytest
import torch

import exact_attention_116_b200 as fa
from exact_attention_116_b200 import binding, build

OK, INVALID, UNSUPPORTED = 0, 1, 2
P = 0x7F0000000000
T = 1 << 42  # fake tensors far apart
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


CACHE = dict(rows_k=P, rows_v=P + T, stride=1024, k=P + 2 * T, v=P + 3 * T, ks=None, vs=None, table=P + 6 * T,
             lens=P + 7 * T, cu=P + 8 * T, B=2, total=10, H=8, d=128, pages=16, page=64, most=8)
F8 = dict(ks=P + 4 * T, vs=P + 5 * T)
CACHE_BAD = [
    (dict(B=0), INVALID), (dict(total=-1), INVALID), (dict(H=0), INVALID), (dict(pages=0), INVALID),
    (dict(page=0), INVALID), (dict(most=0), INVALID), (dict(d=96), UNSUPPORTED), (dict(page=24), UNSUPPORTED),
    (dict(rows_k=None), INVALID), (dict(k=None), INVALID), (dict(table=None), INVALID), (dict(lens=None), INVALID),
    (dict(cu=None), INVALID), (dict(stride=1016), INVALID), (dict(stride=1028), INVALID), (dict(rows_v=P + T + 8), INVALID),
    (dict(k=P + 2 * T + 2), INVALID), (dict(ks=P + 4 * T), INVALID), (dict(F8, vs=P + 5 * T + 4), INVALID),
    (dict(k=P), INVALID), (dict(F8, ks=P + 2 * T), INVALID), (dict(most=1 << 26), INVALID), (dict(total=(1 << 30) + 1), INVALID),
    (dict(stride=(1 << 30) + 8), INVALID), (dict(pages=1 << 28), INVALID), (dict(table=P + 2 * T), INVALID),
    (dict(v=P + 2 * T + 1024), INVALID),
]


def call_cache(lib, write, **kw):
    a = dict(CACHE, **kw)
    rest = (a["B"], a["total"], a["H"], a["d"], a["pages"], a["page"], a["most"], None)
    cache, plan = (a["k"], a["v"], a["ks"], a["vs"]), (a["table"], a["lens"], a["cu"])
    if write:
        return lib.fa_cache_write(a["rows_k"], a["rows_v"], a["stride"], *cache, *plan, *rest)
    return lib.fa_cache_read(*cache, *plan, a["rows_k"], a["rows_v"], a["stride"], *rest)


@pytest.mark.parametrize("kw,expected", CACHE_BAD)
def test_cache_write_refuses(lib, kw, expected):
    assert call_cache(lib, True, **kw) == expected


WRITTEN = (dict(table=P + 2 * T), dict(v=P + 2 * T + 1024), dict(F8, ks=P + 2 * T))  # caches that a read may share


@pytest.mark.parametrize("kw,expected", [c for c in CACHE_BAD if c[0] not in WRITTEN] +
                         [(dict(rows_v=P), INVALID), (dict(table=P + 64), INVALID)])
def test_cache_read_refuses(lib, kw, expected):
    assert call_cache(lib, False, **kw) == expected


CHUNK = dict(q=P, stride=2048, k=P + T, v=P + 2 * T, ks=None, vs=None, table=P + 5 * T, lens=P + 6 * T, cu=P + 7 * T,
             o=P + 8 * T, lse=P + 9 * T, B=2, total=10, Hq=16, Hkv=8, d=128, pages=16, page=64, most=8, scale=0.1,
             causal=1, win_l=-1, win_r=-1, sinks=0, ws=P + 10 * T, wb=1 << 40)
CHUNK_BAD = [
    (dict(Hq=0), INVALID), (dict(Hkv=0), INVALID), (dict(Hq=17), INVALID), (dict(win_l=-2), INVALID),
    (dict(win_r=-2), INVALID), (dict(sinks=-1), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(d=80), UNSUPPORTED), (dict(page=40), UNSUPPORTED),
    (dict(Hq=129, Hkv=1, stride=129 * 128), UNSUPPORTED), (dict(q=None), INVALID), (dict(o=None), INVALID),
    (dict(lse=None), INVALID), (dict(stride=2040), INVALID), (dict(stride=2052), INVALID), (dict(q=P + 4), INVALID),
    (dict(o=P + 8 * T + 8), INVALID), (dict(lse=P + 9 * T + 2), INVALID), (dict(vs=P + 3 * T), INVALID),
    (dict(o=P), INVALID), (dict(lse=P + 8 * T), INVALID), (dict(o=P + T), INVALID), (dict(lse=P + 6 * T), INVALID),
    (dict(B=0), INVALID), (dict(total=-1), INVALID), (dict(cu=None), INVALID), (dict(most=1 << 25), INVALID),
]


def call_chunk(lib, **kw):
    a = dict(CHUNK, **kw)
    return lib.fa_chunk_paged(a["q"], a["stride"], a["k"], a["v"], a["ks"], a["vs"], a["table"], a["lens"], a["cu"],
                              a["o"], a["lse"], a["B"], a["total"], a["Hq"], a["Hkv"], a["d"], a["pages"], a["page"],
                              a["most"], a["scale"], a["causal"], a["win_l"], a["win_r"], a["sinks"], a["ws"], a["wb"],
                              None)


@pytest.mark.parametrize("kw,expected", CHUNK_BAD)
def test_chunk_refuses(lib, kw, expected):
    assert call_chunk(lib, **kw) == expected


@pytest.mark.parametrize("B,total,Hq,Hkv,d", [(0, 1, 1, 1, 64), (1, -1, 1, 1, 64), (1, 1, 3, 2, 64), (1, 1, 1, 1, 32)])
def test_chunk_workspace_of_invalid_sizes_is_none(lib, B, total, Hq, Hkv, d):
    assert fa.chunk_workspace_bytes(B, total, Hq, Hkv, d) == 0


def test_structures_reach_the_same_checks(lib):
    for name in ("fa_cache_write_args", "fa_cache_read_args", "fa_chunk_paged_args"):
        assert getattr(lib, name)(None) == INVALID
    pack = binding._CHUNK_ARGS.pack
    a = CHUNK

    def packed(**kw):
        c = dict(a, **kw)
        return pack(c["q"], c["k"], c["v"], 0, 0, c["table"], c["lens"], c["cu"], c["o"], c["lse"], c["ws"], 0, c["wb"],
                    c["stride"], c["B"], c["total"], c["Hq"], c["Hkv"], c["d"], c["pages"], c["page"], c["most"],
                    c["causal"], c["win_l"], c["win_r"], c["sinks"], c["scale"])

    for kw, expected in CHUNK_BAD:
        if None not in kw.values() and "vs" not in kw:
            assert lib.fa_chunk_paged_args(packed(**kw)) == expected, kw
    rows = binding._CACHE_ARGS.pack(P, P + T, P + 2 * T, P + 3 * T, 0, 0, P + 6 * T, P + 7 * T, P + 8 * T, 0, 1016, 2, 10, 8,
                                    128, 16, 64, 8)
    assert lib.fa_cache_write_args(rows) == INVALID and lib.fa_cache_read_args(rows) == INVALID


def test_structures_are_packed_as_declared():
    """The fields of the header's structures, in order, against the binding's formats."""
    with open(os.path.join(ROOT, "include", "fa_sm100.h")) as f:
        text = f.read()
    kinds = {"int": ctypes.c_int, "long long": ctypes.c_longlong, "float": ctypes.c_float, "size_t": ctypes.c_size_t}
    for name, packer in (("fa_cache_args", binding._CACHE_ARGS), ("fa_chunk_args", binding._CHUNK_ARGS)):
        body = re.search(r"typedef struct \{([^}]*)\} " + name, text).group(1)
        fields = []
        for line in body.split(";")[:-1]:
            kind, names = re.match(r"\s*(?:const )?(void|int|float|size_t|long long|fa_stream_t)\s*(.*)", line.strip(), re.S).groups()
            for one in names.split(","):
                pointer = "*" in one or "*" in names.split(",")[0] and kind == "void" or kind == "fa_stream_t"
                fields.append((one.strip(" *"), ctypes.c_void_p if pointer else kinds[kind]))
        struct = type(name, (ctypes.Structure,), {"_fields_": fields})
        assert ctypes.sizeof(struct) == packer.size
        values = list(range(1, len(fields) + 1))
        got = struct.from_buffer_copy(packer.pack(*values))
        assert [getattr(got, n) for n, _ in fields] == values


def test_binding_has_no_cpu_path():
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    cache = torch.zeros(2, 16, 2, 64, dtype=torch.bfloat16)
    plan = torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    for call in (lambda: fa.cache_write_paged(x, x, cache, cache.clone(), *plan),
                 lambda: fa.cache_read_paged(cache, cache.clone(), *plan, 4),
                 lambda: fa.attention_chunk_paged(x, cache, cache.clone(), *plan)):
        with pytest.raises(ValueError):
            call()


def test_fast_division():
    """n / d = (n + hi32(n m)) >> s with s = ceil(log2 d), m = ceil(2^(32 + s) / d) - 2^32, 0 <= n < 2^31."""
    rng = np.random.default_rng(0)
    for d in [1, 2, 3, 5, 7, 16, 24, 48, 80, 127, 128, 129, 1000, 65535, 65536, 1 << 30, (1 << 30) - 1]:
        s = (d - 1).bit_length()
        m = -(-(1 << (32 + s)) // d) - (1 << 32)
        assert 0 <= m < 1 << 32
        n = np.unique(np.concatenate([np.arange(3 * min(d, 70000)), rng.integers(0, 1 << 31, 20000),
                                      [k * d + e for k in (1, 2, 1000) for e in (-1, 0, 1)], [(1 << 31) - 1]]))
        n = n[(n >= 0) & (n < 1 << 31)].astype(np.uint64)
        got = (n + (n * np.uint64(m) >> np.uint64(32))) >> np.uint64(s)
        assert np.array_equal(got, n // np.uint64(d)) and int((n + (n * np.uint64(m) >> np.uint64(32))).max()) < 1 << 32


@pytest.mark.parametrize("seed", range(6))
def test_pieces_cover_every_tile_once(seed):
    """A model of the work split: pieces of a list of T tiles, the blocks they cut, and their partials' slots."""
    rng = np.random.default_rng(seed)
    for _ in range(200):
        hg = int(rng.choice([1, 2, 4]))
        pieces = int(rng.integers(1, 148 // hg + 1))
        blocks = rng.integers(1, 60, size=rng.integers(1, 80))  # tiles of each block, groups one after another
        T = int(blocks.sum())
        pe = min(pieces, T)
        each, more = T // pe, T % pe
        lo = [each * r + min(r, more) for r in range(pe + 1)]
        assert lo[pe] == T and all(1 <= b - a <= each + 1 for a, b in zip(lo, lo[1:]))
        starts = np.concatenate([[0], np.cumsum(blocks)])
        used = set()
        for s, n in zip(starts, blocks):
            first, last = (next(r for r in range(pe) if lo[r] <= u < lo[r + 1]) for u in (s, s + n - 1))
            head = more * (each + 1)
            u = int(s + n - 1)
            assert last == (u // (each + 1) if u < head else more + (u - head) // each)
            if first == last:
                assert s >= lo[first] and s + n <= lo[first + 1]
                continue
            for e in range(hg):  # the CTAs of the group's heads
                for i, r in enumerate(range(first, last + 1)):
                    cta = r * hg + e
                    slot = 2 * cta + (1 if i == 0 and s > lo[r] else 0)
                    assert slot not in used and slot < 2 * pieces * hg
                    used.add(slot)
                    assert cta == first * hg + e + i * hg
