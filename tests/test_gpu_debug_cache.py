"""Paged cache writes, reads and chunk attention through the bounds-checking build of the library
(test_gpu_debug_build.py says what it checks): oracle parity, and no check fires."""

from __future__ import annotations

import pytest
import torch

import exact_attention_116_b200 as fa
from chunk_cases import Batch, assert_close, call
from exact_attention_116_b200 import binding
from exact_attention_116_b200 import build as cuda_build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def debug_lib():
    return binding.open_library(cuda_build.build(debug=True))


@pytest.fixture(autouse=True)
def use_debug_lib(debug_lib, monkeypatch):
    monkeypatch.setattr(binding, "_lib", debug_lib)
    yield


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("new,keys,Hq,Hkv,d,page,window,sinks", [
    ([1], [1], 1, 1, 64, 16, (-1, -1), 0),
    ([7], [7], 2, 2, 128, 64, (-1, -1), 0),
    ([1, 1], [300, 77], 8, 2, 128, 16, (-1, -1), 0),
    ([130, 0, 3], [400, 9, 3], 5, 1, 64, 48, (40, -1), 6),
    ([300, 1], [1300, 5000], 4, 2, 128, 256, (-1, -1), 0),
    ([200], [900], 7, 1, 128, 32, (100, -1), 200),
    ([9, 3], [4, 0], 4, 2, 128, 16, (-1, -1), 0),
    ([1, 1, 1], [9000, 20000, 1], 16, 1, 64, 128, (-1, -1), 0),
    ([2], [30000], 128, 1, 128, 80, (-1, -1), 0),
    ([1, 1, 1], [9000, 20000, 1], 16, 1, 128, 128, (-1, -1), 0),
    ([4, 2, 0, 4], [500, 2, 7, 1100], 4, 1, 128, 48, (40, -1), 6),
    ([1, 3, 1], [700, 3000, 130], 5, 1, 128, 16, (200, -1), 130),
])
def test_write_attend_read(new, keys, Hq, Hkv, d, page, window, sinks, f8):
    b = Batch(new, keys, Hq, Hkv, d, page, f8, pad=5, seed=sum(keys))
    t = b.gpu()
    rows = fa.cache_read_paged(t["k"], t["v"], t["table"], t["lens"], t["cu"], b.total, t["ks"], t["vs"])
    fa.check()
    fa.cache_write_paged(*rows, t["k"], t["v"], t["table"], t["lens"], t["cu"], t["ks"], t["vs"])
    fa.check()
    again = fa.cache_read_paged(t["k"], t["v"], t["table"], t["lens"], t["cu"], b.total, t["ks"], t["vs"])
    fa.check()
    live = sum(new)
    assert all(torch.equal(x[:live], y[:live]) for x, y in zip(rows, again))
    o, lse = call(t, None, True, window, sinks)
    fa.check()
    assert_close(o, lse, b.reference(d ** -0.5, True, window, sinks), live, "debug build")
