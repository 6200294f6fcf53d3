"""Lengths out of range, the ends of their type among them: such a sequence counts as empty in writes, reads
and attention, the record says so, and the sequences beside it are served."""

from __future__ import annotations

import pytest
import torch

import exact_attention_116_b200 as fa
from chunk_cases import Batch, assert_close, call

pytestmark = pytest.mark.gpu

LENGTHS = [-2 ** 31, -2 ** 31 + 1, -2 ** 31 + 3, -1, 2 ** 31 - 1, 2 ** 30, 65]  # the table has room for 64 keys


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("length", LENGTHS)
def test_a_length_out_of_range(length, f8):
    b = Batch([3, 2, 1], [9, 40, 12], 2, 2, 128, 16, f8, seed=7, stray=0)
    b.table = b.table[:, :4].contiguous()
    t = b.gpu()
    t["lens"][1] = length
    k, v = (torch.randn(b.total, 2, 128, generator=torch.Generator().manual_seed(i)).bfloat16().cuda() for i in (1, 2))
    before = [x.clone() for x in (t["k"], t["v"])]

    def reported():
        with pytest.raises(fa.FaError):
            fa.check()
        fa.check()  # the record was cleared

    fa.cache_write_paged(k, v, t["k"], t["v"], t["table"], t["lens"], t["cu"], t["ks"], t["vs"])
    reported()
    pages = b.table[1, :3].long().cuda()
    for cache, old in zip((t["k"], t["v"]), before):
        assert torch.equal(cache[pages].view(torch.uint8), old[pages].view(torch.uint8))
    rk, rv = fa.cache_read_paged(t["k"], t["v"], t["table"], t["lens"], t["cu"], b.total, t["ks"], t["vs"])
    reported()
    for got, x in ((rk, k), (rv, v)):
        assert (got[3:5] == 0).all()
        if not f8:
            assert torch.equal(got[:3], x[:3]) and torch.equal(got[5:], x[5:])
    o, lse = call(t)
    reported()
    assert (o[3:5] == 0).all() and (lse[:, 3:5] == -float("inf")).all()
    b.k, b.v = t["k"].cpu(), t["v"].cpu()
    b.ks, b.vs = (None, None) if not f8 else (t["ks"].cpu(), t["vs"].cpu())
    ref = b.reference(128 ** -0.5, True, (-1, -1), 0)
    for rows in (slice(0, 3), slice(5, 6)):
        part = tuple(x[:, rows] if i == 1 else x[rows] for i, x in enumerate(ref))
        assert_close(o[rows], lse[:, rows], part, rows.stop - rows.start, str(rows))
