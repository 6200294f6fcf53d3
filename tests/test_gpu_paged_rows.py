"""A paged read into slices of one tensor: interleaved K and V rows come out as they do apart, and what lies
between them stays."""

from __future__ import annotations

import pytest
import torch

import exact_attention_116_b200 as fa
from chunk_cases import Batch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("new", [[9, 70, 1], [1]])
@pytest.mark.parametrize("kv", [(0, 2), (2, 0), (3, 5), (0, 5)])
def test_interleaved_outputs(kv, new, f8):
    H, d = 2, 64
    b = Batch(new, [x + 30 for x in new], H, H, d, 16, f8, seed=len(new))
    t = b.gpu()
    plan = (t["table"], t["lens"], t["cu"])
    k, v = fa.cache_read_paged(t["k"], t["v"], *plan, b.total, t["ks"], t["vs"])
    wide = torch.full((b.total, 7, d), 3.0, dtype=torch.bfloat16, device="cuda")
    fa.cache_read_paged_into(t["k"], t["v"], *plan, wide[:, kv[0]:kv[0] + H], wide[:, kv[1]:kv[1] + H], t["ks"], t["vs"])
    fa.check()
    want = torch.full_like(wide, 3.0)
    want[:, kv[0]:kv[0] + H], want[:, kv[1]:kv[1] + H] = k, v
    assert torch.equal(wide, want)


@pytest.mark.parametrize("kv", [(0, 0), (0, 1), (3, 2)])
def test_overlapping_outputs_are_refused(kv):
    b = Batch([9, 4], [30, 40], 2, 2, 64, 16, False)
    t = b.gpu()
    wide = torch.zeros(b.total, 7, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(fa.FaError):
        fa.cache_read_paged_into(t["k"], t["v"], t["table"], t["lens"], t["cu"], wide[:, kv[0]:kv[0] + 2],
                                 wide[:, kv[1]:kv[1] + 2])
    assert (wide == 0).all()
