"""Scores that pass fp32's range: a visible one makes its row what the formula makes of it (infinity - infinity
is not a number), a masked one leaves no trace, wherever the key lies in its tile and whatever the sign of the
scale. Products of 2^120 and 2^120 overflow in the first sum."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import exact_attention_116_b200 as fa
from chunk_cases import Batch, assert_close, call

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new", [3, 150])
@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("scale", [0.1, -0.1])
@pytest.mark.parametrize("where", [5, 130, 330])
def test_a_key_whose_scores_pass_the_range(d, new, sign, scale, where):
    n = 400
    b = Batch([new], [n], 2, 1, d, 16, False, seed=new + where)
    b.q[:, :, 0] = 2.0 ** 120
    b.k[..., 0] = 0.0
    b.k[int(b.table[0, where // 16]), where % 16, 0, 0] = sign * 2.0 ** 120
    o, lse = call(b.gpu(), scale, True, (100, -1), 3)
    fa.check()
    pos = np.arange(n - new, n)
    sees = torch.from_numpy((where <= pos) & ((where >= pos - 100) | (where < 3)))
    rises = sign * scale > 0  # the score is +infinity: O and LSE are not numbers; -infinity: no weight
    if rises and bool(sees.any()):
        assert bool(o[sees.cuda()].isnan().all()) and bool((~lse[:, sees.cuda()].isfinite()).all())
    keep = ~sees if rises else torch.ones_like(sees)
    if not bool(keep.any()):
        return
    # without the key's overflowing column: it is masked for these rows, or of no weight
    c = Batch([new], [n], 2, 1, d, 16, False, seed=new + where)
    c.q[:, :, 0] = 0.0
    c.k[..., 0] = 0.0
    if not rises:  # no weight: a score far below the others' (scores are within 100 of 0)
        c.q[:, :, 0] = 2.0 ** 7
        c.k[int(c.table[0, where // 16]), where % 16, 0, 0] = sign * 2.0 ** 7
    o_ref, lse_ref, spread = c.reference(scale, True, (100, -1), 3)
    rows = np.flatnonzero(keep.numpy())
    assert_close(o[rows], lse[:, rows], (o_ref[rows], lse_ref[:, rows], spread[rows]), len(rows), "the other rows")
