"""Rows of a few tokens over quantised pages whose values differ widely in size: every row's answer follows
from the keys that it sees and the weight that it gives them, whatever lies in the rows beside them.

Tolerance, for each element: the weights are rounded to 9 bits and O to bf16, the scores and exponentials
add 1e-3 (chunk_cases.py). Besides, a weight times its value's scale, W, is a sum of three E5M2 numbers in
units in which the row's largest W is at least 2^9. Each of the three is rounded on its own, by at most half
the least E5M2 number, 2^-17, where it is below E5M2's normal range, and exactly above it. So W is off by at
most 3 * 2^-17, which is 3 * 2^-26 of the row's largest W, for each key times its code. Nothing is added for
small values.
"""

from __future__ import annotations

import numpy as np
import pytest
import torch

import exact_attention_116_b200 as fa
from chunk_cases import LSE_TOL, Batch, call, np64
from oracle import chunk_paged_fp64 as oracle
from oracle.fp8_e4m3 import decode_e4m3

pytestmark = pytest.mark.gpu

D = 128


def shift(b, s, positions, e):
    """Multiplies the values of some positions of sequence s by 2^e."""
    page = b.k.shape[1]
    for j, x in zip(positions, np.broadcast_to(e, (len(positions),))):
        at = b.vs[int(b.table[s, j // page]), :, j % page]
        at.copy_((at.to(torch.int32) + int(x)).clamp(17, 247).to(torch.uint8))


def point(b, s, position, head, rows, size):
    """Gives the key at a position of sequence s a score of about size / sqrt(d) per row sum."""
    page = b.k.shape[1]
    q = b.q[rows, head * (b.q.shape[1] // b.k.shape[2])].float().mean(0)
    x = (q / q.norm() * size).to(torch.float8_e4m3fn)
    b.k[int(b.table[s, position // page]), position % page, head] = x
    b.ks[int(b.table[s, position // page]), head, position % page] = 127


def products_error(b, scale, win, sinks):
    """3 * 2^-26 of each row's largest weight times value scale, times the codes of the keys that it sees."""
    total, Hq, _ = b.q.shape
    page, H = b.k.shape[1], b.k.shape[2]
    out = np.zeros((total, Hq, D))
    q = np64(b.q)
    for s, n in enumerate(b.keys):
        c0, c1 = int(b.cu[s]), int(b.cu[s + 1])
        see = oracle.visible(np.arange(n - (c1 - c0), n), n, True, *win, sinks)
        at = np.arange(n)
        pages, rows = b.table.numpy()[s, at // page], at % page
        for h in range(Hq):
            kv = h // (Hq // H)
            k = oracle.row_values(b.k.view(torch.uint8).numpy()[pages, rows, kv], b.ks.numpy()[pages, kv, rows])
            codes = np.abs(decode_e4m3(b.v.view(torch.uint8).numpy()[pages, rows, kv]))
            unit = np.exp2(b.vs.numpy()[pages, kv, rows].astype(float) - 127)
            x = np.where(see, scale * (q[c0:c1, h] @ k.T), -np.inf)
            w = np.exp(x - np.maximum(x.max(1, keepdims=True), -1e300))
            w /= np.maximum(w.sum(1, keepdims=True), 1e-300)
            out[c0:c1, h] = 3 * 2.0 ** -26 * (w * unit).max(1, keepdims=True) * (see @ codes)
    return out


def check(b, win=(-1, -1), sinks=0, what=""):
    scale = D ** -0.5
    o, lse = call(b.gpu(), None, True, win, sinks)
    fa.check()
    o_ref, lse_ref, spread = b.reference(scale, True, win, sinks)
    dead = ~np.isfinite(lse_ref)  # rows without a place
    assert np.array_equal(dead, np64(lse) == -np.inf) and (np64(o).transpose(1, 0, 2)[dead] == 0).all(), what
    assert np.abs(np.where(dead, 0, np64(lse)) - np.where(dead, 0, lse_ref)).max() <= LSE_TOL, what
    tol = 1.01 * ((2.0 ** -8 + 1e-3) * spread + 2.0 ** -8 * np.abs(o_ref) + products_error(b, scale, win, sinks))
    worst = np.max(np.abs(np64(o) - o_ref) / np.maximum(tol, 1e-300), axis=(1, 2))  # of each token
    assert (worst <= 1.0).all(), f"{what}: {worst}"


LAYOUTS = [(4, 1), (8, 2), (16, 1), (2, 2)]  # query and cache heads


def rows_of(Hq, Hkv):
    return min(4, 16 // (Hq // Hkv))


@pytest.mark.parametrize("Hq,Hkv", LAYOUTS)
@pytest.mark.parametrize("e", [12, 30, 60, 100])
@pytest.mark.parametrize("keys", [7, 300, 5000])
def test_a_later_token_with_larger_values(Hq, Hkv, e, keys):
    m = rows_of(Hq, Hkv)
    b = Batch([m, m], [keys, 40], Hq, Hkv, D, 16, True, seed=e + keys)
    for s, n in enumerate((keys, 40)):
        shift(b, s, [n - 1], e)
        if m > 2:
            shift(b, s, [n - 2], e // 2)
    check(b, what=f"{e}")
    check(b, (200, -1), 3, what=f"{e} window")


@pytest.mark.parametrize("Hq,Hkv", LAYOUTS)
@pytest.mark.parametrize("e", [12, 30, 100])
def test_large_values_of_negligible_weight(Hq, Hkv, e):
    """Keys that every row sees with a weight of 2^-60 and less."""
    m = rows_of(Hq, Hkv)
    for where in (0, 130, 690):
        b = Batch([m], [700], Hq, Hkv, D, 32, True, seed=e + where)
        b.q[:] = (b.q.float() + 3.0).to(torch.bfloat16)  # rows with a common direction, so that one key opposes all
        for h in range(Hkv):
            point(b, 0, where, h, slice(0, m), -200.0)
        shift(b, 0, [where], e)
        check(b, what=f"{e} at {where}")


@pytest.mark.parametrize("Hq,Hkv", LAYOUTS)
def test_small_values_under_a_large_weight_and_large_ones_under_small(Hq, Hkv):
    """The key that takes nearly all the weight comes first, in the middle or last; values of 2^-40 to 2^40."""
    m = rows_of(Hq, Hkv)
    for where in (0, 300, 690 - m):
        for e in (-40, -9, 40):
            b = Batch([m], [700], Hq, Hkv, D, 16, True, seed=where + e + 41)
            b.q[:] = (b.q.float() + 2.0).to(torch.bfloat16)
            for h in range(Hkv):
                point(b, 0, where, h, slice(0, m), 60.0)
            shift(b, 0, [where], e)
            check(b, what=f"{e} at {where}")


@pytest.mark.parametrize("Hq,Hkv", LAYOUTS)
@pytest.mark.parametrize("keys", [[5, 128, 129], [1000, 3000, 257]])
def test_values_of_all_sizes(Hq, Hkv, keys):
    m = rows_of(Hq, Hkv)
    rng = np.random.default_rng(sum(keys))
    for spread in (4, 20, 90):
        b = Batch([m, 1, m], keys, Hq, Hkv, D, 48, True, seed=spread)
        for s, n in enumerate(keys):
            shift(b, s, range(n), rng.integers(-spread, spread + 1, size=n))
        check(b, what=f"{spread}")
        rising = np.sort(rng.integers(-spread, spread + 1, size=max(keys)))
        for order in (rising, rising[::-1]):
            b = Batch([m, 1, m], keys, Hq, Hkv, D, 48, True, seed=spread)
            for s, n in enumerate(keys):
                shift(b, s, range(n), order[-n:])
            check(b, what=f"{spread} in order")


@pytest.mark.parametrize("Hq,Hkv", LAYOUTS)
@pytest.mark.parametrize("e", [-127, -60, 60, 118])
def test_values_all_small_or_all_large(Hq, Hkv, e):
    m = rows_of(Hq, Hkv)
    keys = [3, 140, 2500]
    b = Batch([m, 1, 1], keys, Hq, Hkv, D, 64, True, seed=e + 200)
    for s, n in enumerate(keys):
        shift(b, s, range(n), e)
    check(b, what=f"{e}")


def test_values_of_zero_leave_the_log_sum_exp():
    b = Batch([4, 1], [2500, 90], 8, 2, D, 64, True, seed=3)
    b.v.view(torch.uint8).zero_()
    b.vs.fill_(17)  # as fa_cache_write gives a row of zeros
    check(b, what="zeros")
    for s, n in enumerate((2500, 90)):
        shift(b, s, [n // 2], 110)
    check(b, what="zeros under different scales")
    b.v.view(torch.uint8)[int(b.table[0, 20])] = 0x30  # 0.5: a page of values in the first sequence
    check(b, what="zeros and values")


@pytest.mark.parametrize("Hq,Hkv", LAYOUTS)
@pytest.mark.parametrize("keys", [5, 700])
def test_the_log_sum_exp_does_not_depend_on_the_values(Hq, Hkv, keys):
    """Value scales from the least to the largest in one block, in either order, in so many sequences that whole
    blocks lie on one CTA: no row's log-sum-exp moves by more than rounding (references below 2^8 in size, so
    2^-16 for each of two, and 2e-5 for the sums)."""
    m, B = rows_of(Hq, Hkv), 150
    b = Batch([m] * B, [keys] * B, Hq, Hkv, D, 16, True, seed=keys)
    plain = np64(call(b.gpu())[1])
    pages = b.table[:, :-(-min(keys - 1, 300) // 16)].reshape(-1).long()
    for first, rest in ((17, 240), (240, 17)):
        b.vs.fill_(rest)
        b.vs[pages] = first
        lse = np64(call(b.gpu())[1])
        fa.check()
        dead = plain == -np.inf
        assert np.array_equal(dead, lse == -np.inf), (first, rest)
        assert np.abs(np.where(dead, 0, lse) - np.where(dead, 0, plain)).max() <= 6e-5, (first, rest)
