"""Pins of the float64 oracle of ragged chunks over a paged cache: hand-worked rows, the definitions
by brute force, and agreement with the decode and plain attention oracles where they overlap."""

from __future__ import annotations

import numpy as np
import pytest

from oracle import attention_fp64, chunk_paged_fp64 as oracle, decode_paged_fp64
from oracle.fp8_e4m3 import decode_e4m3


def test_quantise_hand_worked():
    # max 448: e = 0, so 1.0625 = 17/16 lies midway between 1 and 1.125: to the even code, 1
    codes, s = oracle.quantise_rows([[448.0, 1.0625, -1.1875, 0.0]])
    assert s[0] == 127 and decode_e4m3(codes)[0].tolist() == [448.0, 1.0, -1.25, 0.0]
    # just above 448: e = 1
    codes, s = oracle.quantise_rows([[450.0, 1.0]])
    assert s[0] == 128 and oracle.row_values(codes, s)[0].tolist() == [448.0, 1.0]
    # 1 = 256 * 2^-8 and 1.75 = 448 * 2^-8, but 1.76 needs 2^-7
    assert [int(oracle.quantise_rows([[a]])[1][0]) for a in (1.0, 1.75, 1.76)] == [119, 119, 120]
    assert int(oracle.quantise_rows([[0.0, 0.0]])[1][0]) == 17
    assert np.isnan(oracle.row_values(*oracle.quantise_rows([[1.0, np.inf]]))).all()


def test_quantise_is_nearest_and_reading_back_is_idempotent():
    rng = np.random.default_rng(1)
    x = rng.normal(size=(50, 64)) * np.exp2(rng.integers(-30, 30, size=(50, 1)))
    codes, s = oracle.quantise_rows(x)
    y = oracle.row_values(codes, s)
    unit = np.exp2(s.astype(float) - 127)[:, None]
    best = np.abs(np.abs(x / unit)[..., None] - oracle.E4M3_VALUES).min(-1)
    assert np.allclose(np.abs(x - y) / unit, best, rtol=0, atol=1e-12)
    assert (np.abs(x).max(1) <= 448 * unit[:, 0]).all() and (np.abs(x).max(1) > 448 * unit[:, 0] / 2).all()
    again = oracle.row_values(*oracle.quantise_rows(y))
    assert np.array_equal(again, y)


@pytest.mark.parametrize("causal,win,sinks", [(True, (-1, -1), 0), (False, (3, 2), 0), (True, (4, -1), 2),
                                              (False, (-1, -1), 5), (False, (0, -1), 1)])
def test_visible_by_definition(causal, win, sinks):
    pos, n = np.arange(-2, 9), 9
    see = oracle.visible(pos, n, causal, *win, sinks)
    for r, p in enumerate(pos):
        for j in range(n):
            right = 0 if causal else win[1]
            want = p >= 0 and (right < 0 or j <= p + right) and (win[0] < 0 or j >= p - win[0] or j < sinks)
            assert bool(see[r, j]) == want


def _cache(rng, lens, page, H, d):
    pages = [-(-n // page) for n in lens]
    table = np.full((len(lens), max(1, max(pages))), -1, dtype=np.int32)
    order = rng.permutation(sum(pages) + 1)
    at = 0
    for b, m in enumerate(pages):
        table[b, :m] = order[at:at + m]
        at += m
    return rng.normal(size=(sum(pages) + 1, page, H, d)), rng.normal(size=(sum(pages) + 1, page, H, d)), table


@pytest.mark.parametrize("causal,win", [(True, (-1, -1)), (False, (5, 3)), (False, (-1, -1))])
def test_agrees_with_the_decode_oracle(causal, win):
    rng = np.random.default_rng(2)
    lens, Sq, H, d = np.array([20, 3, 33]), 3, 2, 8
    kc, vc, table = _cache(rng, lens, 16, H, d)
    q = rng.normal(size=(3, Sq, H, d))
    o, lse, _ = oracle.chunk_forward(q.reshape(-1, H, d), kc, vc, table, lens, np.arange(4) * Sq, 0.3, causal, *win)
    o_ref, lse_ref = decode_paged_fp64.decode_forward(q, kc, vc, table, lens, 0.3, causal, *win)
    assert np.allclose(o.reshape(o_ref.shape), o_ref) and np.allclose(lse.reshape(H, 3, Sq).transpose(1, 0, 2), lse_ref)


def test_grouped_heads_are_repeated_heads_and_a_whole_prompt_is_plain_attention():
    rng = np.random.default_rng(3)
    n, H, G, d = 21, 2, 3, 8
    kc, vc, table = _cache(rng, [n], 16, H, d)
    q = rng.normal(size=(n, H * G, d))
    o, lse, _ = oracle.chunk_forward(q, kc, vc, table, [n], [0, n], 0.4, True)
    k, v = (np.repeat(oracle.sequence_rows(c, None, table, 0, n), G, axis=1) for c in (kc, vc))
    o_ref, lse_ref = attention_fp64.attention_forward(q[None], k[None], v[None], 0.4, True)
    assert np.allclose(o, o_ref[0]) and np.allclose(lse, lse_ref[0])


def test_a_window_with_sinks_by_hand():
    # four keys of equal score; the row at position 3 with a window of one key back and one sink sees 0, 2, 3
    cache = np.zeros((1, 16, 1, 1))
    vals = np.zeros((1, 16, 1, 1))
    vals[0, :4, 0, 0] = [1.0, 10.0, 100.0, 1000.0]
    o, lse, spread = oracle.chunk_forward(np.ones((1, 1, 1)), cache, vals, np.zeros((1, 1), int), [4], [0, 1], 1.0,
                                          True, 1, -1, 1)
    assert np.isclose(o[0, 0, 0], 1101.0 / 3) and np.isclose(lse[0, 0], np.log(3.0))
    assert np.isclose(spread[0, 0, 0], (366 + 267 + 633) / 3)
