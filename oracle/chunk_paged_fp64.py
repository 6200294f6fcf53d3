"""Ragged chunks over a paged cache in float64: writing rows (quantised to E4M3 with a power-of-two
scale per row, or as they are), reading them back, and the attention of the chunks.

TEST INFRASTRUCTURE, as the rest of this package: the CUDA library never calls it, and it shares
no code with the CUDA path.

Sequence b's new rows are the packed rows [cu[b], cu[b + 1]); they are the last new_b of its
seqlens[b] positions. Layout: pages (num_pages, page_size, H, d), scale bytes
(num_pages, H, page_size), packed rows (total, H, d), LSE (Hq, total).
"""

from __future__ import annotations

import numpy as np

from oracle.fp8_e4m3 import decode_e4m3

E4M3_VALUES = np.sort(decode_e4m3(np.arange(127)))  # the finite magnitudes, 0 first
MIN_EXPONENT = -110
TOP_EXPONENT = 120


def quantise_rows(x):
    """(codes, scale bytes) of the rows (last axis) of x: nearest E4M3 values of x * 2^-e, ties to the even
    code, with the least e >= -110 such that max |x| <= 448 * 2^e. Rows with a NaN or an infinity: scale 255,
    code 0x7F. With e = 120 codes stop at 240: 256 * 2^120 is beyond bf16."""
    x = np.asarray(x, dtype=np.float64)
    flat = x.reshape(-1, x.shape[-1])
    codes = np.zeros(flat.shape, dtype=np.uint8)
    scale = np.zeros(flat.shape[0], dtype=np.uint8)
    for r, row in enumerate(flat):
        if not np.isfinite(row).all():
            codes[r], scale[r] = 0x7F, 255
            continue
        e = MIN_EXPONENT
        while np.abs(row).max() > 448.0 * 2.0 ** e:
            e += 1
        v = np.abs(row) * 2.0 ** -e
        hi = np.clip(np.searchsorted(E4M3_VALUES, v), 1, 126)  # E4M3_VALUES[hi - 1] <= v <= E4M3_VALUES[hi]
        below, above = v - E4M3_VALUES[hi - 1], E4M3_VALUES[hi] - v
        pick = np.where((below < above) | ((below == above) & ((hi - 1) % 2 == 0)), hi - 1, hi)
        if e == TOP_EXPONENT:
            pick = np.minimum(pick, 0x77)
        codes[r] = pick + np.where(np.signbit(row), 128, 0)
        scale[r] = e + 127
    return codes.reshape(x.shape), scale.reshape(x.shape[:-1])


def row_values(codes, scale):
    """float64 values of quantised rows (NaN for scale byte 255)."""
    unit = np.where(np.asarray(scale) == 255, np.nan, np.exp2(np.asarray(scale, dtype=np.float64) - 127.0))
    return decode_e4m3(codes) * unit[..., None]


def place(block_table, seqlens, cu, page_size, b, i):
    """(page, row) of new row i of sequence b, or None for a negative position."""
    pos = int(seqlens[b]) - int(cu[b + 1] - cu[b]) + i
    return None if pos < 0 else (int(block_table[b, pos // page_size]), pos % page_size)


def sequence_rows(cache, scale, block_table, b, n):
    """(n, H, d) float64 rows of sequence b, with zeros for pages outside the pool."""
    num_pages, page_size, H, d = cache.shape
    out = np.zeros((n, H, d))
    for j0 in range(0, n, page_size):
        page, m = int(block_table[b, j0 // page_size]), min(page_size, n - j0)
        if 0 <= page < num_pages:
            rows = cache[page, :m]
            out[j0:j0 + m] = row_values(rows, scale[page, :, :m].T) if scale is not None else rows
    return out


def visible(pos, n, causal, win_l, win_r, sinks):
    """(rows, n) mask: row at position p sees key j."""
    j, p = np.arange(n)[None, :], np.asarray(pos)[:, None]
    right = 0 if causal else win_r
    see = (p >= 0) & (j < n)
    if right >= 0:
        see = see & (j <= p + right)
    if win_l >= 0:
        see = see & ((j >= p - win_l) | (j < sinks))
    return see


def chunk_forward(q, k_cache, v_cache, block_table, seqlens, cu, scale, causal=False, win_l=-1, win_r=-1, sinks=0,
                  k_scale=None, v_scale=None):
    """(O, LSE, spread): spread = sum_j softmax_j |v_j - O|, by which a relative error of the weights moves O."""
    q = np.asarray(q, dtype=np.float64)
    total, Hq, d = q.shape
    H = k_cache.shape[2]
    o, lse, spread = np.zeros((total, Hq, d)), np.full((Hq, total), -np.inf), np.zeros((total, Hq, d))
    for b in range(len(seqlens)):
        c0, c1, n = int(cu[b]), int(cu[b + 1]), int(seqlens[b])
        if c1 == c0 or n == 0:
            continue
        k = sequence_rows(k_cache, k_scale, block_table, b, n)
        v = sequence_rows(v_cache, v_scale, block_table, b, n)
        see = visible(np.arange(n - (c1 - c0), n), n, causal, win_l, win_r, sinks)
        for h in range(Hq):
            kv = h // (Hq // H)
            keys, vals = np.where(see.any(0)[:, None], k[:, kv], 0.0), np.where(see.any(0)[:, None], v[:, kv], 0.0)
            s = np.where(see, scale * (q[c0:c1, h] @ keys.T), -np.inf)
            m = s.max(axis=1, keepdims=True)
            w = np.where(see, np.exp(s - np.where(np.isfinite(m), m, 0.0)), 0.0)
            z = w.sum(axis=1, keepdims=True)
            w = np.divide(w, z, out=np.zeros_like(w), where=z > 0)
            o[c0:c1, h] = w @ vals
            with np.errstate(divide="ignore"):
                lse[h, c0:c1] = np.where(z[:, 0] > 0, m[:, 0] + np.log(z[:, 0]), -np.inf)
            for i in range(c1 - c0):
                spread[c0 + i, h] = w[i] @ np.abs(vals - o[c0 + i, h])
    return o, lse, spread
