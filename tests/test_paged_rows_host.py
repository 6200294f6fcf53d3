"""The rows that a paged read writes: K and V rows may interleave (slices of one tensor), but not overlap. The
refusals are the host's (fake pointers are never dereferenced); no GPU is touched."""

from __future__ import annotations

import pytest

from exact_attention_116_b200 import binding, build

INVALID = 1
P, T = 0x7F0000000000, 1 << 42  # fake tensors far apart
H, D = 2, 64
W = H * D  # elements of a token's row


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


OVERLAPPING = [  # elements from K's first row to V's, rows apart, tokens
    (0, W, 10), (8, W, 10), (W, W, 10), (0, 3 * W, 10), (W // 2, 3 * W, 10), (-W // 2, 3 * W, 10), (3 * W, 3 * W, 10),
    (2 * W + 8, 3 * W, 10), (-2 * W - 8, 3 * W, 10), (27 * W, 3 * W, 10), (-27 * W - W // 2, 3 * W, 10),
    (W - 8, W + 8, 10), (W, W + 8, 10), (0, 3 * W, 1), (W // 2, 3 * W, 1),
]


@pytest.mark.parametrize("offset,stride,total", OVERLAPPING)
def test_overlapping_outputs_are_refused(lib, offset, stride, total):
    args = (P, P + T, None, None, P + 2 * T, P + 3 * T, P + 4 * T)
    assert lib.fa_cache_read(*args, P + 5 * T, P + 5 * T + 2 * offset, stride, 2, total, H, D, 16, 64, 8, None) == INVALID


def rows_meet(offset, stride, total):
    spans = [[(i * stride + base, i * stride + base + W) for i in range(total)] for base in (0, offset)]
    return any(a < d and c < b for a, b in spans[0] for c, d in spans[1])


@pytest.mark.parametrize("stride", [W, W + 8, 2 * W, 2 * W + 8, 3 * W, 5 * W - 8])
@pytest.mark.parametrize("total", [1, 2, 7])
def test_the_rule_is_exact(stride, total):
    """Rows `stride` apart, their spans meeting: they overlap exactly when the offset's remainder is within a
    row of a multiple of the stride."""
    for offset in range(-total * stride - 2 * W, total * stride + 2 * W, 8):
        span = (total - 1) * stride + W
        spans_meet = offset < span and -offset < span
        low = abs(offset) % stride
        assert rows_meet(offset, stride, total) == (spans_meet and (low < W or low > stride - W))
