"""Ragged chunks over a paged cache for the GPU tests: inputs, the float64 oracle's answer and the
tolerance of the attention.

The kernel's O is sum_j w_j v_j / sum_j w_j with weights rounded to bf16: w_j = p_j (1 + e_j),
|e_j| <= u = 2^-8 (bf16 has 8 significant bits: half a step is 2^-8 of the value), so to first
order |dO| <= u * spread with spread = sum_j p_j |v_j - O|. Scores carry the error of fp32 sums of
d products and exponentials one of 7.5e-5 at most; both move p_j by a relative amount well below
1e-3 (the bound the forward's tests put on the log-sum-exp), which adds 1e-3 * spread. O is rounded
once to bf16, 2^-8 |O|; 1.01 covers the second-order terms, 1e-6 sums of subnormal size.
"""

from __future__ import annotations

import numpy as np
import torch

import exact_attention_116_b200 as fa
from oracle import chunk_paged_fp64 as oracle

LSE_TOL = 1e-3


def np64(t):
    return None if t is None else t.detach().to("cpu", torch.float64).numpy()


def quantise(pool):
    """E4M3 codes and scale bytes of (num_pages, page_size, H, d) rows with elementary operations."""
    most = pool.float().abs().amax(-1)
    m, x = torch.frexp(most)
    e = torch.where(most > 0, (x - 9 + (m > 0.875).int()).clamp(min=-110), -110)
    codes = torch.ldexp(pool.float(), -e[..., None]).to(torch.float8_e4m3fn)
    return codes, (e + 127).to(torch.uint8).transpose(1, 2).contiguous()


class Batch:
    """Inputs on the CPU: new[b] query rows at the end of keys[b] keys, pages scattered over the pool and
    table entries past a sequence's pages that must not be followed."""

    def __init__(self, new, keys, Hq, Hkv, d, page, f8=False, pad=0, seed=0, spare=2, stray=-5):
        g = torch.Generator().manual_seed(seed)
        self.new, self.keys, self.f8, self.d = new, keys, f8, d
        pages = [-(-n // page) for n in keys]
        count = sum(pages) + spare
        order = torch.randperm(count, generator=g)
        self.table = torch.full((len(new), max(1, max(pages)) + 1), stray, dtype=torch.int32)
        at = 0
        for b, m in enumerate(pages):
            self.table[b, :m] = order[at:at + m].to(torch.int32)
            at += m
        self.total = sum(new) + pad
        self.lens = torch.tensor(keys, dtype=torch.int32)
        self.cu = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32)
        self.q = torch.randn(self.total, Hq, d, generator=g).to(torch.bfloat16)
        pools = [torch.randn(count, page, Hkv, d, generator=g).to(torch.bfloat16) for _ in range(2)]
        self.ks = self.vs = None
        if f8:
            (self.k, self.ks), (self.v, self.vs) = (quantise(p) for p in pools)
        else:
            self.k, self.v = pools

    def gpu(self, device="cuda"):
        return {n: None if getattr(self, n) is None else getattr(self, n).to(device)
                for n in ("q", "k", "v", "table", "lens", "cu", "ks", "vs")}

    def reference(self, scale, causal, window, sinks):
        def codes(t):
            return t.view(torch.uint8).numpy() if self.f8 else np64(t)

        def scales(t):
            return None if t is None else t.numpy()

        return oracle.chunk_forward(np64(self.q), codes(self.k), codes(self.v), self.table.numpy(), self.lens.numpy(),
                                    self.cu.numpy(), scale, causal, *window, sinks, scales(self.ks), scales(self.vs))


def call(t, scale=None, causal=True, window=(-1, -1), sinks=0, **more):
    return fa.attention_chunk_paged(t["q"], t["k"], t["v"], t["table"], t["lens"], t["cu"], scale, causal, window, sinks,
                                    t["ks"], t["vs"], **more)


def assert_close(o, lse, ref, rows, what=""):
    """rows: the packed rows that belong to a sequence."""
    o_ref, lse_ref, spread = (x[:rows] if i != 1 else x[:, :rows] for i, x in enumerate(ref))
    o, lse = np64(o)[:rows], np64(lse)[:, :rows]
    dead = ~np.isfinite(lse_ref)
    assert np.array_equal(dead, lse == -np.inf), f"{what}: rows without a key"
    assert (o.transpose(1, 0, 2)[dead] == 0).all(), f"{what}: O of rows without a key"
    e_lse = np.abs(np.where(dead, 0, lse) - np.where(dead, 0, lse_ref)).max()
    assert e_lse <= LSE_TOL, f"{what}: LSE error {e_lse:.3e}"
    tol = 1.01 * (2.0 ** -8 + 1e-3) * spread + 2.0 ** -8 * np.abs(o_ref) + 1e-6
    worst = (np.abs(o - o_ref) / tol).max()
    assert np.isfinite(o).all() and worst <= 1.0, f"{what}: O error {worst:.3f} of its bound"
