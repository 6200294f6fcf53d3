"""Attention of ragged chunks over a paged cache on the GPU, against the float64 oracle (tolerances:
chunk_cases.py): head layouts, page sizes, types, masks, lengths around the tile borders, rows
without a key, strides, streams, graphs, and values in places that no row sees."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import exact_attention_116_b200 as fa
from chunk_cases import Batch, assert_close, call, np64

pytestmark = pytest.mark.gpu

MASKS = {"causal": (True, (-1, -1), 0), "full": (False, (-1, -1), 0), "window": (True, (100, -1), 0),
         "sinks": (True, (100, -1), 5), "both": (False, (90, 30), 0), "far": (True, (20, -1), 200),
         "own": (True, (0, -1), 0)}


def check(b, mask="causal", scale=None, what=""):
    causal, window, sinks = MASKS[mask]
    o, lse = call(b.gpu(), scale, causal, window, sinks)
    fa.check()
    ref = b.reference(b.d ** -0.5 if scale is None else scale, causal, window, sinks)
    assert_close(o, lse, ref, sum(b.new), f"{what} {mask}")
    return o, lse


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("mask", list(MASKS))
def test_masks(f8, d, mask):
    check(Batch([130, 1, 300, 0, 7], [700, 520, 300, 10, 128], 4, 2, d, 32, f8, seed=11), mask)


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (5, 5), (8, 2), (6, 2), (7, 1), (16, 1), (40, 2), (128, 1)])
def test_head_layouts(f8, Hq, Hkv):
    check(Batch([1, 50, 19], [257, 301, 19], Hq, Hkv, 128, 16, f8, seed=Hq))
    check(Batch([1, 2], [300, 5], Hq, Hkv, 64, 64, f8, seed=Hq), "sinks")


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("page", [16, 32, 48, 64, 80, 128, 256, 512])
def test_page_sizes(f8, page):
    check(Batch([1, 33, 140], [page + 1, 5 * page - 1, 300], 4, 2, 128, page, f8, seed=page))
    check(Batch([1, 3], [2 * page, 3 * page + 7], 4, 4, 64, page, f8, seed=page))


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 127, 128, 129, 255, 256, 257, 383, 385, 1000])
def test_lengths_around_the_tiles(n):
    for f8 in (False, True):
        check(Batch([n], [n], 2, 2, 128, 16, f8, seed=n), what=f"prompt {n}")
        check(Batch([1], [n], 2, 1, 64, 16, f8, seed=n), what=f"step {n}")
        check(Batch([min(n, 9)] * 3, [n, n + 1, n + 120], 4, 2, 128, 64, f8, seed=n), "sinks", what=f"few {n}")


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("new,keys", [([1], [30000]), ([3, 1], [9000, 20011]), ([200], [8200]), ([129, 64], [4000, 5001])])
def test_long_axes_are_split_and_joined(f8, new, keys):
    check(Batch(new, keys, 2, 1, 128, 128, f8, seed=sum(keys)))
    check(Batch(new, keys, 2, 2, 64, 64, f8, seed=sum(keys)), "full")


def test_many_sequences():
    rng = np.random.default_rng(0)
    keys = [int(x) for x in rng.integers(1, 400, size=700)]
    new = [int(min(n, m)) for n, m in zip(keys, rng.choice([0, 1, 1, 1, 2, 40], size=700))]
    check(Batch(new, keys, 2, 1, 64, 16, False, seed=1))
    check(Batch(new, keys, 4, 2, 128, 32, True, seed=2), "sinks")


@pytest.mark.parametrize("mask", list(MASKS))
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (4, 4), (4, 2), (6, 2), (8, 2), (5, 1), (7, 1), (16, 2), (16, 1)])
def test_few_rows_over_quantised_pages(mask, Hq, Hkv):
    """Blocks of up to 16 rows (tokens times heads), d = 128: steps, short speculative chunks, empty sequences."""
    most = max(1, 16 // (Hq // Hkv))
    check(Batch([1] * 5, [1, 130, 128, 777, 2000], Hq, Hkv, 128, 16, True, seed=Hq), mask)
    check(Batch([most, 0, 1, most], [most, 9, 300, 1500], Hq, Hkv, 128, 48, True, seed=Hq + 1, pad=2), mask)


def test_few_rows_cut_from_a_longer_chunk():
    check(Batch([50] + [0] * 3 + [1] * 20, [700] + [40] * 23, 4, 1, 128, 64, True, seed=3))
    check(Batch([60] + [1] * 59, [333] + [2] * 59, 8, 1, 128, 64, True, seed=4), "far")


@pytest.mark.parametrize("scale", [0.0, -0.3, 1.7, 1e-4, 30.0])
def test_few_rows_scales_and_dominant_keys(scale):
    b = Batch([4, 1], [400, 3000], 4, 2, 128, 16, True, seed=13)
    check(b, "causal", scale)
    b.q[:] = b.q * 30
    check(b, "sinks", scale if scale < 1 else 0.1)


def test_few_rows_references_move():
    """Scores and value scales that grow, fall and jump from tile to tile; queries of very different size."""
    b = Batch([3], [2000], 2, 1, 128, 16, False, seed=14, spare=0)
    rows = [(b.table[0, j // 16], j % 16) for j in range(2000)]
    for j, at in enumerate(rows):
        b.k[at] = (b.k[at].float() * (0.2 + j / 400)).bfloat16()
        b.v[at] = (b.v[at].float() * 2.0 ** ((j // 128) % 5 * 3 - 6)).bfloat16()
    b.q[0] = b.q[0] * 2.0 ** -20
    b.q[1, 0, 5:] = b.q[1, 0, 5:] * 2.0 ** -18
    from chunk_cases import quantise
    (b.k, b.ks), (b.v, b.vs), b.f8 = quantise(b.k), quantise(b.v), True
    check(b)
    check(b, "sinks")


@pytest.mark.parametrize("f8", [False, True])
def test_rows_without_a_key_or_a_place(f8):
    # more new rows than positions, an empty sequence with new rows, an empty cache
    b = Batch([9, 3, 150], [4, 0, 140], 4, 2, 128, 16, f8, seed=6)
    o, lse = check(b)
    assert (lse[:, :5] == -np.inf).all() and (lse[:, 9:12] == -np.inf).all() and (o[9:12] == 0).all()
    check(b, "own")
    check(Batch([9, 3], [4, 0], 1, 1, 64, 16, f8, seed=6), "full")


@pytest.mark.parametrize("scale", [0.0, -0.3, 1.7, 1e-4])
def test_scales(scale):
    check(Batch([40, 1], [200, 129], 4, 2, 64, 16, False, seed=9), "sinks", scale)
    check(Batch([40, 1], [200, 129], 4, 2, 128, 16, True, seed=9), "causal", scale)


def test_large_scores_and_a_dominant_key():
    b = Batch([20, 1], [400, 300], 4, 2, 128, 16, False, seed=12)
    b.q[:] = b.q * 30
    check(b)
    b.k[:, 3] = b.k[:, 3] * 20
    check(b, "sinks")


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_nothing_unseen_matters(f8, d):
    """NaN in the cache where no row sees it (past the end of a sequence inside its last page, left of
    the window outside the sinks), table entries of pages that no row sees, unused pages."""
    b = Batch([3, 1], [300, 333], 4, 2, d, 16, f8, seed=21)
    causal, window, sinks = True, (40, -1), 5
    ref = b.reference(d ** -0.5, causal, window, sinks)
    seen = torch.zeros(b.k.shape[0], 16, dtype=torch.bool)
    for s, (new, n) in enumerate(zip(b.new, b.keys)):
        for j in [*range(sinks), *range(n - new - 40, n)]:
            seen[b.table[s, j // 16], j % 16] = True
    for t in (b.k, b.v):
        if f8:
            t.view(torch.uint8)[~seen] = 0x7F
        else:
            t[~seen] = float("nan")
    if f8:
        for t in (b.ks, b.vs):
            t.transpose(1, 2)[~seen] = 255
    for s, n in enumerate(b.keys):
        for pg in range(b.table.shape[1]):
            if pg * 16 >= n or (pg > 0 and (pg + 1) * 16 <= n - b.new[s] - 40):
                b.table[s, pg] = 2 ** 31 - 1 if pg % 2 else -7
    o, lse = call(b.gpu(), None, causal, window, sinks)
    fa.check()
    assert_close(o, lse, ref, 4, "unseen")


def test_a_quantised_cache_is_its_values():
    """E4M3 pages give what bf16 pages of the values they stand for give, bit for bit."""
    b = Batch([40, 1, 7], [333, 700, 7], 8, 2, 128, 32, True, seed=30)
    t = b.gpu()
    u = dict(t)
    for n in "kv":
        x = t[n].float() * torch.exp2(t[n + "s"].transpose(1, 2).float() - 127)[..., None]
        u[n], u[n + "s"] = x.to(torch.bfloat16), None
    for got, ref in zip(call(t), call(u)):
        assert torch.equal(got, ref)
    fa.check()


@pytest.mark.parametrize("f8", [False, True])
def test_scales_over_the_whole_range(f8):
    """Rows from 2^-100 to 2^118: the scores of the small ones vanish, the weights are the values' own."""
    b = Batch([6], [64], 2, 1, 64, 16, False, seed=31)
    power = torch.linspace(-100, 118, 64).round()
    for j in range(64):
        b.v[b.table[0, j // 16], j % 16] = (b.v[b.table[0, j // 16], j % 16].float() * 2.0 ** float(power[j])).bfloat16()
    if f8:
        from chunk_cases import quantise
        (b.k, b.ks), (b.v, b.vs), b.f8 = quantise(b.k), quantise(b.v), True
    check(b, "full")


def test_padded_rows_are_left_as_they_were():
    for f8 in (False, True):
        for new in ([5, 1], [300, 20]):
            b = Batch(new, [500, 77], 4, 2, 128, 16, f8, pad=9, seed=41)
            t = b.gpu()
            o = torch.full_like(t["q"], 3.0)
            lse = torch.full((4, b.total), -8.0, device="cuda")
            t["q"][sum(new):] = float("nan")
            fa.chunk_paged_into(t["q"], t["k"], t["v"], t["table"], t["lens"], t["cu"], o, lse, None, True,
                                k_scale=t["ks"], v_scale=t["vs"])
            fa.check()
            assert (o[sum(new):] == 3.0).all() and (lse[:, sum(new):] == -8.0).all()
            assert_close(o, lse, b.reference(128 ** -0.5, True, (-1, -1), 0), sum(new), "padded")


def test_sliced_queries_and_a_caller_workspace():
    b = Batch([40, 1], [200, 700], 8, 2, 128, 16, False, seed=51)
    t = b.gpu()
    wide = torch.randn(b.total, 12, 128, device="cuda").bfloat16()
    wide[:, 2:10] = t["q"]
    ref = call(t)
    o, lse = torch.empty_like(t["q"]), torch.empty(8, b.total, device="cuda")
    ws = torch.full((fa.chunk_workspace_bytes(2, b.total, 8, 2, 128),), 255, dtype=torch.uint8, device="cuda")
    fa.chunk_paged_into(wide[:, 2:10], t["k"], t["v"], t["table"], t["lens"], t["cu"], o, lse, None, True, workspace=ws)
    fa.check()
    assert torch.equal(o, ref[0]) and torch.equal(lse, ref[1])
    check(b)


def test_agrees_with_the_decode_call():
    b = Batch([4, 4, 4], [300, 4, 1030], 3, 3, 128, 64, False, seed=61, stray=0)
    t = b.gpu()
    o, lse = call(t)
    o2, lse2 = fa.attention_decode_paged(t["q"].view(3, 4, 3, 128), t["k"], t["v"], t["table"], t["lens"], causal=True)
    fa.check()
    _, _, spread = b.reference(128 ** -0.5, True, (-1, -1), 0)
    tol = 2.02 * (2.0 ** -8 + 1e-3) * spread + 2.0 ** -7 * np64(o.abs()) + 2e-6  # each is within its own bound
    assert (np.abs(np64(o) - np64(o2.view_as(o))) <= tol).all()
    assert float((lse.view(3, 3, 4).transpose(0, 1) - lse2).abs().max()) <= 2e-3


@pytest.mark.parametrize("f8", [False, True])
def test_repeats_are_bitwise_equal_and_streams_do_not_disturb(f8):
    batches = [Batch([1] * 5, [4000, 1, 300, 2222, 900], 8, 2, 128, 64, f8, seed=70),
               Batch([300, 17], [1400, 5000], 8, 2, 128, 16, f8, seed=71),
               Batch([64], [16000], 4, 1, 64, 128, f8, seed=72)]
    data = [b.gpu() for b in batches]
    alone = [call(t) for t in data]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in data]
    out = []
    for rep in range(4):
        for t, s in zip(data, streams):
            s.wait_stream(torch.cuda.current_stream())
            out.append(call(t, stream=s))
    torch.cuda.synchronize()
    fa.check()
    for i, got in enumerate(out):
        for x, y in zip(got, alone[i % len(alone)]):
            assert torch.equal(x, y)


@pytest.mark.parametrize("f8", [False, True])
def test_a_step_in_a_graph_follows_its_inputs(f8):
    """A captured decoding step (write, attention, read back) replayed with other lengths, offsets and rows."""
    H, G, d, page, B = 2, 2, 128, 16, 4
    b = Batch([1] * B, [40, 300, 17, 129], H * G, H, d, page, f8, seed=80)
    t = b.gpu()
    kn, vn = (torch.randn(B, H, d, device="cuda").bfloat16() for _ in range(2))
    o, lse = torch.zeros_like(t["q"]), torch.zeros(H * G, B, device="cuda")
    back = [torch.zeros_like(kn) for _ in range(2)]
    ws = torch.empty(fa.chunk_workspace_bytes(B, B, H * G, H, d), dtype=torch.uint8, device="cuda")

    def step(o, lse, back, ws):
        fa.cache_write_paged(kn, vn, t["k"], t["v"], t["table"], t["lens"], t["cu"], t["ks"], t["vs"])
        fa.chunk_paged_into(t["q"], t["k"], t["v"], t["table"], t["lens"], t["cu"], o, lse, None, True,
                            k_scale=t["ks"], v_scale=t["vs"], workspace=ws)
        fa.cache_read_paged_into(t["k"], t["v"], t["table"], t["lens"], t["cu"], *back, t["ks"], t["vs"])

    step(o, lse, back, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(o, lse, back, ws)
    for rep in range(3):
        t["q"].normal_()
        kn.normal_()
        vn.normal_()
        t["lens"].copy_(torch.tensor([40 - rep, 299, 17 - 5 * rep, 129 - 60 * rep]))
        if rep == 2:
            t["cu"].copy_(torch.tensor([0, 1, 2, 2, 3]))  # the third sequence pauses
        graph.replay()
        torch.cuda.synchronize()
        fa.check()
        b.q, b.k, b.v, b.lens, b.cu = t["q"].cpu(), t["k"].cpu(), t["v"].cpu(), t["lens"].cpu(), t["cu"].cpu()
        if f8:
            b.ks, b.vs = t["ks"].cpu(), t["vs"].cpu()
        rows = int(b.cu[-1])
        assert_close(o, lse, b.reference(d ** -0.5, True, (-1, -1), 0), rows, f"replay {rep}")
        if not f8:
            assert torch.equal(back[0][:rows], kn[:rows]) and torch.equal(back[1][:rows], vn[:rows])


@pytest.mark.parametrize("f8", [False, True])
def test_serving_a_prompt_in_chunks_and_steps(f8):
    """A sequence written and attended in chunks and single steps beside another one equals plain attention
    over the rows the cache holds."""
    H, G, d, page, n = 2, 2, 128, 16, 301
    g = torch.Generator().manual_seed(90)
    q = torch.randn(2, n, H * G, d, generator=g).bfloat16().cuda()
    k, v = (torch.randn(2, n, H, d, generator=g).bfloat16().cuda() for _ in range(2))
    pages = -(-n // page)
    table = torch.randperm(2 * pages, generator=g).to(torch.int32).view(2, pages).cuda()
    shape = (2 * pages, page, H, d)
    dt = torch.float8_e4m3fn if f8 else torch.bfloat16
    kc, vc = torch.empty(shape, dtype=dt, device="cuda"), torch.empty(shape, dtype=dt, device="cuda")
    ks, vs = ((torch.empty(2 * pages, H, page, dtype=torch.float8_e8m0fnu, device="cuda") for _ in range(2)) if f8
              else (None, None))
    out = torch.zeros_like(q)
    done = [0, 0]
    for new in ([128, 1], [100, 150], [1, 0], [70, 1], [1, 148], [1, 1]):
        rows = [torch.arange(done[s], done[s] + new[s]) for s in range(2)]
        pick = [x.cuda() for x in rows]
        cu = torch.tensor([0, new[0], new[0] + new[1]], dtype=torch.int32, device="cuda")
        done = [done[s] + new[s] for s in range(2)]
        lens = torch.tensor(done, dtype=torch.int32, device="cuda")

        def packed(x):
            return torch.cat([x[s][pick[s]] for s in range(2)])

        fa.cache_write_paged(packed(k), packed(v), kc, vc, table, lens, cu, ks, vs)
        o, _ = fa.attention_chunk_paged(packed(q), kc, vc, table, lens, cu, causal=True, k_scale=ks, v_scale=vs)
        for s in range(2):
            out[s, pick[s]] = o[int(cu[s]):int(cu[s + 1])]
    fa.check()
    assert done == [n, n]
    cu = torch.tensor([0, n, 2 * n], dtype=torch.int32, device="cuda")
    rk, rv = fa.cache_read_paged(kc, vc, table, lens, cu, 2 * n, ks, vs)
    kf, vf = (x.view(2, n, H, 1, d).expand(2, n, H, G, d).reshape(2, n, H * G, d).contiguous() for x in (rk, rv))
    ref, _ = fa.attention_fwd(q, kf, vf, causal=True)
    fa.check()
    if not f8:
        assert torch.equal(rk.view_as(k), k) and torch.equal(rv.view_as(v), v)
    # both are within 2^-8 (spread) + 2^-8 |O| of the exact value, and spread <= 2 max |v|
    bound = 2 * (2.0 ** -8 + 1e-3) * 2 * float(vf.abs().max()) + 2.0 ** -7 * ref.float().abs()
    assert bool(((out.float() - ref.float()).abs() <= bound).all())
    assert float((out.float() - ref.float()).norm() / ref.float().norm()) <= 2.0 ** -7


def test_bad_pages_and_lengths_are_reported_and_not_followed():
    for what in ("page", "length", "offsets"):
        b = Batch([4, 1, 6], [40, 300, 60], 2, 2, 64, 16, False, seed=95)
        t = b.gpu()
        if what == "page":
            t["table"][1, 3] = t["k"].shape[0]
        elif what == "length":
            t["lens"][1] = -3
        else:
            t["cu"][3] = b.total + 1
        o, lse = call(t)
        with pytest.raises(fa.FaError):
            fa.check()
        good = slice(0, 4)
        ref = b.reference(64 ** -0.5, True, (-1, -1), 0)
        assert_close(o[good], lse[:, good], tuple(x[:, good] if i == 1 else x[good] for i, x in enumerate(ref)), 4, what)
        if what == "length":
            assert (o[4] == 0).all() and (lse[:, 4] == -np.inf).all()
        fa.check()  # the record was cleared


def test_caches_past_2_31_elements():
    H, d, page, num_pages = 8, 128, 256, 9000   # 2.36e9 elements
    k = torch.empty(num_pages, page, H, d, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    b = Batch([5], [500], 2 * H, H, d, page, False, seed=97, spare=0)
    t = b.gpu()
    for i, pg in enumerate((num_pages - 1, 8191)):
        src = int(b.table[0, i])
        k[pg], v[pg] = t["k"][src], t["v"][src]
        t["table"][0, i] = pg
    t["k"], t["v"] = k, v
    o, lse = call(t)
    fa.check()
    assert_close(o, lse, b.reference(d ** -0.5, True, (-1, -1), 0), 5, "far pages")


def test_no_rows():
    b = Batch([2], [2], 2, 1, 64, 16, False)
    t = b.gpu()
    t["q"], t["cu"] = t["q"][:0], torch.zeros_like(t["cu"])
    o, lse = call(t)
    fa.check()
    assert o.shape == (0, 2, 64) and lse.shape == (2, 0)
    t = b.gpu()
    t["cu"].zero_()  # rows, but none of a sequence
    o, lse = torch.ones_like(t["q"]), torch.ones(2, 2, device="cuda")
    fa.chunk_paged_into(t["q"], t["k"], t["v"], t["table"], t["lens"], t["cu"], o, lse)
    fa.check()
    assert (o == 1).all() and (lse == 1).all()


@pytest.mark.parametrize("f8", [False, True])
def test_the_log_sum_exp_is_an_fp32_output(f8):
    """Relative to its own size, over rows of a few keys and of many. A score is a sum of d exact products, each
    of the at most d additions off by 2^-24 of the partial sum (|partial sums| <= sum |q k| scale, here at most
    128 * 12 / 11 = 140 and 20 times a score's size at most), and is scaled and rounded twice more; the
    exponentials are off by 2.5e-7, a sum of n of them by (n / 64 + 64) 2^-24 (64 added in order, then tiles),
    the logarithm by 2^-22: 2e-5 in all for an LSE of order 1 and more."""
    for new, keys, Hq, Hkv in (([7], [7], 4, 4), ([1, 2, 3], [1, 5, 40], 8, 2), ([1, 1], [3000, 90], 4, 1),
                               ([150, 1], [700, 300], 4, 2)):
        b = Batch(new, keys, Hq, Hkv, 128, 16, f8, seed=len(new))
        o, lse = call(b.gpu())
        fa.check()
        ref = b.reference(128 ** -0.5, True, (-1, -1), 0)[1]
        err = np.linalg.norm(np64(lse) - ref) / np.linalg.norm(ref)
        assert err <= 2e-5, err
        assert np.abs(np64(lse) - ref).max() <= 2e-5 * max(1.0, np.abs(ref).max())


def test_results_on_a_side_stream_need_no_more_than_its_events():
    """Calls that allocate their results and workspace for another stream, while the current one frees and
    reuses memory of the same sizes."""
    b = Batch([200, 1], [900, 3000], 8, 2, 128, 32, False, seed=77)
    t = b.gpu()
    alone = call(t)
    rk, rv = fa.cache_read_paged(t["k"], t["v"], t["table"], t["lens"], t["cu"], b.total)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        junk = [torch.full_like(t["q"], 5.0) for _ in range(3)] + [torch.full((8, b.total), 9.0, device="cuda")]
        del junk
        o, lse = call(t, stream=side)
        k, v = fa.cache_read_paged(t["k"], t["v"], t["table"], t["lens"], t["cu"], b.total, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        same = torch.equal(o, alone[0]) and torch.equal(lse, alone[1]) and torch.equal(k, rk) and torch.equal(v, rv)
        assert same
        del o, lse, k, v
    fa.check()


def test_refusals_of_the_binding():
    b = Batch([4, 1], [40, 20], 4, 2, 64, 16, False, seed=5)
    f = Batch([4, 1], [40, 20], 4, 2, 64, 16, True, seed=5)
    t, u = b.gpu(), f.gpu()
    bad = [dict(q=t["q"].float()), dict(q=t["q"][:, :3]), dict(q=t["q"][..., ::2]), dict(k=t["k"].transpose(1, 2)),
           dict(k=t["k"][:, :8]), dict(v=t["v"].float()), dict(table=t["table"].long()), dict(lens=t["lens"][:1]),
           dict(cu=t["cu"][:2]), dict(table=t["table"][0]), dict(lens=t["lens"].cpu()), dict(ks=u["ks"], vs=None),
           dict(ks=u["ks"], vs=u["vs"]), dict(cu=t["cu"].repeat(2)[::2])]
    for kw in bad:
        with pytest.raises(ValueError):
            call(dict(t, **kw))
    for kw in (dict(ks=None, vs=None), dict(ks=u["ks"].transpose(1, 2)), dict(vs=u["vs"][:1]), dict(ks=u["ks"].int())):
        with pytest.raises(ValueError):
            call(dict(u, **kw))
    o, lse = torch.empty_like(t["q"]), torch.empty(4, 5, device="cuda")
    for oo, ll in ((o.float(), lse), (o[:4], lse), (o, lse.t().contiguous()), (o, lse.double()), (o, lse[:, ::2])):
        with pytest.raises(ValueError):
            fa.chunk_paged_into(t["q"], t["k"], t["v"], t["table"], t["lens"], t["cu"], oo, ll)
    with pytest.raises(fa.FaError):  # the output over the queries
        fa.chunk_paged_into(t["q"], t["k"], t["v"], t["table"], t["lens"], t["cu"], t["q"], lse)
    with pytest.raises(fa.FaError):  # a workspace that is too small
        fa.chunk_paged_into(t["q"], t["k"], t["v"], t["table"], t["lens"], t["cu"], o, lse,
                            workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises((ValueError, fa.FaError)):
        call(t, window=(2 ** 40, -1))
    with pytest.raises(fa.FaError):
        call(t, sinks=-1)
    rows = torch.zeros(5, 2, 64, dtype=torch.bfloat16, device="cuda")
    for kn, vn in ((rows, rows[:4]), (rows.half(), rows.half()), (rows[:, :1], rows[:, :1])):
        with pytest.raises(ValueError):
            fa.cache_write_paged(kn, vn, t["k"], t["v"], t["table"], t["lens"], t["cu"])
    with pytest.raises(fa.FaError):  # K and V written to the same pages
        fa.cache_write_paged(rows, rows.clone(), t["k"], t["k"], t["table"], t["lens"], t["cu"])
    fa.check()


@pytest.mark.parametrize("f8", [False, True])
def test_calls_that_depend_on_each_other_without_a_pause(f8):
    """Writes, attention, reads back, the decode and the plain forward one after another on a stream, each on the
    results of the one before, give what the same calls give with the device idle between them."""
    new, keys = [4, 4, 4], [300, 44, 1030]
    b = Batch(new, keys, 3, 3, 128, 64, f8, seed=61, stray=0)
    rows = [[torch.randn(b.total, 3, 128, generator=torch.Generator().manual_seed(100 + i)).bfloat16().cuda()
             for _ in range(3)] for i in range(8)]

    def run(pause):
        t, out = b.gpu(), []
        x = t["q"]
        for q, k, v in rows:
            steps = [lambda: fa.cache_write_paged(k, v, t["k"], t["v"], t["table"], t["lens"], t["cu"], t["ks"], t["vs"]),
                     lambda: call(dict(t, q=(x + q).bfloat16()))[0],
                     lambda: fa.cache_read_paged(t["k"], t["v"], t["table"], t["lens"], t["cu"], b.total, t["ks"], t["vs"])]
            got = []
            for step in steps:
                got.append(step())
                if pause:
                    torch.cuda.synchronize()
            x, (rk, rv) = got[1], got[2]
            y, _ = fa.attention_fwd(x.view(3, 4, 3, 128), rk.view(3, 4, 3, 128), rv.view(3, 4, 3, 128), causal=True)
            if pause:
                torch.cuda.synchronize()
            if not f8:
                z, _ = fa.attention_decode_paged(y, t["k"], t["v"], t["table"], t["lens"], causal=True)
                y = y + z
            x = y.reshape(b.total, 3, 128)
            if pause:
                torch.cuda.synchronize()
            out += [x, rk, rv]
        torch.cuda.synchronize()
        fa.check()
        return out + [t["k"].view(torch.uint8), t["v"].view(torch.uint8)]

    slow = run(True)
    for _ in range(3):
        for got, ref in zip(run(False), slow):
            assert torch.equal(got, ref)
