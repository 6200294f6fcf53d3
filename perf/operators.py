"""Work to measure on the paged KV cache: writing new rows into it (quantised to E4M3 on the way,
or as they are), reading rows back, and the attention of chunks of new tokens over it.

With ``own`` false every pass is elementary torch operations in 32 bits; with ``own`` true it is
the library's calls. A batch is ragged: sequence b has new[b] new tokens, packed one sequence
after another, which are the last of its keys[b] keys; its pages are scattered over the pool.
"""

import math

import torch

own = False


def listed():
    """Cases are made by _case; the comments say what each stands for in use."""
    return [
        # one decoding step's new rows of 64 sequences, quantised into their pages
        _case("write", "write_step", "1*64", "100+37*64", hkv=8, d=128, page=64, cache="e4m3"),
        # the rows of several prompts at once, ragged, quantised: a prefill step's cache write
        _case("write", "write_prompts", "4096,1777,8191,513,2048", "=", hkv=8, d=128, page=64, cache="e4m3"),
        # a few rows of narrow heads into small pages, unquantised
        _case("write", "write_narrow", "3,129,1,64", "19,129,400,1000", hkv=16, d=64, page=16, cache="bf16"),
        # whole contexts back from the quantised cache (to move or share a prefix)
        _case("read", "read_contexts", "8192,4097,6001,7168,5555,4608,8000,6144", "=", hkv=16, d=128, page=256,
              cache="e4m3"),
        # a short prefix back from small pages
        _case("read", "read_prefix", "331,77", "=", hkv=8, d=128, page=16, cache="e4m3"),
        # a first prompt of a few tokens: the smallest call
        _case("chunk", "chunk_tiny", "7", "=", hq=16, hkv=16, d=128, page=64, cache="bf16"),
        # a decoding step, a key/value head per query head, contexts of 4K to 8K keys
        _case("chunk", "step_bf16", "1*8", "8192,4096,5000,6777,7001,4444,8001,6100", hq=16, hkv=16, d=128, page=256,
              cache="bf16"),
        # a decoding step of many sequences with shared heads over the quantised cache
        _case("chunk", "step_e4m3", "1*48", "2000+290*48", hq=32, hkv=8, d=128, page=64, cache="e4m3"),
        # one sequence with a long context and a few new tokens: few rows, a long axis
        _case("chunk", "long_few", "16", "131072", hq=32, hkv=8, d=128, page=128, cache="bf16"),
        # long prompts processed in chunks over what is already cached
        _case("chunk", "prompt_bf16", "2048,1500", "16384,9001", hq=32, hkv=8, d=128, page=64, cache="bf16"),
        # chunks and decoding steps in one batch over the quantised cache, in a padded buffer
        _case("chunk", "mixed_e4m3", "512,1*6,333,1*7,64", "4096,300+531*6,2200,77+400*7,4000", hq=32, hkv=8, d=128,
              page=16, cache="e4m3", pad=37),
        # a window with the first tokens kept visible, narrow heads, a long context
        _case("chunk", "window_sinks", "1024,1000", "32768,20001", hq=16, hkv=16, d=64, page=32, cache="bf16",
              left=1023, sinks=4),
    ]


def _case(kind, name, new, keys, hkv, d, page, cache, hq=0, left=-1, right=-1, causal=True, sinks=0, pad=0):
    return {"kind": kind, "name": name, "new": new, "keys": keys, "hq": hq or hkv, "hkv": hkv, "d": d, "page": page,
            "cache": cache, "causal": causal, "left": left, "right": right, "sinks": sinks, "pad": pad}


def _counts(text):
    """"a,b" lists numbers, "a*n" repeats a, "a+s*n" counts a, a + s, ... (n of them)."""
    got = []
    for part in text.split(","):
        value, _, times = part.partition("*")
        start, _, step = value.partition("+")
        got += [int(start) + i * int(step or 0) for i in range(int(times or 1))]
    return got


def _lengths(case):
    new = _counts(case["new"])
    keys = new if case["keys"] == "=" else _counts(case["keys"])
    return new, keys


def _spread(rng, low, high):
    """Spread over the logarithm of the range, ends included."""
    return min(high, max(low, round(math.exp(rng.uniform(math.log(low), math.log(high))))))


def draw(rng):
    """One more case: sizes, head layouts, pages, masks and types over the ranges the list stands for."""
    while True:
        kind = rng.choice(["write", "read", "chunk", "chunk", "chunk"])
        d, page, cache = rng.choice([64, 128, 128]), rng.choice([16, 32, 48, 64, 128, 256]), rng.choice(["bf16", "e4m3"])
        hkv = rng.choice([1, 2, 4, 5, 8, 8, 16])
        batch = _spread(rng, 1, 48)
        pad = rng.choice([0, 0, 0, 5, 64])
        if kind == "read":
            cache = "e4m3"
        if kind != "chunk":
            if rng.random() < 0.3:
                new, keys = [1] * batch, [_spread(rng, 1, 4096) for _ in range(batch)]
            else:
                new = [_spread(rng, 1, 8192) for _ in range(batch)]
                keys = [n + rng.choice([0, 0, _spread(rng, 1, 500)]) for n in new]
            case = _case(kind, "", _text(new), _text(keys), hkv, d, page, cache)
            if sum(keys) * hkv * d > 2 ** 26 or sum(new) * hkv * d < 2 ** 10:
                continue
        else:
            use = rng.choice(["step", "step", "prompt", "mixed"])
            most = _spread(rng, 16, 32768)
            if use == "step":
                new = [rng.choice([1, 1, 1, 2, 4])] * batch
            elif use == "prompt":
                batch = min(batch, 4)
                new = [_spread(rng, 1, 2048) for _ in range(batch)]
            else:
                new = [_spread(rng, 2, 512) if rng.random() < 0.3 else 1 for _ in range(batch)]
            keys = [n + _spread(rng, 1, most) - 1 for n in new]
            left, right, sinks, causal = -1, -1, 0, True
            mask = rng.choice(["causal", "causal", "window", "window", "full"])
            if mask == "window":
                left, sinks = _spread(rng, 1, 4096), rng.choice([0, 1, 4, 64, 200])
            elif mask == "full":
                causal = False
            case = _case("chunk", "", _text(new), _text(keys), hkv, d, page, cache,
                         hq=hkv * rng.choice([1, 1, 2, 4, 4, 5, 7, 8, 16]), left=left, right=right, causal=causal,
                         sinks=sinks, pad=pad)
            scores = batch * case["hq"] * max(new) * max(keys)
            top = work(listed()[9])
            if case["hq"] > 64 or scores > 2 ** 31 or batch * max(keys) * hkv * d > 2 ** 30 or \
                    work(case)["flops"] > top["flops"]:
                continue
        del case["name"]
        return case


def _text(numbers):
    return ",".join(str(n) for n in numbers)


def prepare(case, seed):
    """Inputs on the GPU: new rows (queries, or keys and values to write), the paged cache with
    content, block table, lengths. Keys have a few channels larger than the others, as caches do."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    cpu = torch.Generator()
    cpu.manual_seed(seed)
    new, keys = _lengths(case)
    batch, page, hkv, d = len(new), case["page"], case["hkv"], case["d"]
    pages = [-(-n // page) for n in keys]
    widest, count = max(pages), sum(pages) + 2
    order = torch.randperm(count, generator=cpu)
    table = torch.full((batch, widest), -1, dtype=torch.int32)
    start = 0
    for b, n in enumerate(pages):
        table[b, :n] = order[start:start + n].to(torch.int32)
        start += n
    gain = torch.ones(d, device="cuda")
    gain[torch.randperm(d, generator=cpu)[:4].cuda()] = 4.0

    def rows(*shape, gains=None):
        x = torch.randn(*shape, d, device="cuda", generator=g, dtype=torch.bfloat16)
        return x if gains is None else x * gains.to(torch.bfloat16)

    total = sum(new) + case["pad"]
    state = {"case": case, "table": table.cuda(), "total": total, "most_new": max(new), "most_keys": max(keys),
             "lens": torch.tensor(keys, dtype=torch.int32, device="cuda"),
             "cu": torch.tensor([sum(new[:b]) for b in range(batch + 1)], dtype=torch.int32, device="cuda")}
    for name, gains in (("k", gain), ("v", None)):
        pool = rows(count, page, hkv, gains=gains)
        if case["cache"] == "e4m3":
            state[name + "_cache"], state[name + "_scale"] = _quantise(pool)
            state[name + "_scale"] = state[name + "_scale"].transpose(1, 2).contiguous()
            del pool
        else:
            state[name + "_cache"], state[name + "_scale"] = pool, None
    if case["kind"] == "chunk":
        state["q"] = rows(total, case["hq"])
        if case["pad"]:
            state["o"] = torch.zeros(total, case["hq"], d, device="cuda", dtype=torch.bfloat16)
            state["lse"] = torch.zeros(case["hq"], total, device="cuda")
    elif case["kind"] == "write":
        state["k_new"], state["v_new"] = rows(total, hkv, gains=gain), rows(total, hkv)
    return state


def _quantise(x):
    """E4M3 codes of the rows of x and their power-of-two scales: 2^e, the least with
    max |x| <= 448 * 2^e. Dividing by a power of two is exact, so each value is rounded once."""
    most = x.abs().amax(dim=-1).float()
    mantissa, exponent = torch.frexp(most)  # most = mantissa * 2^exponent, mantissa in [0.5, 1)
    e = (exponent - 9 + (mantissa > 0.875).int()).clamp(-110, 127)
    e = torch.where(most > 0, e, -110)
    codes = torch.ldexp(x.float(), -e[..., None]).to(torch.float8_e4m3fn)
    return codes, (e + 127).to(torch.uint8)


def run(state):
    """One pass: a cache write (the caches after it), a read (the rows) or the attention (o, lse)."""
    return globals()["_run_" + state["case"]["kind"]](state)


def _run_write(s):
    if own:
        import exact_attention_116_b200 as fa
        fa.cache_write_paged(s["k_new"], s["v_new"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s["cu"],
                             k_scale=s["k_scale"], v_scale=s["v_scale"])
    else:
        page, row, _ = _places(s)
        for x, cache, scale in (("k_new", "k_cache", "k_scale"), ("v_new", "v_cache", "v_scale")):
            if s[scale] is None:
                s[cache][page, row] = s[x]
            else:
                codes, scales = _quantise(s[x])
                s[cache].view(torch.uint8)[page, row] = codes.view(torch.uint8)
                s[scale][page, :, row] = scales
    caches = [s["k_cache"], s["v_cache"]]
    if s["k_scale"] is not None:
        caches += [s["k_scale"].view(torch.float8_e8m0fnu), s["v_scale"].view(torch.float8_e8m0fnu)]
    return caches


def _run_read(s):
    if own:
        import exact_attention_116_b200 as fa
        return fa.cache_read_paged(s["k_cache"], s["v_cache"], s["table"], s["lens"], s["cu"], s["total"],
                                   k_scale=s["k_scale"], v_scale=s["v_scale"])
    page, row, _ = _places(s)
    return [_values(s[n + "_cache"][page, row], s[n + "_scale"][page, :, row]).to(torch.bfloat16) for n in ("k", "v")]


def _places(s):
    """Page, row in the page and sequence of every packed new token."""
    token = torch.arange(s["total"], device="cuda", dtype=torch.int32)
    b = torch.searchsorted(s["cu"][1:], token, right=True).clamp(max=len(s["lens"]) - 1)
    position = s["lens"][b] - s["cu"][b + 1] + token
    return s["table"][b, position // s["case"]["page"]].long(), (position % s["case"]["page"]).long(), b


def _values(codes, scale):
    return codes.float() if scale is None else torch.ldexp(codes.float(), scale.int()[..., None] - 127)


def _run_chunk(s):
    c = s["case"]
    if own:
        import exact_attention_116_b200 as fa
        plan = dict(causal=c["causal"], window=(c["left"], c["right"]), sinks=c["sinks"], k_scale=s["k_scale"],
                    v_scale=s["v_scale"])
        if not c["pad"]:
            return fa.attention_chunk_paged(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s["cu"], **plan)
        fa.chunk_paged_into(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s["cu"], s["o"], s["lse"], **plan)
        return s["o"], s["lse"]
    hq, hkv, d, page = c["hq"], c["hkv"], c["d"], c["page"]
    batch, most, n = len(s["lens"]), s["most_new"], s["most_keys"]
    # the visible part of the cache, padded to the longest sequence; pages past a sequence read page 0
    key = torch.arange(n, device="cuda")
    where = s["table"][:, key // page].clamp(min=0).long()
    got = []
    for name in ("k", "v"):
        codes, scale = s[name + "_cache"][where, key % page], s[name + "_scale"]
        got.append(_values(codes, None if scale is None else scale[where, :, key % page]).permute(0, 2, 1, 3))
    # queries padded to the longest chunk: (batch, kv head, new * heads of the group, d)
    new = s["cu"][1:] - s["cu"][:-1]
    i = torch.arange(most, device="cuda")
    live = i < new[:, None]
    token = (s["cu"][:-1, None] + i).clamp(max=s["total"] - 1)
    q = s["q"][token].float().view(batch, most, hkv, hq // hkv, d).transpose(1, 2).reshape(batch, hkv, -1, d)
    scores = torch.matmul(q, got[0].transpose(2, 3)).mul_(1.0 / math.sqrt(d)).view(batch, hkv, most, hq // hkv, n)
    position = (s["lens"] - new)[:, None, None] + i[None, :, None]
    seen = (key < s["lens"][:, None, None]) & (position >= 0)
    if c["causal"]:
        seen = seen & (key <= position)
    if c["left"] >= 0:
        seen = seen & ((key >= position - c["left"]) | (key < c["sinks"]))
    scores.masked_fill_(~seen[:, None, :, None], -math.inf)
    peak = scores.amax(dim=-1, keepdim=True).clamp(min=-1e30)
    weights = scores.sub_(peak).exp_()
    total = weights.sum(dim=-1, keepdim=True)
    o = torch.matmul(weights.view(batch, hkv, -1, n), got[1]).view(batch, hkv, most, hq // hkv, d)
    o = (o / total.clamp(min=1e-30)).permute(0, 2, 1, 3, 4).reshape(batch, most, hq, d)
    lse = (peak + total.log()).squeeze(-1).permute(0, 2, 1, 3).reshape(batch, most, hq)
    out, stats = s.get("o"), s.get("lse")
    if out is None:
        out, stats = torch.empty_like(s["q"]), torch.empty(hq, s["total"], device="cuda")
    out[token[live]] = o[live].to(torch.bfloat16)
    stats[:, token[live]] = lse[live].t()
    return out, stats


def work(case):
    """Bytes: every input row that some output needs once, every output once. Operations: two
    products of d for each visible pair and query head."""
    new, keys = _lengths(case)
    d, hkv, hq = case["d"], case["hkv"], case["hq"]
    row = hkv * (2 * d if case["cache"] == "bf16" else d + 1)  # of one cache
    table = sum(-(-n // case["page"]) for n in keys) * 4 + 8 * len(keys)
    if case["kind"] != "chunk":
        return {"bytes": 2 * sum(new) * (row + hkv * d * 2) + table, "flops": 4 * sum(new) * hkv * d}
    pairs = touched = 0
    left, sinks = case["left"], case["sinks"]
    for s, n in zip(new, keys):
        first = n - s
        if not case["causal"] and left < 0:
            pairs, touched = pairs + s * n, touched + n
            continue
        low = max(0, first - left) if left >= 0 else 0
        touched += n - low + min(low, sinks)
        for p in range(first, n):
            top = p + 1 if case["causal"] else n
            at = max(0, p - left) if left >= 0 else 0
            pairs += top - at + min(at, sinks)
    return {"bytes": 2 * touched * row + 2 * sum(new) * hq * d * 2 + sum(new) * hq * 4 + table,
            "flops": 4 * d * hq * pairs}


def exact(case, seed):
    """What run() returns, in 64 bits from the definition, sequence by sequence."""
    s = prepare(case, seed)
    new, keys = _lengths(case)
    kind, page, d = case["kind"], case["page"], case["d"]
    quantised = case["cache"] == "e4m3"

    def row(name, b, first, last):  # rows [first, last) of a sequence, in 64 bits
        at = torch.arange(first, last, device="cuda")
        pages, rows = s["table"][b].long()[at // page], at % page
        x = s[name + "_cache"][pages, rows].to(torch.float64)
        if quantised:
            x = x * torch.exp2(s[name + "_scale"].to(torch.float64) - 127.0).transpose(1, 2)[pages, rows].unsqueeze(-1)
        return x

    starts = [sum(new[:b]) for b in range(len(new))]
    if kind == "read":
        return [torch.cat([row(n, b, keys[b] - new[b], keys[b]) for b in range(len(new))]) for n in ("k", "v")]
    if kind == "write":
        caches = [s["k_cache"].double(), s["v_cache"].double()]
        scales = [torch.exp2(s[n].double() - 127.0) for n in ("k_scale", "v_scale")] if quantised else []
        for b in range(len(new)):
            at = torch.arange(keys[b] - new[b], keys[b], device="cuda")
            pages, rows = s["table"][b].long()[at // page], at % page
            for i, name in enumerate(("k_new", "v_new")):
                x = s[name][starts[b]:starts[b] + new[b]].double()
                if quantised:
                    power = torch.ceil(torch.log2(x.abs().amax(-1) / 448.0))
                    power = torch.where(x.abs().amax(-1) > 448.0 * torch.exp2(power), power + 1, power)
                    power = torch.where(x.abs().amax(-1) <= 448.0 * torch.exp2(power - 1), power - 1, power)
                    unit = torch.exp2(power)
                    scales[i][pages, :, rows] = unit
                    x = x / unit[..., None]
                    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
                    x = torch.round(x / step) * step
                caches[i][pages, rows] = x
        return caches + scales
    hq, hkv = case["hq"], case["hkv"]
    o = torch.zeros(s["total"], hq, d, dtype=torch.float64, device="cuda")
    lse = torch.zeros(hq, s["total"], dtype=torch.float64, device="cuda")
    for b in range(len(new)):
        k, v = row("k", b, 0, keys[b]), row("v", b, 0, keys[b])
        j = torch.arange(keys[b], device="cuda")
        block = max(1, 2 ** 27 // (keys[b] * (hq // hkv)))
        for t in range(0, new[b], block):
            rows = slice(starts[b] + t, starts[b] + min(new[b], t + block))
            p = (keys[b] - new[b] + torch.arange(t, min(new[b], t + block), device="cuda"))[:, None]
            dark = torch.zeros_like(p >= j)
            if case["causal"]:
                dark = dark | (j > p)
            if case["left"] >= 0:
                dark = dark | ((j < p - case["left"]) & (j >= case["sinks"]))
            for h in range(hkv):
                heads = slice(h * (hq // hkv), (h + 1) * (hq // hkv))
                q = s["q"][rows, heads].double()
                x = torch.einsum("tgd,nd->gtn", q, k[:, h]) / math.sqrt(d)
                x = x.masked_fill(dark, -math.inf)
                lse[heads, rows] = torch.logsumexp(x, dim=-1)
                o[rows, heads] = torch.einsum("gtn,nd->tgd", torch.softmax(x, dim=-1), v[:, h])
    return o, lse
