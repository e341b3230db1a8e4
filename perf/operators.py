"""The position and score operators of this library, as they are measured.

Three operators: rotary positions applied to new queries and keys on their way
into the cache (``rope_append``), attention of one new token per sequence whose
scores are capped, biased by distance or masked (``*_decode_attention_scored``),
and the same for chunks of new tokens (``*_prefill_attention_scored``).

``own`` is set by whoever measures: true runs the library's calls, false their
plain form in elementary torch operations.
"""
import math
import random

import torch

own = False

D = 128  # head size of the library


# ------------------------------------------------------------------ the cases

def _rope(name, tokens, hq, hkv, rotary, interleaved, scaling, far, pad=0, block=16, salt=1):
    return {"name": name, "op": "rope", "tokens": tokens, "q_heads": hq, "kv_heads": hkv,
            "rotary": rotary, "interleaved": interleaved, "scaling": scaling, "far": far,
            "pad": pad, "block": block, "salt": salt}


def _decode(name, layout, batch, hq, hkv, ctx_min, ctx_max, block=16, softcap=0.0, window=0,
            slopes=False, documents=0, salt=1):
    return {"name": name, "op": "decode", "layout": layout, "batch": batch, "q_heads": hq,
            "kv_heads": hkv, "ctx_min": ctx_min, "ctx_max": ctx_max, "block": block,
            "softcap": softcap, "window": window, "slopes": slopes, "documents": documents,
            "salt": salt}


def _prefill(name, layout, batch, hq, hkv, new_min, new_max, cached_min, cached_max, block=16,
             softcap=0.0, window=0, slopes=False, documents=0, prefix=False, salt=1):
    return {"name": name, "op": "prefill", "layout": layout, "batch": batch, "q_heads": hq,
            "kv_heads": hkv, "new_min": new_min, "new_max": new_max, "cached_min": cached_min,
            "cached_max": cached_max, "block": block, "softcap": softcap, "window": window,
            "slopes": slopes, "documents": documents, "prefix": prefix, "salt": salt}


def listed():
    return [
        # one sequence's next token: only the call's latency counts
        _rope("rope 1 token", 1, 32, 8, 128, False, "none", 8192),
        # a decode batch at far positions of a long-context server, half of each head rotated
        _rope("rope 64 far half heads", 64, 56, 8, 64, True, "parts", 1 << 20),
        # a ragged step padded to a fixed size for a captured graph, an odd rotary size
        _rope("rope 333 padded odd size", 333, 32, 4, 50, False, "linear", 30000, pad=13, block=48),
        # whole prompts of a batch: bandwidth
        _rope("rope 16384 prompt tokens", 16384, 32, 8, 128, False, "smooth", 131072),

        # one chat alone on the machine, capped scores: latency
        _decode("decode b1 capped", "paged", 1, 32, 8, 1000, 1000, softcap=50.0),
        # a full ragged batch of a model whose layers see a window, capped scores
        _decode("decode b64 capped window", "paged", 64, 32, 8, 16, 8192, softcap=50.0,
                window=1024),
        # requests in contiguous rows, scores biased by distance, 8 query heads per KV head
        _decode("decode b32 slopes contig", "contig", 32, 32, 4, 100, 4095, slopes=True),
        # packed documents of a large batch at full contexts, 7 query heads per KV head: bandwidth
        _decode("decode b128 documents capped", "paged", 128, 56, 8, 8000, 8192, block=32,
                softcap=30.0, documents=6000),

        # a few short chunks among running sequences: latency
        _prefill("prefill 4 short chunks", "paged", 4, 32, 8, 1, 40, 0, 500, softcap=50.0,
                 window=256),
        # fresh prompts under capped scores: tensor cores and the exponentials
        _prefill("prefill 8 x 2048 capped", "paged", 8, 32, 8, 2048, 2048, 0, 0, softcap=50.0),
        # long prompts of a layer that sees a window
        _prefill("prefill 2 x 8192 window", "contig", 2, 32, 8, 8100, 8192, 0, 0, window=1024),
        # chunks after cached positions, distance bias, packed documents, bidirectional prefixes
        _prefill("prefill chunks all masks", "paged", 6, 56, 8, 100, 1500, 0, 3000, block=32,
                 slopes=True, documents=1024, prefix=True),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    hq, hkv = rng.choice([(32, 8), (32, 4), (56, 8), (4, 4), (20, 4), (10, 2), (6, 1)])
    salt = rng.randrange(1, 1 << 30)
    op = rng.choice(["rope", "decode", "prefill"])
    if op == "rope":
        tokens = _log(rng, 1, 12000)
        return _unnamed(_rope("", tokens, hq, hkv, 2 * rng.randint(1, 64), rng.random() < 0.5,
                              rng.choice(["none", "linear", "parts", "smooth"]),
                              _log(rng, 100, 1 << 20), rng.choice([0, 0, min(3, tokens - 1)]),
                              rng.choice([16, 32, 48, 128]), salt))
    cap = rng.choice([0.0, 15.0, 30.0, 50.0])
    window = rng.choice([0, 0, _log(rng, 1, 4096)])
    slopes = rng.random() < 0.3
    documents = rng.choice([0, 0, _log(rng, 64, 4096)])
    layout = rng.choice(["paged", "contig"])
    block = rng.choice([16, 32, 64, 128])
    if op == "decode":
        top = _log(rng, 1, 8192)
        return _unnamed(_decode("", layout, _log(rng, 1, 100), hq, hkv, max(1, top // rng.choice([1, 3, 100])),
                                top, block, cap, window, slopes, documents, salt))
    new = _log(rng, 1, 4096)
    cached = rng.choice([0, _log(rng, 1, 4096)])
    batch = max(1, min(_log(rng, 1, 32), (1 << 24) // (new * (new + cached))))
    return _unnamed(_prefill("", layout, batch, hq, hkv, max(1, new // rng.choice([1, 4])), new,
                             cached // rng.choice([1, 4]), cached, block, cap, window, slopes,
                             documents, rng.random() < 0.3, salt))


def _unnamed(case):
    return {k: v for k, v in case.items() if k != "name"}


# ------------------------------------------ what a case's sequences look like

def _lengths(case, low, high, salt):
    rng = random.Random(case["salt"] * 7919 + salt)
    return [max(low, min(high, _log(rng, max(low, 1), max(high, 1)))) if high else 0
            for _ in range(case["batch"])]


def _ctx_and_new(case):
    """Per sequence: positions in the cache (new ones included), new positions."""
    if case["op"] == "decode":
        return _lengths(case, case["ctx_min"], case["ctx_max"], 1), [1] * case["batch"]
    new = _lengths(case, case["new_min"], case["new_max"], 2)
    cached = _lengths(case, case["cached_min"], case["cached_max"], 3)
    return [n + c for n, c in zip(new, cached)], new


def _first_keys(case, ctx, new):
    """The start of each new token's document: lengths around case["documents"]."""
    out = []
    for i, (c, n) in enumerate(zip(ctx, new)):
        rng = random.Random(case["salt"] * 104729 + i)
        starts = [0]
        while starts[-1] < c:
            starts.append(starts[-1] + _log(rng, max(1, case["documents"] // 4), 2 * case["documents"]))
        k = 0
        for p in range(c - n, c):
            while starts[k + 1] <= p:
                k += 1
            out.append(starts[k])
    return out


def _prefixes(case, ctx):
    rng = random.Random(case["salt"] * 31337)
    return [rng.randint(0, c) for c in ctx]


def _ranges(case):
    """Per sequence and new token: (first visible key, last visible key + 1)."""
    ctx, new = _ctx_and_new(case)
    first = iter(_first_keys(case, ctx, new)) if case["documents"] else None
    prefix = _prefixes(case, ctx) if case.get("prefix") else [0] * len(ctx)
    out = []
    for c, n, x in zip(ctx, new, prefix):
        rows = []
        for p in range(c - n, c):
            low = next(first) if first else 0
            if case["window"]:
                low = max(low, p - case["window"] + 1)
            rows.append((low, max(p + 1, min(x, c))))
        out.append(rows)
    return out


def work(case):
    hq, hkv = case["q_heads"], case["kv_heads"]
    if case["op"] == "rope":
        t, p = case["tokens"], case["pad"]
        # q in and out, k and v in, k and v into the cache; position and slot of each token
        size = t * hq * D * 2 * 2 + (t - p) * 2 * hkv * D * 2 * 2 + t * 12
        return {"bytes": size, "flops": t * (hq + hkv) * case["rotary"] * 3}
    keys = pairs = tokens = 0
    for rows in _ranges(case):
        keys += max(b for _, b in rows) - min(a for a, _ in rows)
        pairs += sum(b - a for a, b in rows)
        tokens += len(rows)
    return {"bytes": keys * hkv * D * 2 * 2 + tokens * hq * D * 2 * 2,
            "flops": pairs * hq * D * 4}


# ------------------------------------------------------------------- the inputs

SCALING = {  # as long-context checkpoints carry them
    "none": None,
    "linear": {"kind": "linear", "factor": 4.0},
    "parts": {"kind": "parts", "factor": 16.0, "original": 8192, "beta_fast": 32.0,
              "beta_slow": 1.0},
    "smooth": {"kind": "smooth", "factor": 8.0, "original": 8192, "low": 1.0, "high": 4.0},
}
THETA = 500000.0


def _frequencies(rotary, scaling):
    """(radians per position of each pair in 64 bits, factor on cos and sin)."""
    half = rotary // 2
    inv = [THETA ** (-2.0 * i / rotary) for i in range(half)]
    s = SCALING[scaling]
    if s is None:
        return inv, 1.0
    f = s["factor"]
    if s["kind"] == "linear":
        return [w / f for w in inv], 1.0
    if s["kind"] == "smooth":
        out = []
        for w in inv:
            turns = s["original"] * w / (2 * math.pi)  # turns over the original length
            keep = min(1.0, max(0.0, (turns - s["low"]) / (s["high"] - s["low"])))
            out.append((1 - keep) * w / f + keep * w)
        return out, 1.0

    def pair_of(turns):  # the (fractional) pair that makes so many turns over the original length
        return rotary * math.log(s["original"] / (turns * 2 * math.pi)) / (2 * math.log(THETA))

    low = max(0, math.floor(pair_of(s["beta_fast"])))
    high = min(rotary - 1, math.ceil(pair_of(s["beta_slow"])))
    span = max(high - low, 0.001)
    out = []
    for i, w in enumerate(inv):
        slow = min(1.0, max(0.0, (i - low) / span))
        out.append(slow * w / f + (1 - slow) * w)
    return out, 0.1 * math.log(f) + 1.0


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    hq, hkv, bs = case["q_heads"], case["kv_heads"], case["block"]

    def normal(*shape, by=1.0):
        x = torch.randn(shape, generator=g, device=dev, dtype=torch.bfloat16)
        return x if by == 1.0 else x.mul_(by)

    if case["op"] == "rope":
        t = case["tokens"]
        blocks = (t + bs - 1) // bs + 2
        qkv = normal(t, (hq + 2 * hkv) * D)  # the projection's output; q, k, v are views of it
        q, k, v = (x.unflatten(1, (-1, D)) for x in qkv.split([hq * D, hkv * D, hkv * D], 1))
        slots = torch.randperm(blocks * bs, generator=g, device=dev)[:t].contiguous()
        if case["pad"]:
            slots[t - case["pad"]:] = -1
        state = {"q": q, "k": k, "v": v, "slots": slots,
                 "positions": torch.randint(0, case["far"], (t,), generator=g, device=dev,
                                            dtype=torch.int32),
                 "k_cache": normal(blocks, hkv, bs, D), "v_cache": normal(blocks, hkv, bs, D),
                 "out": torch.empty(t, hq, D, dtype=torch.bfloat16, device=dev)}
        inv, gain = _frequencies(case["rotary"], case["scaling"])
        state["inv_freq"] = torch.tensor(inv, dtype=torch.float64, device=dev)
        state["gain"] = gain
        if own:  # the plan that a program keeps next to its model
            import paged_kv_cache_245_gb300 as pkv
            state["rope"] = pkv.RopePlan(case["rotary"], theta=THETA,
                                         interleaved=case["interleaved"],
                                         scaling=SCALING[case["scaling"]])
        return {**state, "case": case}

    ctx, new = _ctx_and_new(case)
    batch, top = len(ctx), max(ctx)
    state = {"max_context": top, "max_new": max(new), "scale": D ** -0.5,
             "ctx": torch.tensor(ctx, dtype=torch.int32, device=dev)}
    if case["layout"] == "paged":
        need = [(c + bs - 1) // bs for c in ctx]
        pool = torch.randperm(sum(need) + 3, generator=g, device=dev).to(torch.int32)
        tables = torch.zeros(batch, max(need), dtype=torch.int32, device=dev)
        have = torch.arange(max(need), device=dev)[None] < torch.tensor(need, device=dev)[:, None]
        tables[have] = pool[:sum(need)]
        state["tables"] = tables
        shape = (sum(need) + 3, hkv, bs, D)
    else:
        state["req_ids"] = torch.randperm(batch + 1, generator=g, device=dev)[:batch].to(torch.int32)
        shape = (batch + 1, hkv, (top + 15) // 16 * 16, D)
    state["k"], state["v"] = normal(*shape), normal(*shape)
    # scores with a standard deviation of 4: sharp rows, as trained heads have
    state["q"] = normal(sum(new), hq, D, by=4.0)
    state["out"] = torch.empty_like(state["q"])
    if case["op"] == "prefill":
        ends = torch.tensor([0] + new, dtype=torch.int32).cumsum(0).to(torch.int32)
        state["cu"] = ends.to(dev)
    state["slopes"] = state["first"] = state["prefix"] = None
    if case["slopes"]:
        state["slopes"] = torch.tensor([2.0 ** (-8.0 * (h + 1) / hq) for h in range(hq)],
                                       dtype=torch.float32, device=dev)
    if case["documents"]:
        state["first"] = torch.tensor(_first_keys(case, ctx, new), dtype=torch.int32, device=dev)
    if case.get("prefix"):
        state["prefix"] = torch.tensor(_prefixes(case, ctx), dtype=torch.int32, device=dev)
    if own and case["op"] == "decode":
        import paged_kv_cache_245_gb300 as pkv
        size = pkv.scored_decode_workspace_size(batch, hq, hkv, top, case["window"])
        state["workspace"] = torch.empty(max(size, 16), dtype=torch.uint8, device=dev)
    return {**state, "case": case}


# -------------------------------------------------------------------- one pass

def run(state):
    op = state["case"]["op"]
    if own:
        return {"rope": _own_rope, "decode": _own_decode, "prefill": _own_prefill}[op](state)
    return {"rope": _plain_rope, "decode": _plain_decode, "prefill": _plain_prefill}[op](state)


def _own_rope(s):
    import paged_kv_cache_245_gb300 as pkv
    out = pkv.rope_append(s["positions"], s["slots"], s["q"], s["k"], s["v"], s["k_cache"],
                          s["v_cache"], s["rope"], out=s["out"])
    return [out, s["k_cache"], s["v_cache"]]


def _own_decode(s):
    import paged_kv_cache_245_gb300 as pkv
    c = s["case"]
    call, where = (pkv.paged_decode_attention_scored, "tables") if c["layout"] == "paged" else (
        pkv.contig_decode_attention_scored, "req_ids")
    return call(s["q"], s["k"], s["v"], s[where], s["ctx"], s["max_context"], s["scale"],
                softcap=c["softcap"], window=c["window"], alibi_slopes=s["slopes"],
                first_key=s["first"], out=s["out"], workspace=s["workspace"])


def _own_prefill(s):
    import paged_kv_cache_245_gb300 as pkv
    c = s["case"]
    call, where = (pkv.paged_prefill_attention_scored, "tables") if c["layout"] == "paged" else (
        pkv.contig_prefill_attention_scored, "req_ids")
    return call(s["q"], s["cu"], s["k"], s["v"], s[where], s["ctx"], s["max_new"], s["scale"],
                softcap=c["softcap"], window=c["window"], alibi_slopes=s["slopes"],
                first_key=s["first"], prefix_lens=s["prefix"], out=s["out"])


# ------------------------------------------------------------------ plain forms

def _plain_rope(s):
    c = s["case"]
    half = c["rotary"] // 2
    # far positions: the angle is a number of thousands of radians, taken in 64 bits
    angle = s["positions"].double()[:, None] * s["inv_freq"]
    turns = [(f(angle) * s["gain"]).float()[:, None] for f in (torch.cos, torch.sin)]

    def turn(x):
        cos, sin = (f[:x.shape[0]] for f in turns)
        x = x.float()
        if c["interleaved"]:
            a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
            both = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = x[..., :half], x[..., half:2 * half]
            both = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        return torch.cat([both, x[..., 2 * half:]], -1).bfloat16()

    # rows of padding tokens (a negative slot) go nowhere
    n = c["tokens"] - c["pad"]
    slots = s["slots"][:n]
    block, off = slots // c["block"], slots % c["block"]
    s["k_cache"][block, :, off] = turn(s["k"][:n])
    s["v_cache"][block, :, off] = s["v"][:n]
    return [turn(s["q"]), s["k_cache"], s["v_cache"]]


def _rows(s, x):
    """The cache rows of every sequence in order: [B, Hkv, positions, D] in 32 bits."""
    if s["case"]["layout"] == "contig":
        return x[s["req_ids"].long()].float()
    return x[s["tables"].long()].transpose(1, 2).flatten(2, 3).float()


def _attend(s, q, position, first, prefix):
    """q [B, L, Hq, D] at positions [B, L] -> [B, L, Hq, D] in 32 bits."""
    c = s["case"]
    b, n, hq, _ = q.shape
    hkv = c["kv_heads"]
    group = hq // hkv
    k, v = _rows(s, s["k"]), _rows(s, s["v"])
    keys = torch.arange(k.shape[2], device=k.device)
    q = q.float().unflatten(2, (hkv, group)).permute(0, 2, 3, 1, 4).reshape(b, hkv, group * n, D)
    x = (q @ k.transpose(-1, -2)).mul_(s["scale"])
    if c["softcap"]:
        x = x.div_(c["softcap"]).tanh_().mul_(c["softcap"])
    x = x.view(b, hkv, group, n, -1)
    p = position[:, :, None]
    if s["slopes"] is not None:
        x -= s["slopes"].view(1, hkv, group, 1, 1) * (p - keys).abs().float()[:, None, None]
    seen = (keys <= p) if prefix is None else (keys <= p) | (keys < prefix[:, None, None])
    seen = seen & (keys < s["ctx"][:, None, None])
    if c["window"]:
        seen = seen & (keys > p - c["window"])
    if first is not None:
        seen = seen & (keys >= first[:, :, None])
    x = x.masked_fill_(~seen[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    x = x.sub_(top.masked_fill_(top == -math.inf, 0.0)).exp_()
    total = x.sum(-1, keepdim=True)
    o = x.view(b, hkv, group * n, -1) @ v
    o = o.view(b, hkv, group, n, D) / total.masked_fill_(total == 0, 1.0)
    return o.permute(0, 3, 1, 2, 4).reshape(b, n, hq, D)


def _plain_decode(s):
    position = (s["ctx"] - 1)[:, None]
    first = None if s["first"] is None else s["first"][:, None]
    return _attend(s, s["q"][:, None], position, first, None)[:, 0].bfloat16()


def _plain_prefill(s):
    q, cu = s["q"], s["cu"].long()
    n = cu.diff()
    batch, longest = n.shape[0], s["max_new"]
    seq = torch.repeat_interleave(torch.arange(batch, device=q.device), n, output_size=q.shape[0])
    at = torch.arange(q.shape[0], device=q.device) - cu[seq]
    padded = q.new_zeros(batch, longest, *q.shape[1:])
    padded[seq, at] = q
    position = (s["ctx"] - n)[:, None] + torch.arange(longest, device=q.device)
    first = None
    if s["first"] is not None:
        first = s["first"].new_zeros(batch, longest)
        first[seq, at] = s["first"]
    return _attend(s, padded, position, first, s["prefix"])[seq, at].bfloat16()


# ---------------------------------------------------------------- in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(case, s)
    hq, hkv = case["q_heads"], case["kv_heads"]
    group = hq // hkv
    ctx, new = _ctx_and_new(case)
    out = torch.zeros(sum(new), hq, D, dtype=torch.float64, device="cuda")
    slopes = None if s["slopes"] is None else s["slopes"].double()
    at = 0
    for i, rows in enumerate(_ranges(case)):
        c, n = ctx[i], new[i]
        if case["layout"] == "paged":
            blocks = s["tables"][i, :(c + case["block"] - 1) // case["block"]].long()
            k, v = (torch.cat(list(x[blocks].unbind(0)), 1)[:, :c] for x in (s["k"], s["v"]))
        else:
            k, v = (x[int(s["req_ids"][i])][:, :c] for x in (s["k"], s["v"]))
        low, end = torch.tensor(rows, device="cuda").unbind(1)
        key = torch.arange(c, device="cuda")
        hidden = (key < low[:, None]) | (key >= end[:, None])
        away = (torch.arange(c - n, c, device="cuda")[:, None] - key).abs().double()
        for h in range(hq):
            z = torch.einsum("nd,kd->nk", s["q"][at:at + n, h].double(), k[h // group].double())
            z *= s["scale"]
            if case["softcap"]:
                e = torch.exp(2 * z / case["softcap"])
                z = case["softcap"] * (1 - 2 / (e + 1))
            if slopes is not None:
                z = z - slopes[h] * away
            z[hidden] = -math.inf
            w = torch.exp(z - torch.logsumexp(z, -1, keepdim=True))
            w[hidden] = 0
            out[at:at + n, h] = torch.einsum("nk,kd->nd", w, v[h // group].double())
        at += n
    return out


def _exact_rope(case, s):
    half, n = case["rotary"] // 2, case["tokens"] - case["pad"]
    angle = torch.outer(s["positions"].double(), s["inv_freq"])
    unit = torch.polar(torch.full_like(angle, s["gain"]), angle)[:, None]

    def turn(x):
        y = x.double().clone()
        even = slice(0, 2 * half, 2) if case["interleaved"] else slice(0, half)
        odd = slice(1, 2 * half, 2) if case["interleaved"] else slice(half, 2 * half)
        z = torch.complex(y[..., even].contiguous(), y[..., odd].contiguous()) * unit[:x.shape[0]]
        y[..., even], y[..., odd] = z.real, z.imag
        return y

    caches = [s["k_cache"].double(), s["v_cache"].double()]
    for cache, rows in zip(caches, (turn(s["k"][:n]), s["v"][:n].double())):
        flat = cache.transpose(1, 2).reshape(-1, case["kv_heads"], D)
        flat[s["slots"][:n]] = rows
        cache.copy_(flat.view(cache.shape[0], case["block"], case["kv_heads"], D).transpose(1, 2))
    return [turn(s["q"]), *caches]
