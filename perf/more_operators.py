"""The 8-bit KV cache of this library, as it is measured.

The cache holds K and V as 8-bit codes, int8 or float8_e4m3fn, with one fp32
scale for every 16 positions of a block and KV head: value = code * scale.
Four operators: the append that quantises new keys and values into it
(``kv_append_q8``), the same with rotary positions applied on the way
(``rope_append_q8``), attention of one new token per sequence over it
(``*_decode_attention_q8``) and attention of chunks of new tokens
(``*_prefill_attention_q8``).

``own`` is set by whoever measures: true runs the library's calls, false their
plain form in elementary torch operations.
"""
import math
import random

import torch

own = False

D = 128       # head size of the library
ROWS = 16     # positions that share a scale
QMAX = {"int8": 127.0, "e4m3": 448.0}
CODES = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}
TINY = 2.0 ** -100  # a scale below this holds zeros
THETA = 500000.0


# ------------------------------------------------------------------ the cases

def _append(name, op, kind, batch, hq, hkv, new_min, new_max, cached_min, cached_max, block=16,
            pad=0, shuffled=False, rotary=128, interleaved=False, salt=1):
    return {"name": name, "op": op, "kind": kind, "layout": "paged", "batch": batch,
            "q_heads": hq, "kv_heads": hkv, "new_min": new_min, "new_max": new_max,
            "cached_min": cached_min, "cached_max": cached_max, "block": block, "pad": pad,
            "shuffled": shuffled, "rotary": rotary, "interleaved": interleaved, "salt": salt}


def _decode(name, kind, layout, batch, hq, hkv, ctx_min, ctx_max, block=16, salt=1):
    return {"name": name, "op": "decode", "kind": kind, "layout": layout, "batch": batch,
            "q_heads": hq, "kv_heads": hkv, "ctx_min": ctx_min, "ctx_max": ctx_max,
            "block": block, "salt": salt}


def _prefill(name, kind, layout, batch, hq, hkv, new_min, new_max, cached_min, cached_max,
             block=16, salt=1):
    return {"name": name, "op": "prefill", "kind": kind, "layout": layout, "batch": batch,
            "q_heads": hq, "kv_heads": hkv, "new_min": new_min, "new_max": new_max,
            "cached_min": cached_min, "cached_max": cached_max, "block": block, "salt": salt}


def listed():
    return [
        # a decode step of a large ragged batch: one token into the middle of each tail group
        _append("append 256 decode tokens int8", "append", "int8", 256, 8, 8, 1, 1, 16, 8000),
        # ragged chunks after cached positions, blocks of 48, padded for a captured graph
        _append("append ragged chunks e4m3", "append", "e4m3", 7, 4, 4, 1, 300, 0, 500, block=48,
                pad=9),
        # whole prompts of a batch: bandwidth
        _append("append 16384 prompt tokens int8", "append", "int8", 8, 8, 8, 2048, 2048, 0, 0),

        # one chat's next token: only the call's latency counts
        _append("rope append 1 token e4m3", "rope", "e4m3", 1, 32, 8, 1, 1, 1000, 1000),
        # whole prompts with the query heads turned on the way: bandwidth
        _append("rope append 16384 prompt tokens e4m3", "rope", "e4m3", 8, 32, 8, 2048, 2048, 0,
                0),

        # one chat alone on the machine: latency
        _decode("decode b1 int8", "int8", "paged", 1, 32, 8, 1000, 1000),
        # a full ragged batch
        _decode("decode b64 ragged e4m3", "e4m3", "paged", 64, 32, 8, 16, 8192),
        # requests in contiguous rows, 8 query heads per KV head
        _decode("decode b32 contig int8", "int8", "contig", 32, 32, 4, 100, 4095),
        # a large batch at full contexts, 7 query heads per KV head: bandwidth
        _decode("decode b128 full e4m3", "e4m3", "paged", 128, 56, 8, 8000, 8192, block=32),

        # a few draft tokens of each sequence checked at once: latency and bandwidth
        _prefill("prefill 16 x drafts e4m3", "e4m3", "paged", 16, 32, 8, 2, 8, 500, 4000),
        # fresh prompts: tensor cores and the exponentials
        _prefill("prefill 8 x 2048 int8", "int8", "paged", 8, 32, 8, 2048, 2048, 0, 0),
        # chunks after cached positions, contiguous rows, 7 query heads per KV head
        _prefill("prefill chunks e4m3", "e4m3", "contig", 6, 56, 8, 100, 1500, 0, 3000),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    hq, hkv = rng.choice([(32, 8), (32, 4), (56, 8), (4, 4), (20, 4), (10, 2), (6, 1)])
    salt = rng.randrange(1, 1 << 30)
    kind = rng.choice(["int8", "e4m3"])
    op = rng.choice(["append", "rope", "decode", "prefill"])
    if op in ("append", "rope"):
        new = _log(rng, 1, 2048)
        cached = rng.choice([0, _log(rng, 1, 8000)])
        batch = max(1, min(_log(rng, 1, 256), 12000 // new))
        # the rope cases are all in e4m3: fp32 rotations that differ in the last bit may
        # differ by a code where a value lies on the border of two
        return _unnamed(_append("", op, "e4m3" if op == "rope" else kind, batch, hq, hkv,
                                max(1, new // rng.choice([1, 5])), new,
                                cached // rng.choice([1, 10]), cached,
                                rng.choice([16, 32, 48, 128]), rng.choice([0, 0, 3]),
                                rng.random() < 0.3, 2 * rng.randint(1, 64), rng.random() < 0.5,
                                salt))
    layout = rng.choice(["paged", "contig"])
    block = rng.choice([16, 32, 48, 64, 128])
    if op == "decode":
        top = _log(rng, 1, 8192)
        return _unnamed(_decode("", kind, layout, _log(rng, 1, 100), hq, hkv,
                                max(1, top // rng.choice([1, 3, 100])), top, block, salt))
    new = _log(rng, 1, 4096)
    cached = rng.choice([0, _log(rng, 1, 4096)])
    batch = max(1, min(_log(rng, 1, 32), (1 << 24) // (new * (new + cached))))
    return _unnamed(_prefill("", kind, layout, batch, hq, hkv, max(1, new // rng.choice([1, 4])),
                             new, cached // rng.choice([1, 4]), cached, block, salt))


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


def work(case):
    hq, hkv = case["q_heads"], case["kv_heads"]
    ctx, new = _ctx_and_new(case)
    if case["op"] in ("append", "rope"):
        # k and v in (bf16) and out (8 bits); a slot each, and the scales of the groups
        tokens = sum(new)
        groups = sum((c + ROWS - 1) // ROWS - (c - n) // ROWS for c, n in zip(ctx, new))
        size = tokens * (2 * hkv * D * 3 + 8) + groups * 2 * hkv * 4
        flops = tokens * 2 * hkv * D * 2
        if case["op"] == "rope":  # positions; q in and out
            size += (tokens + case["pad"]) * (hq * D * 2 * 2 + 4)
            flops += tokens * (hq + hkv) * case["rotary"] * 3
        return {"bytes": size, "flops": flops}
    pairs = sum(n * (c - n) + n * (n + 1) // 2 for c, n in zip(ctx, new))
    keys = sum(ctx)
    return {"bytes": keys * hkv * 2 * (D + 4.0 / ROWS) + sum(new) * hq * D * 2 * 2,
            "flops": pairs * hq * D * 4}


# ------------------------------------------------------------------- the inputs

def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    hq, hkv, bs = case["q_heads"], case["kv_heads"], case["block"]
    ctx, new = _ctx_and_new(case)
    batch, top = len(ctx), max(ctx)

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.bfloat16)

    def codes(*shape):  # what rows of unit variance are held as
        x = normal(*shape)
        if case["kind"] == "int8":
            return x.mul_(42.0).round_().clamp_(-127.0, 127.0).to(torch.int8)
        return x.mul_(150.0).clamp_(-448.0, 448.0).to(torch.float8_e4m3fn)

    def scales(*shape):  # largest values between 1 and 6 or so, from group to group
        x = torch.randn(shape, generator=g, device=dev).mul_(0.4).exp_()
        return x.mul_(3.0 / QMAX[case["kind"]])

    state = {"case": case, "ctx": torch.tensor(ctx, dtype=torch.int32, device=dev)}
    if case["layout"] == "paged":
        need = [(c + bs - 1) // bs for c in ctx]
        pool = torch.randperm(sum(need) + 3, generator=g, device=dev).to(torch.int32)
        tables = torch.zeros(batch, max(need), dtype=torch.int32, device=dev)
        have = torch.arange(max(need), device=dev)[None] < torch.tensor(need, device=dev)[:, None]
        tables[have] = pool[:sum(need)]
        state["tables"] = tables
        shape = (sum(need) + 3, hkv, bs)
    else:
        state["req_ids"] = torch.randperm(batch + 1, generator=g, device=dev)[:batch].to(torch.int32)
        shape = (batch + 1, hkv, (top + 15) // 16 * 16)
    state["k"], state["v"] = codes(*shape, D), codes(*shape, D)
    group_shape = (*shape[:2], shape[2] // ROWS)
    state["k_scale"], state["v_scale"] = scales(*group_shape), scales(*group_shape)

    if case["op"] in ("append", "rope"):
        n = torch.tensor(new, device=dev)
        seq = torch.repeat_interleave(torch.arange(batch, device=dev), n, output_size=sum(new))
        first = n.cumsum(0) - n
        pos = state["ctx"][seq] - n[seq] + torch.arange(sum(new), device=dev) - first[seq]
        slots = state["tables"][seq, pos // bs].long() * bs + pos % bs
        if case["shuffled"]:  # tokens of a step in the order in which the requests arrived
            order = torch.randperm(sum(new), generator=g, device=dev)
            pos, slots = pos[order], slots[order]
        pad = case["pad"]
        state["positions"] = torch.cat([pos, pos.new_zeros(pad)]).to(torch.int32)
        state["slots"] = torch.cat([slots, slots.new_full((pad,), -1)])
        tokens = sum(new) + pad
        if case["op"] == "append":
            state["k_new"], state["v_new"] = normal(tokens, hkv, D), normal(tokens, hkv, D)
            return state
        qkv = normal(tokens, (hq + 2 * hkv) * D)  # the projection's output, q, k, v views of it
        state["q"], state["k_new"], state["v_new"] = (
            x.unflatten(1, (-1, D)) for x in qkv.split([hq * D, hkv * D, hkv * D], 1))
        state["out"] = torch.empty(tokens, hq, D, dtype=torch.bfloat16, device=dev)
        state["inv_freq"] = torch.tensor([THETA ** (-2.0 * i / case["rotary"])
                                          for i in range(case["rotary"] // 2)],
                                         dtype=torch.float64, device=dev)
        if own:  # the plan that a program keeps next to its model
            import paged_kv_cache_245_gb300 as pkv
            state["rope"] = pkv.RopePlan(case["rotary"], theta=THETA,
                                         interleaved=case["interleaved"])
        return state

    # scores with a standard deviation of 4: sharp rows, as trained heads have
    state["q"] = normal(sum(new), hq, D).mul_(4.0)
    state["out"] = torch.empty_like(state["q"])
    state["max_context"], state["max_new"], state["scale"] = top, max(new), D ** -0.5
    if case["op"] == "prefill":
        state["cu"] = torch.tensor([0] + new, dtype=torch.int32).cumsum(0).to(torch.int32).to(dev)
    elif own:
        import paged_kv_cache_245_gb300 as pkv
        size = pkv.q8_decode_workspace_size(batch, hq, hkv, top)
        state["workspace"] = torch.empty(max(size, 16), dtype=torch.uint8, device=dev)
    return state


# -------------------------------------------------------------------- one pass

def run(state):
    op = state["case"]["op"]
    if own:
        return {"append": _own_append, "rope": _own_rope, "decode": _own_decode,
                "prefill": _own_prefill}[op](state)
    return {"append": _plain_append, "rope": _plain_rope, "decode": _plain_decode,
            "prefill": _plain_prefill}[op](state)


def _own_append(s):
    import paged_kv_cache_245_gb300 as pkv
    pkv.kv_append_q8(s["slots"], s["k_new"], s["v_new"], s["k"], s["v"], s["k_scale"],
                     s["v_scale"])
    return [s["k"], s["v"], s["k_scale"], s["v_scale"]]


def _own_rope(s):
    import paged_kv_cache_245_gb300 as pkv
    out = pkv.rope_append_q8(s["positions"], s["slots"], s["q"], s["k_new"], s["v_new"], s["k"],
                             s["v"], s["k_scale"], s["v_scale"], s["rope"], out=s["out"])
    return [out, s["k"], s["v"], s["k_scale"], s["v_scale"]]


def _own_decode(s):
    import paged_kv_cache_245_gb300 as pkv
    call, where = (pkv.paged_decode_attention_q8, "tables") if "tables" in s else (
        pkv.contig_decode_attention_q8, "req_ids")
    return call(s["q"], s["k"], s["v"], s["k_scale"], s["v_scale"], s[where], s["ctx"],
                s["max_context"], s["scale"], out=s["out"], workspace=s["workspace"])


def _own_prefill(s):
    import paged_kv_cache_245_gb300 as pkv
    call, where = (pkv.paged_prefill_attention_q8, "tables") if "tables" in s else (
        pkv.contig_prefill_attention_q8, "req_ids")
    return call(s["q"], s["cu"], s["k"], s["v"], s["k_scale"], s["v_scale"], s[where], s["ctx"],
                s["max_new"], s["scale"], out=s["out"])


# ------------------------------------------------------------------ plain forms

def _code(x, kind):
    """Values in units of the scale as codes: the nearest, ties to even."""
    if kind == "int8":
        return x.round().clamp_(-127.0, 127.0).to(torch.int8)
    return x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)


def _put(s, x, slots, cache, scale):
    """New rows x [T, Hkv, D] (fp32) of distinct slots into the cache."""
    c = s["case"]
    kind, qmax, hkv, per = c["kind"], QMAX[c["kind"]], c["kv_heads"], c["block"] // ROWS
    # the call's groups (16 slots each), and the row of each token in its group
    groups, at = torch.unique(slots // ROWS, return_inverse=True)
    block, part = groups // per, groups % per
    rows = cache.unflatten(2, (per, ROWS))
    held = rows.view(torch.int8)[block, :, part].view(cache.dtype)  # [groups, Hkv, 16, D]
    old = scale[block, :, part]
    started = torch.zeros_like(groups).index_add_(0, at, (slots % ROWS == 0).long()) > 0
    old = old.masked_fill(started[:, None], 0.0)
    top = x.abs().amax(-1)
    new = torch.zeros_like(old).scatter_reduce_(0, at[:, None].expand(-1, hkv), top, "amax")
    new = torch.maximum(old, new / qmax)
    inv = torch.where(new >= TINY, 1.0 / new, torch.zeros_like(new))
    value = held.float() * old[:, :, None, None]
    code = torch.where((new == old)[:, :, None, None], held.float(),
                       _code(value * inv[:, :, None, None], kind).float())
    code[at, :, slots % ROWS] = _code(x * inv[at][:, :, None], kind).float()
    rows.view(torch.int8)[block, :, part] = code.to(cache.dtype).view(torch.int8)
    scale[block, :, part] = new


def _plain_append(s):
    n = s["slots"].shape[0] - s["case"]["pad"]  # rows of padding tokens go nowhere
    _put(s, s["k_new"][:n].float(), s["slots"][:n], s["k"], s["k_scale"])
    _put(s, s["v_new"][:n].float(), s["slots"][:n], s["v"], s["v_scale"])
    return [s["k"], s["v"], s["k_scale"], s["v_scale"]]


def _plain_rope(s):
    c = s["case"]
    half = c["rotary"] // 2
    # far positions: the angle is a number of thousands of radians, taken in 64 bits
    angle = s["positions"].double()[:, None] * s["inv_freq"]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def turn(x):
        x = x.float()
        if c["interleaved"]:
            a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
            both = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = x[..., :half], x[..., half:2 * half]
            both = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        return torch.cat([both, x[..., 2 * half:]], -1)

    n = s["slots"].shape[0] - c["pad"]
    _put(s, turn(s["k_new"])[:n], s["slots"][:n], s["k"], s["k_scale"])
    _put(s, s["v_new"][:n].float(), s["slots"][:n], s["v"], s["v_scale"])
    return [turn(s["q"]).bfloat16(), s["k"], s["v"], s["k_scale"], s["v_scale"]]


def _rows(s, x, scale):
    """The values of every sequence's rows in order: [B, Hkv, positions, D] in 32 bits."""
    # (indexed by bytes: not every torch build indexes float8)
    if "req_ids" in s:
        at = s["req_ids"].long()
        return x.view(torch.int8)[at].view(x.dtype).float().mul_(
            scale[at].repeat_interleave(ROWS, 2)[..., None])
    at = s["tables"].long()
    x = x.view(torch.int8)[at].view(x.dtype).float()
    x = x.mul_(scale[at].repeat_interleave(ROWS, 3)[..., None])
    return x.transpose(1, 2).flatten(2, 3)


def _attend(s, q, position):
    """q [B, L, Hq, D] at positions [B, L] -> [B, L, Hq, D] in 32 bits."""
    b, n, hq, _ = q.shape
    hkv = s["case"]["kv_heads"]
    group = hq // hkv
    k = _rows(s, s["k"], s["k_scale"])
    keys = torch.arange(k.shape[2], device=k.device)
    q = q.float().unflatten(2, (hkv, group)).permute(0, 2, 3, 1, 4).reshape(b, hkv, group * n, D)
    x = (q @ k.transpose(-1, -2)).mul_(s["scale"])
    del k
    x = x.view(b, hkv, group, n, -1)
    x = x.masked_fill_((keys > position[:, :, None])[:, None, None], -math.inf)
    x = x.sub_(x.amax(-1, keepdim=True)).exp_()
    total = x.sum(-1, keepdim=True)
    v = _rows(s, s["v"], s["v_scale"])
    o = x.view(b, hkv, group * n, -1) @ v
    o = o.view(b, hkv, group, n, D) / total
    return o.permute(0, 3, 1, 2, 4).reshape(b, n, hq, D)


def _plain_decode(s):
    return _attend(s, s["q"][:, None], (s["ctx"] - 1)[:, None])[:, 0].bfloat16()


def _plain_prefill(s):
    q, cu = s["q"], s["cu"].long()
    n = cu.diff()
    batch, longest = n.shape[0], s["max_new"]
    seq = torch.repeat_interleave(torch.arange(batch, device=q.device), n, output_size=q.shape[0])
    at = torch.arange(q.shape[0], device=q.device) - cu[seq]
    padded = q.new_zeros(batch, longest, *q.shape[1:])
    padded[seq, at] = q
    position = (s["ctx"] - n)[:, None] + torch.arange(longest, device=q.device)
    return _attend(s, padded, position)[seq, at].bfloat16()


# ---------------------------------------------------------------- in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("append", "rope"):
        return _exact_append(case, s)
    hq, hkv, bs = case["q_heads"], case["kv_heads"], case["block"]
    group = hq // hkv
    ctx, new = _ctx_and_new(case)
    out = torch.zeros(sum(new), hq, D, dtype=torch.float64, device="cuda")
    at = 0
    for i, (c, n) in enumerate(zip(ctx, new)):
        pair = []
        for x, scale in ((s["k"], s["k_scale"]), (s["v"], s["v_scale"])):
            if "tables" in s:
                blocks = s["tables"][i, :(c + bs - 1) // bs].long()
                x = torch.cat([x[b] for b in blocks.tolist()], 1)
                scale = scale[blocks].transpose(0, 1).flatten(1)
            else:
                x, scale = x[int(s["req_ids"][i])], scale[int(s["req_ids"][i])]
            each = scale.double().repeat_interleave(ROWS, 1)[:, :c]
            pair.append(x[:, :c].to(torch.float64) * each[..., None])
        k, v = pair
        late = torch.arange(c, device="cuda") > torch.arange(c - n, c, device="cuda")[:, None]
        for h in range(hkv):
            q = s["q"][at:at + n, h * group:(h + 1) * group].double()
            z = torch.einsum("ngd,kd->gnk", q, k[h]) * s["scale"]
            z[:, late] = -math.inf
            w = torch.exp(z - torch.logsumexp(z, -1, keepdim=True))
            out[at:at + n, h * group:(h + 1) * group] = torch.einsum("gnk,kd->ngd", w, v[h])
        at += n
    return out


def _exact_append(case, s):
    """Outputs in 64 bits; the codes in int8 are whole numbers and have no other value."""
    n, bs, hkv = s["slots"].shape[0] - case["pad"], case["block"], case["kv_heads"]
    qmax = QMAX[case["kind"]]
    turned = []
    if case["op"] == "rope":
        half = case["rotary"] // 2
        angle = torch.outer(s["positions"].double(), s["inv_freq"])
        unit = torch.polar(torch.ones_like(angle), angle)[:, None]
        even = slice(0, 2 * half, 2) if case["interleaved"] else slice(0, half)
        odd = slice(1, 2 * half, 2) if case["interleaved"] else slice(half, 2 * half)
        for x in (s["q"], s["k_new"]):
            y = x.double().clone()
            z = torch.complex(y[..., even].contiguous(), y[..., odd].contiguous()) * unit
            y[..., even], y[..., odd] = z.real, z.imag
            turned.append(y)
    k = turned[1] if turned else s["k_new"].double()
    slots, caches, scales = s["slots"][:n], [], []
    for x, cache, scale in ((k, s["k"], s["k_scale"]), (s["v_new"].double(), s["v"], s["v_scale"])):
        # everything by slot: [slots, Hkv, D], its scale by group [groups, Hkv]
        code = cache.to(torch.float64).transpose(1, 2).reshape(-1, hkv, D)
        flat = scale.double().transpose(1, 2).reshape(-1, hkv)
        fresh = torch.zeros(code.shape[0], dtype=torch.bool, device="cuda")
        fresh[slots] = True
        touched = fresh.view(-1, ROWS).any(1)
        before = torch.where(fresh[::ROWS, None], 0.0, flat)
        value = code * before.repeat_interleave(ROWS, 0)[..., None]
        value[slots] = x[:n]
        size = torch.where(fresh[:, None], value.abs().amax(-1), 0.0)
        after = torch.maximum(before, size.view(-1, ROWS, hkv).amax(1) / qmax)
        after = torch.where(touched[:, None], after, flat)
        unit = (value / after.repeat_interleave(ROWS, 0)[..., None]).clamp(-qmax, qmax)
        if case["kind"] == "int8":
            unit = unit.round()
        else:  # three bits behind the leading one, steps of 2^-9 at the least
            step = torch.exp2(torch.floor(torch.log2(unit.abs().clamp(min=2.0 ** -6))) - 3)
            unit = torch.round(unit / step) * step
        unit = torch.where(touched.repeat_interleave(ROWS)[:, None, None], unit, code)
        caches.append(unit.view(-1, bs, hkv, D).transpose(1, 2))
        scales.append(after.view(-1, bs // ROWS, hkv).transpose(1, 2))
    caches = [None, None] if case["kind"] == "int8" else caches
    return [*turned[:1], *caches, *scales]
