"""Appends to the 8-bit cache (pkv_kv_append_q8, pkv_rope_append_q8): codes and
scales against the plain loop bit for bit, the turned keys within a code."""
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_245_gb300 as pkv
import q8_ref

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
D = 128


@pytest.fixture(autouse=True)
def _reset():
    pkv.set_checked(False)
    yield
    pkv.set_checked(False)
    torch.cuda.synchronize()


class Cache:
    def __init__(self, blocks, hkv, bs, dtype, seed=0, garbage=False):
        g = torch.Generator().manual_seed(seed)
        shape, per = (blocks, hkv, bs, D), (blocks, hkv, bs // 16)
        self.k, self.v = (q8_ref.random_codes(shape, dtype, g, "cpu") for _ in range(2))
        self.ks, self.vs = (q8_ref.random_scales(per, dtype, g, "cpu") for _ in range(2))
        self.dev = [x.to(DEV) for x in (self.k, self.v, self.ks, self.vs)]

    def put(self, slots, k, v):
        pkv.kv_append_q8(slots.to(DEV), k.to(DEV), v.to(DEV), *self.dev)
        self.expect(slots, k.float(), v.float())
        self.check()

    def expect(self, slots, k, v):
        q8_ref.append(self.k, self.ks, slots, k)
        q8_ref.append(self.v, self.vs, slots, v)

    def check(self):
        for name, want, got in zip(("k", "v", "k_scale", "v_scale"),
                                   (self.k, self.v, self.ks, self.vs), self.dev):
            if want.dtype == torch.float32:
                assert torch.equal(got.cpu(), want), name
            else:
                a, b = got.cpu().view(torch.int8), want.view(torch.int8)
                bad = (a != b).nonzero()
                assert bad.numel() == 0, "%s: %d codes differ, first at %s: %d for %d" % (
                    name, bad.shape[0], bad[0].tolist(), a[tuple(bad[0])], b[tuple(bad[0])])


def rows(T, hkv, seed=1, by=1.0):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(T, hkv, D, generator=g) * by).bfloat16() for _ in range(2)]


@pytest.mark.parametrize("dtype", q8_ref.FORMATS)
@pytest.mark.parametrize("hkv,bs", [(1, 16), (8, 16), (3, 48), (2, 128)])
@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 33, 200])
def test_prompt_rows(dtype, hkv, bs, T):
    c = Cache(T // bs + 3, hkv, bs, dtype)
    # from the start of a block, and from the middle of a group
    for start in (bs, bs + 5):
        c.put(torch.arange(start, start + T), *rows(T, hkv, seed=start))


@pytest.mark.parametrize("dtype", q8_ref.FORMATS)
def test_token_by_token(dtype):
    c = Cache(4, 2, 16, dtype)
    for i in range(40):  # rows that grow, then shrink
        c.put(torch.tensor([i]), *rows(1, 2, seed=i, by=math.exp(2 * math.sin(i))))


@pytest.mark.parametrize("dtype", q8_ref.FORMATS)
@pytest.mark.parametrize("T,spread", [(40, 64), (300, 4000), (700, 800), (3000, 40000)])
def test_any_order(dtype, T, spread):
    """Tokens of a group far apart in the call, some slots twice, some skipped."""
    c = Cache(spread // 32 + 1, 2, 32, dtype, seed=T)
    g = torch.Generator().manual_seed(T)
    slots = torch.randint(0, spread, (T,), generator=g)
    slots[torch.randint(0, T, (T // 9,), generator=g)] = -1
    c.put(slots, *rows(T, 2, seed=T))


def test_same_slot_many_times():
    c = Cache(2, 2, 16, torch.int8)
    c.put(torch.tensor([3, 3, 3, 17, 3, 16, 17]), *rows(7, 2))
    c.put(torch.full((500,), 9), *rows(500, 2))


def test_many_tiles():
    """More tokens than 32 a CTA in 304 CTAs, every group cut by a tile's edge."""
    T = 34000
    c = Cache(T // 128 + 2, 1, 128, torch.float8_e4m3fn)
    c.put(torch.arange(7, T + 7), *rows(T, 1))


def test_more_tokens_than_one_round():
    """More tokens than 512 a CTA on every SM; a group's rows far apart in the call."""
    T = 152 * 512 + 3000
    c = Cache(T // 64 + 2, 1, 64, torch.int8)
    slots = torch.arange(T) + 9
    slots[100], slots[T - 1] = slots[T - 1].clone(), slots[100].clone()
    slots[500] = slots[T - 2]  # the later token's row stays
    c.put(slots, *rows(T, 1))


@pytest.mark.parametrize("dtype", q8_ref.FORMATS)
def test_sizes_and_non_finite_rows(dtype):
    c = Cache(4, 2, 16, dtype)
    k, v = rows(48, 2)
    k[0] = 0
    k[16:32] = 0                       # a group of zeros: scale 0
    v[0, 0, 5] = math.inf
    v[1, 0, 6] = -math.inf
    v[2, 1, 7] = math.nan
    v[16:32] *= 2.0 ** -110            # below the smallest scale: zeros
    v[32:48, 0] *= 2.0 ** 120          # near the top of bf16's range
    k[32:48, 1] = math.inf             # nothing finite
    c.put(torch.arange(48), k, v)
    # rows that join groups of scale 0, and of a tiny and a huge one
    c.put(torch.tensor([20, 35, 3]), *rows(3, 2, seed=5))
    # a scale that no append wrote (uninitialised): counts as none
    for s in (c.ks, c.vs):
        s[3, 0, 0], s[3, 1, 0] = math.nan, -1.0
    for got, want in zip(c.dev[2:], (c.ks, c.vs)):
        got.copy_(want)
    k, v = rows(1, 2, seed=6)
    pkv.kv_append_q8(torch.tensor([50], device=DEV), k.to(DEV), v.to(DEV), *c.dev)
    for s in (c.ks, c.vs):
        s[3] = 0
    c.expect(torch.tensor([50]), k.float(), v.float())
    c.check()


def test_strides_and_layouts():
    """Views of one projection output; the contiguous layout; a stream of its own."""
    T, hq, hkv = 37, 6, 2
    qkv = torch.randn(T, (hq + 2 * hkv) * D, device=DEV).bfloat16()
    q, k, v = (x.unflatten(1, (-1, D)) for x in qkv.split([hq * D, hkv * D, hkv * D], 1))
    c = Cache(3, hkv, 160, torch.int8)
    slots = torch.arange(T) + 160 + 100
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        pkv.kv_append_q8(slots.to(DEV), k, v, *c.dev)
    s.synchronize()
    c.expect(slots, k.cpu().float(), v.cpu().float())
    c.check()


@pytest.mark.parametrize("dtype", q8_ref.FORMATS)
def test_captured(dtype):
    """A captured append replayed with other rows, slots and scales."""
    c = Cache(6, 2, 16, dtype)
    T = 20
    k, v = (x.to(DEV) for x in rows(T, 2))
    slots = torch.arange(T, device=DEV)
    pkv.kv_append_q8(slots, k, v, *c.dev)
    c.expect(slots.cpu(), k.cpu().float(), v.cpu().float())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pkv.kv_append_q8(slots, k, v, *c.dev)
    for i in range(3):
        nk, nv = rows(T, 2, seed=10 + i, by=1.0 + i)
        ns = torch.randperm(96)[:T]
        ns[i] = -1
        k.copy_(nk), v.copy_(nv), slots.copy_(ns)
        g.replay()
        c.expect(ns, nk.float(), nv.float())
        c.check()


def test_checked():
    c = Cache(2, 2, 16, torch.int8)
    pkv.set_checked(True)
    k, v = rows(3, 2)
    pkv.kv_append_q8(torch.tensor([4, 32, 1 << 40], device=DEV), k.to(DEV), v.to(DEV), *c.dev)
    assert pkv.get_device_error() == "slot"
    assert pkv.get_device_error() == "none"
    c.expect(torch.tensor([4, -1, -1]), k.float(), v.float())
    c.check()


def test_no_tokens():
    c = Cache(1, 2, 16, torch.int8)
    k, v = (x.to(DEV) for x in rows(0, 2))
    pkv.kv_append_q8(torch.zeros(0, dtype=torch.int64, device=DEV), k, v, *c.dev)
    c.check()


def test_block_copy_and_swap():
    c = Cache(6, 4, 16, torch.float8_e4m3fn)
    pairs = torch.tensor([[0, 5], [2, 3]], device=DEV)
    pkv.block_copy(pairs, [c.dev[0]], [c.dev[1]])
    pkv.block_copy(pairs, [c.dev[2]], [c.dev[3]])
    for x in (c.k, c.v, c.ks, c.vs):
        x = x.view(torch.int8) if x.dtype == torch.float8_e4m3fn else x
        x[5], x[3] = x[0].clone(), x[2].clone()
    c.check()
    host = [torch.zeros_like(x).pin_memory() for x in (c.k, c.v, c.ks, c.vs)]
    for i in (0, 2):
        pkv.block_swap(pairs, [c.dev[i]], [c.dev[i + 1]], [host[i]], [host[i + 1]])
    torch.cuda.synchronize()
    for got, want in zip(host, (c.k, c.v, c.ks, c.vs)):
        a, b = got.view(torch.int8), want.view(torch.int8)
        assert torch.equal(a[5], b[0]) and torch.equal(a[3], b[2])


# ------------------------------------------------------------------ with rotary positions

def turned(x, pos, plan):
    """x [T, H, D] (fp64) turned, in 64 bits, and the sizes that an fp32 turn's error goes by."""
    rd, half = plan.c.rotary_dim, plan.c.rotary_dim // 2
    turn = [int(t) for t in plan.c.turn[:half]]
    frac = np.array([[((int(p) * t) % 2 ** 64) / 2 ** 64 for t in turn] for p in pos])
    c, s = (f(2 * math.pi * frac)[:, None] * float(plan.c.gain) for f in (np.cos, np.sin))
    even, odd = (slice(0, rd, 2), slice(1, rd, 2)) if plan.c.interleaved else (
        slice(0, half), slice(half, rd))
    y, size = x.copy(), np.zeros_like(x)
    a, b = x[..., even], x[..., odd]
    y[..., even], y[..., odd] = a * c - b * s, b * c + a * s
    size[..., even] = size[..., odd] = (np.abs(a) + np.abs(b)) * abs(float(plan.c.gain))
    return y, size


@pytest.mark.parametrize("dtype", q8_ref.FORMATS)
@pytest.mark.parametrize("rotary,interleaved", [(128, False), (128, True), (64, False), (50, False),
                                                (50, True), (2, False), (48, False), (126, False)])
@pytest.mark.parametrize("T,start", [(1, 21), (45, 7), (700, 0)])
def test_rope(dtype, rotary, interleaved, T, start):
    hq, hkv, bs = 6, 2, 48
    plan = pkv.RopePlan(rotary, theta=500000.0, interleaved=interleaved)
    c = Cache(T // bs + 3, hkv, bs, dtype)
    qkv = torch.randn(T, (hq + 2 * hkv) * D, device=DEV).bfloat16()
    q, k, v = (x.unflatten(1, (-1, D)) for x in qkv.split([hq * D, hkv * D, hkv * D], 1))
    pos = torch.randint(0, 1 << 20, (T,), dtype=torch.int32)
    slots = torch.arange(T) + start
    slots[T // 3] = -1
    before = q8_ref.values(c.k, c.ks)
    out = pkv.rope_append_q8(pos.to(DEV), slots.to(DEV), q, k, v, *c.dev, plan)
    q8_ref.append(c.v, c.vs, slots, v.cpu().float())
    assert torch.equal(c.dev[1].cpu().view(torch.int8), c.v.view(torch.int8))
    assert torch.equal(c.dev[3].cpu(), c.vs)
    # queries: as rope_append turns them (one rounding to bf16)
    want, size = turned(q.double().cpu().numpy(), pos, plan)
    off = np.abs(out.double().cpu().numpy() - want)
    assert np.all(off <= size * 2.0 ** -20 + np.abs(want) * 2.0 ** -8)
    # keys: the scale is the largest turned element's, and each value is within half a
    # step of its code (one more rounding where a kept row was rounded again)
    want, size = turned(k.double().cpu().numpy(), pos, plan)
    want, size = torch.from_numpy(want), torch.from_numpy(size)
    qmax = float(q8_ref.QMAX[dtype])
    flat = before.transpose(1, 2).reshape(-1, hkv, D)
    old = c.ks.double().transpose(1, 2).reshape(-1, hkv)
    new_rows = torch.zeros(flat.shape[0], dtype=torch.bool)
    held = slots >= 0
    new_rows[slots[held]] = True
    starts = new_rows[::16]
    old = torch.where(starts[:, None], 0.0, old)
    amax = torch.zeros(flat.shape[0], hkv, dtype=torch.float64)
    amax[slots[held]] = want[held].abs().amax(-1)
    err = torch.zeros_like(amax)
    err[slots[held]] = size[held].amax(-1) * 2.0 ** -20
    touched = new_rows.view(-1, 16).any(1)
    expect = torch.where(touched[:, None], torch.maximum(old, amax.view(-1, 16, hkv).amax(1) / qmax),
                         old)
    slack = err.view(-1, 16, hkv).amax(1) / qmax + expect * 2.0 ** -22
    got_scale = c.dev[2].cpu().double().transpose(1, 2).reshape(-1, hkv)
    assert bool(((got_scale - expect).abs() <= torch.where(touched[:, None], slack, 0.0))[
        touched].all())
    got = q8_ref.values(c.dev[0].cpu(), c.dev[2].cpu()).transpose(1, 2).reshape(-1, hkv, D)
    s = got_scale.repeat_interleave(16, 0)[..., None]
    target = flat.clone()
    target[slots[held]] = want[held]
    fuzz = torch.zeros_like(target)
    fuzz[slots[held]] = size[held] * 2.0 ** -20
    keep = touched.repeat_interleave(16) & ~starts.repeat_interleave(16)
    check = new_rows | keep
    if dtype == torch.int8:
        half = s * 0.5
    else:  # half a step of e4m3: 2^-4 relative, 2^-10 below the normal range
        half = torch.maximum(target.abs() * 2.0 ** -4, s * 2.0 ** -10)
    bound = half * (1 + 2.0 ** -20) + fuzz + target.abs() * 2.0 ** -22
    assert bool(((got - target).abs() <= bound)[check].all())
    empty = starts.repeat_interleave(16) & ~new_rows  # rows of a new group that nothing wrote
    assert bool((got[empty] == 0).all())


@pytest.mark.parametrize("dtype", q8_ref.FORMATS)
@pytest.mark.parametrize("interleaved,rotary", [(False, 64), (False, 50), (True, 64)])
def test_rope_non_finite(dtype, interleaved, rotary):
    """NaN and infinities among the keys change no other code and no scale."""
    T, hq, hkv = 40, 4, 2
    plan = pkv.RopePlan(rotary, interleaved=interleaved)
    q, k, v = (torch.randn(T, n, D, device=DEV).bfloat16() for n in (hq, hkv, hkv))
    pos = torch.arange(T, dtype=torch.int32, device=DEV) + 77
    slots = torch.arange(T, device=DEV)
    odd = {(3, 0, 100): math.nan, (3, 1, 127): math.inf, (20, 0, 64): -math.inf,
           (39, 1, 90): math.nan}  # past the rotated part
    caches = [Cache(3, hkv, 16, dtype) for _ in range(2)]
    for c, put in zip(caches, (False, True)):
        for at, x in odd.items():
            k[at] = x if put else 0.0
        pkv.rope_append_q8(pos, slots, q, k, v, *c.dev, plan)
    clean, got = ([x.cpu() for x in c.dev] for c in caches)
    for (t, h, e), x in odd.items():
        code = got[0][t // 16, h, t % 16, e].float()
        assert code.isnan() if math.isnan(x) and dtype != torch.int8 else \
            code == (0.0 if math.isnan(x) else math.copysign(float(q8_ref.QMAX[dtype]), x))
        got[0].view(torch.int8)[t // 16, h, t % 16, e] = clean[0].view(torch.int8)[t // 16, h,
                                                                                   t % 16, e]
    for a, b in zip(clean, got):
        assert torch.equal(a.view(torch.int8), b.view(torch.int8))


@pytest.mark.parametrize("interleaved,rotary", [(False, 128), (False, 50), (True, 128)])
def test_rope_one_launch_or_two(interleaved, rotary):
    """Queries and keys of 1000 tokens in one launch, of more in two: the same bits."""
    T, hq, hkv = 1040, 4, 1
    plan = pkv.RopePlan(rotary, interleaved=interleaved)
    q, k, v = (torch.randn(T, n, D, device=DEV).bfloat16() for n in (hq, hkv, hkv))
    pos = torch.arange(T, dtype=torch.int32, device=DEV) + 70000
    slots = torch.arange(T, device=DEV)
    both = [Cache(66, hkv, 16, torch.int8) for _ in range(2)]
    whole = pkv.rope_append_q8(pos, slots, q, k, v, *both[0].dev, plan)
    parts = [pkv.rope_append_q8(*(x[at] for x in (pos, slots, q, k, v)), *both[1].dev, plan)
             for at in (slice(0, 992), slice(992, T))]  # whole groups
    assert torch.equal(whole, torch.cat(parts))
    for a, b in zip(both[0].dev, both[1].dev):
        assert torch.equal(a, b)


def test_rope_equals_the_parts():
    """Queries are what rope_append gives, values what kv_append_q8 gives; in place too.
    Both calls turn in fp32 and round once, but which of a turn's two products is
    rounded before the sum is each kernel's own: the fp32 results are within
    2 * 2^-24 of |a cos| + |b sin| <= |a| + |b| of one another, and two numbers that
    close round to the same bf16 or to neighbours, a step (2^-7 of the value) apart."""
    T, hq, hkv = 130, 8, 4
    plan = pkv.RopePlan(96, scaling={"kind": "linear", "factor": 4.0})
    q, k, v = (torch.randn(T, n, D, device=DEV).bfloat16() for n in (hq, hkv, hkv))
    pos = torch.arange(T, dtype=torch.int32, device=DEV) + 5000
    slots = torch.arange(T, device=DEV)
    c = Cache(9, hkv, 16, torch.int8)
    bk, bv = (torch.zeros(9, hkv, 16, D, device=DEV).bfloat16() for _ in range(2))
    want = pkv.rope_append(pos, slots, q, k, v, bk, bv, plan)
    mine = q.clone()
    got = pkv.rope_append_q8(pos, slots, mine, k, v, *c.dev, plan, out=mine)
    assert got is mine
    _, size = turned(q.double().cpu().numpy(), pos.cpu(), plan)
    off = (got.double() - want.double()).abs().cpu().numpy()
    assert np.all(off <= np.abs(want.double().cpu().numpy()) * 2.0 ** -7 + size * 2.0 ** -23)
    assert np.mean(off > 0) < 0.001
    q8_ref.append(c.v, c.vs, slots.cpu(), v.cpu().float())
    assert torch.equal(c.dev[1].cpu(), c.v) and torch.equal(c.dev[3].cpu(), c.vs)
