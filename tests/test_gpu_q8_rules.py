"""Rules of the appends to the 8-bit cache, each by its own small case: slots that tokens
share, groups without a finite value but zero, rows that are written over later
(rejected drafts)."""
import math

import pytest
import torch

import paged_kv_cache_245_gb300 as pkv
import q8_ref

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
D = 128


class Group:
    """One block of 16 rows and one head, with the append (and the rotary append)."""

    def __init__(self, dtype, rope=False):
        self.k, self.v = (torch.zeros(1, 1, 16, D, device=DEV).to(dtype) for _ in range(2))
        self.ks, self.vs = (torch.zeros(1, 1, 1, device=DEV) for _ in range(2))
        self.plan = pkv.RopePlan(128) if rope else None
        self.dtype = dtype

    def put(self, slots, x):
        x = x.to(DEV).bfloat16()[:, None]
        slots = torch.tensor(slots, device=DEV)
        cache = (self.k, self.v, self.ks, self.vs)
        if self.plan is None:
            pkv.kv_append_q8(slots, x, x, *cache)
        else:  # position 0: keys as they are
            pos = torch.zeros(len(slots), dtype=torch.int32, device=DEV)
            pkv.rope_append_q8(pos, slots, x, x, x, *cache, self.plan)
        return self

    def same_as(self, other):
        for a, b in ((self.k, other.k), (self.v, other.v), (self.ks, other.ks), (self.vs, other.vs)):
            assert torch.equal(a.view(torch.int8), b.view(torch.int8))


def rows(g):
    return [q8_ref.values(c.cpu(), s.cpu())[0, 0] for c, s in ((g.k, g.ks), (g.v, g.vs))]


def normal(n, seed=0, by=1.0):
    return (torch.randn(n, D, generator=torch.Generator().manual_seed(seed)) * by).bfloat16().float()


both = pytest.mark.parametrize("rope", [False, True])
formats = pytest.mark.parametrize("dtype", q8_ref.FORMATS)


@both
@formats
@pytest.mark.parametrize("slots", [[0, 1, 1], [1, 0, 1], [5, 5, 5]])
def test_the_last_token_of_a_slot_counts_alone(dtype, rope, slots):
    """A larger row that a later token of the call overwrites leaves no mark."""
    x = normal(3)
    for t in range(2):
        if slots[t] in slots[t + 1:]:
            x[t] *= 1000.0
    got = Group(dtype, rope).put(slots, x)
    last = {s: t for t, s in enumerate(slots)}
    want = Group(dtype, rope).put(list(last), x[list(last.values())])
    got.same_as(want)
    assert float(got.ks) < 1.0 and float(got.vs) < 1.0


@formats
def test_infinities(dtype):
    """The largest code beside finite values; with inv 0 what inf x 0 is: NaN, in int8 0."""
    x = normal(2)
    x[0, 3], x[1, 7] = math.inf, -math.inf
    g = Group(dtype).put([0, 1], x)
    top = float(q8_ref.QMAX[dtype])
    assert float(g.k[0, 0, 0, 3].float()) == top and float(g.v[0, 0, 1, 7].float()) == -top
    x = torch.zeros(2, D)
    x[0, 3], x[1, 7] = math.inf, -math.inf
    g = Group(dtype).put([0, 1], x)
    assert float(g.ks) == 0.0
    for c in (g.k[0, 0, 0, 3].float(), g.v[0, 0, 1, 7].float()):
        assert float(c) == 0.0 if dtype == torch.int8 else bool(c.isnan())
    assert float(g.k.float().nan_to_num().abs().sum()) == 0.0


def half_step(x, scale, dtype):
    """Half a step of the codes of values x with the given scale."""
    if dtype == torch.int8:
        return torch.full_like(x, scale / 2)
    return torch.maximum(x.abs() * 2.0 ** -4, torch.full_like(x, scale * 2.0 ** -10))


@both
@formats
@pytest.mark.parametrize("by", [1.0, 4.0, 30.0])
def test_rejected_drafts(dtype, rope, by):
    """Five rows, three drafts `by` times as large, then other rows in the drafts' slots: the
    scale stays that of the drafts.  Each row is within half a step of it, the rows before the
    drafts by one more rounding with the smaller scale (2^-20: fp32's own)."""
    x, drafts, after = normal(5), normal(3, 1, by), normal(4, 2)
    g = Group(dtype, rope).put(range(5), x)
    first = float(g.ks)
    g.put([5, 6, 7], drafts)
    grown = float(g.ks)
    assert grown >= first and (by == 1.0 or grown > first)
    g.put([5, 6, 7, 8], after)
    assert float(g.ks) == pytest.approx(
        max(grown, float(after.abs().max()) / float(q8_ref.QMAX[dtype])), rel=2.0 ** -22)
    scale = float(g.ks)
    for got in rows(g):
        want = torch.cat([x, after]).double()
        bound = half_step(want, scale, dtype)
        once = half_step(want[:5], first, dtype)
        if scale > first:  # the second rounding is of a value that the first has moved
            bound[:5] = once + half_step(want[:5].abs() + once, scale, dtype)
        assert bool(((got[:9] - want).abs() <= bound * (1 + 2.0 ** -20)).all())
        assert bool((got[9:] == 0).all())


@both
@formats
def test_drafts_taken_back(dtype, rope):
    """The tail block copied before the drafts, and back, leaves no trace of them."""
    x, drafts, after = normal(5), normal(3, 1, 30.0), normal(2, 2)
    want = Group(dtype, rope).put(range(5), x).put([5, 6], after)
    g = Group(dtype, rope)
    for name in ("k", "v", "ks", "vs"):  # a second block to keep the tail in
        t = getattr(g, name)
        setattr(g, name, torch.cat([t.view(torch.int8), t.view(torch.int8)]).view(t.dtype))
    g.put(range(5), x)
    there, back = (torch.tensor([p], device=DEV) for p in ([0, 1], [1, 0]))
    for pairs, put in ((there, lambda: g.put([5, 6, 7], drafts)), (back, lambda: g.put([5, 6], after))):
        pkv.block_copy(pairs, [g.k], [g.v])
        pkv.block_copy(pairs, [g.ks], [g.vs])
        put()
    for name in ("k", "v", "ks", "vs"):
        assert torch.equal(getattr(g, name)[:1].view(torch.int8), getattr(want, name).view(torch.int8))
