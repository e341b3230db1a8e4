"""Prefill attention with capped, biased and masked scores against the formula
in 64 bits: head groups, block sizes, chunks over cached positions, prefixes,
documents, rows that see nothing, poisoned masked places, graphs, refusals;
and a layer's flow: rotary append, prefill, decode steps."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import paged_kv_cache_245_gb300 as pkv
from scored_ref import Sequences, assert_close, attend64, visible

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
D = 128
SCALE = D ** -0.5


@pytest.fixture(autouse=True)
def _reset():
    pkv.set_checked(False)
    yield
    pkv.set_checked(False)
    torch.cuda.synchronize()


class Chunks(Sequences):
    def __init__(self, cached, new, hq, hkv, bs, contig=False, seed=1, by=4.0, tail=0):
        super().__init__([c + n for c, n in zip(cached, new)], hkv, bs, contig, seed)
        self.new, self.hq = list(new), hq
        self.cu = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device=DEV)
        self.T = sum(new)
        self.q = (torch.randn(self.T + tail, hq, D, generator=self.g, device=DEV) * by).bfloat16()

    def positions(self):
        return [(i, p) for i, (c, n) in enumerate(zip(self.ctx, self.new)) for p in range(c - n, c)]

    def ranges(self, window=0, first=None, prefix=None):
        return [visible(p, 0 if first is None else int(first[t]), window,
                        0 if prefix is None else int(prefix[i]), self.ctx[i])
                for t, (i, p) in enumerate(self.positions())]

    def reference(self, window=0, first=None, prefix=None, softcap=0.0, slopes=None, scale=SCALE):
        first = None if first is None else first.tolist()
        rng = self.ranges(window, first, prefix)
        out = torch.zeros(self.T, self.hq, D, dtype=torch.float64, device=DEV)
        tol = torch.zeros_like(out)
        at = 0
        for i, n in enumerate(self.new):
            if n == 0:
                continue
            r = rng[at:at + n]
            out[at:at + n], tol[at:at + n] = attend64(
                self.q[at:at + n], self.rows(i, self.k), self.rows(i, self.v),
                list(range(self.ctx[i] - n, self.ctx[i])), r, scale, softcap, slopes)
            at += n
        return out, tol

    def call(self, k=None, v=None, scale=SCALE, q=None, **kw):
        f = pkv.contig_prefill_attention_scored if self.contig else pkv.paged_prefill_attention_scored
        return f(self.q if q is None else q, self.cu, self.k if k is None else k,
                 self.v if v is None else v, self.where, self.ctx_t, max(max(self.new), 1), scale,
                 **kw)


def documents(s, every, seed=0):
    """The start of each token's document, `every` positions long on average."""
    r, out = np.random.default_rng(seed), []
    for c, n in zip(s.ctx, s.new):
        starts = np.concatenate([[0], np.cumsum(r.integers(1, 2 * every, size=c + 1))])
        out += [int(starts[starts <= p][-1]) for p in range(c - n, c)]
    return torch.tensor(out, dtype=torch.int32, device=DEV)


def slopes_of(hq):
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / hq) for h in range(hq)], device=DEV)


SCORES = {
    "plain": dict(),
    "cap": dict(softcap=50.0),
    "small cap": dict(softcap=0.5),
    "wide cap": dict(softcap=80.0),
    "huge cap": dict(softcap=1e6),
    "window 1": dict(window=1),
    "window 100": dict(window=100),
    "cap, window 33": dict(window=33, softcap=30.0),
    "window past all": dict(window=2 ** 31 - 1),
    "slopes": dict(slopes=True),
    "slopes, cap": dict(slopes=True, softcap=30.0),
    "documents": dict(first=37),
    "cap, documents": dict(first=150, softcap=50.0),
    "prefix": dict(prefix=True),
    "all": dict(softcap=20.0, window=130, slopes=True, first=90, prefix=True),
}


def make(name, s):
    kw = dict(SCORES[name])
    if kw.pop("slopes", False):
        kw["slopes"] = slopes_of(s.hq)
    if "first" in kw:
        kw["first"] = documents(s, kw["first"])
    if kw.pop("prefix", False):
        # none, inside the cached part, inside the chunk, all, past the context
        kw["prefix"] = torch.tensor([[0, c // 3, c - n // 2, c, c + 500, 1][i % 6]
                                     for i, (c, n) in enumerate(zip(s.ctx, s.new))],
                                    dtype=torch.int32, device=DEV)
    return kw, dict(softcap=kw.get("softcap", 0.0), window=kw.get("window", 0),
                    alibi_slopes=kw.get("slopes"), first_key=kw.get("first"),
                    prefix_lens=kw.get("prefix"))


CACHED, NEW = [0, 3, 100, 64, 17, 0, 500], [1, 5, 64, 65, 130, 300, 0]


@pytest.mark.parametrize("name", list(SCORES))
@pytest.mark.parametrize("contig", [False, True])
def test_scores(name, contig):
    s = Chunks(CACHED, NEW, 32, 8, 16, contig, seed=3)
    ref, kw = make(name, s)
    assert_close(s.call(**kw), *s.reference(**ref), what=name)


@pytest.mark.parametrize("hq,hkv", [(2, 2), (4, 2), (3, 1), (8, 2), (10, 2), (6, 1), (56, 8), (32, 4)])
@pytest.mark.parametrize("bs", [16, 48, 128, 256])
def test_groups_and_block_sizes(hq, hkv, bs):
    s = Chunks([0, 130, 7, 600], [200, 70, 1, 33], hq, hkv, bs, seed=hq + bs)
    for name in ("cap", "all", "window 100"):
        ref, kw = make(name, s)
        assert_close(s.call(**kw), *s.reference(**ref), what=name)


@pytest.mark.parametrize("name", ["cap", "cap, window 33", "slopes", "cap, documents", "all", "window 100"])
def test_long_chunks(name):
    """Many key tiles, several work items a sequence."""
    s = Chunks([0, 1500, 20], [900, 700, 1300], 8, 2, 16, seed=5)
    ref, kw = make(name, s)
    assert_close(s.call(**kw), *s.reference(**ref), what=name)


@pytest.mark.parametrize("hq,hkv", [(32, 8), (7, 1), (4, 4)])
@pytest.mark.parametrize("name", ["plain", "cap", "small cap", "window 100", "slopes", "documents", "all"])
@pytest.mark.parametrize("contig", [False, True])
def test_few_tokens_after_many(name, hq, hkv, contig):
    """Few work items with many key tiles: several CTAs share an item."""
    for cached, new in (([4000], [1]), ([3000, 0], [70, 3]), ([257, 2600, 0], [40, 1, 0])):
        s = Chunks(cached, new, hq, hkv, 16, contig, seed=hq + len(cached))
        ref, kw = make(name, s)
        assert_close(s.call(**kw), *s.reference(**ref), what=name)


def test_few_tokens_after_many_poisoned_captured_and_side_by_side():
    s = Chunks([4000, 1500], [33, 2], 8, 2, 16, seed=31)
    first = torch.tensor([0] * 10 + [2500] * 23 + [700, 1200], dtype=torch.int32, device=DEV)
    want = s.reference(first=first, softcap=30.0)
    k, v = s.poison([(0, 4032), (700, 1501)])
    bad = (int(s.where[0, 1000 // 16]), 1000 % 16)  # seen by the first ten tokens alone
    k[bad[0], :, bad[1]] = v[bad[0], :, bad[1]] = float("nan")
    got = s.call(k=k, v=v, softcap=30.0, first_key=first)
    assert bool(torch.isnan(got[:10]).all())
    assert_close(got[10:], want[0][10:], want[1][10:])
    k[bad[0], :, bad[1]] = s.k[bad[0], :, bad[1]]
    v[bad[0], :, bad[1]] = s.v[bad[0], :, bad[1]]
    out = torch.empty(s.T, 8, D, dtype=torch.bfloat16, device=DEV)
    kw = dict(softcap=30.0, first_key=first)
    s.call(k=k, v=v, out=out, **kw)
    assert_close(out, *want)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        s.call(k=k, v=v, out=out, **kw)
    other = torch.empty_like(out)
    for _ in range(5):
        out.fill_(7.0)
        other.fill_(7.0)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            s.call(k=k, v=v, out=other, **kw)
        graph.replay()
        torch.cuda.current_stream().wait_stream(side)
        assert_close(out, *want)
        assert torch.equal(out, other)


@pytest.mark.parametrize("cap", [20.0, 200.0])
def test_results_do_not_hang_on_what_stands_in_shared_memory(cap):
    """The same bits whatever the kernel before left behind for masked columns."""
    s = Chunks([40, 300, 5], [100, 30, 260], 32, 8, 16, seed=33, by=1.0)
    big = Chunks([0], [600], 32, 8, 16, seed=34, by=400.0)
    big.k *= 20.0
    kw = dict(softcap=cap, window=90)
    want = s.call(**kw)
    for _ in range(3):
        big.call(softcap=cap)
        assert torch.equal(s.call(**kw), want)


@pytest.mark.parametrize("name", ["plain", "documents", "prefix", "cap", "window 100"])
def test_slopes_of_any_size(name):
    """From none to so steep that a row sees one key, rising instead of falling too."""
    s = Chunks([0, 500, 30], [400, 33, 200], 16, 4, 16, seed=41)
    slopes = torch.tensor([0.0, 1e-6, 0.3, 1.3, 0.5, 1.0, 1.38, 1.4, 3.0, 100.0, 2.0, 0.1,
                           -0.01, -0.5, -4.0, 1e4], device=DEV)
    ref, kw = make(name, s)
    ref["slopes"] = kw["alibi_slopes"] = slopes
    want, tol = s.reference(**ref)
    assert_close(s.call(**kw), want, tol)


RAGGED = ([0, 3, 700, 0, 64, 900, 17, 0, 5, 300, 0, 2], [0, 1, 500, 64, 65, 3, 700, 129, 0, 40, 900, 5])


@pytest.mark.parametrize("hq,hkv", [(32, 8), (56, 8), (6, 6)])
@pytest.mark.parametrize("name", ["window 100", "cap", "slopes", "cap, documents", "all"])
def test_more_items_than_sms(name, hq, hkv):
    """A ragged batch whose work items are sorted and dealt on demand."""
    s = Chunks(*RAGGED, hq, hkv, 16, seed=hq)
    ref, kw = make(name, s)
    assert_close(s.call(**kw), *s.reference(**ref), what=name)


@pytest.mark.parametrize("count", [160, 700, 730])
def test_hundreds_of_short_chunks(count):
    """One item a sequence: up to the sorted list's length, and past it."""
    s = Chunks([i % 50 for i in range(count)], [1 + i % 3 for i in range(count)], 8, 1, 16, seed=7)
    for name in ("cap", "window 33", "documents"):
        kw = dict(window=33) if name == "window 33" else make(name, s)[1]
        ref = dict(window=33) if name == "window 33" else make(name, s)[0]
        assert_close(s.call(**kw), *s.reference(**ref), what=name)


def test_more_items_than_sms_checked_captured_and_on_two_streams():
    s = Chunks(*RAGGED, 32, 8, 16, seed=21)
    ref, kw = make("cap", s)
    want, tol = s.reference(**ref)
    out = torch.empty(s.T, 32, D, dtype=torch.bfloat16, device=DEV)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    s.call(out=out, **kw)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        s.call(out=out, **kw)
    other = torch.empty_like(out)
    for _ in range(5):  # each replay beside an eager call on another stream
        out.fill_(7.0)
        other.fill_(7.0)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            s.call(out=other, **kw)
        graph.replay()
        torch.cuda.current_stream().wait_stream(side)
        assert_close(out, want, tol)
        assert_close(other, want, tol)
    # a sequence longer than its context is left unwritten, the others are not
    pkv.set_checked(True)
    s.ctx_t = s.ctx_t.clone()
    s.ctx_t[4] = 64
    out.fill_(7.0)
    s.call(out=out, **kw)
    assert pkv.get_device_error() == "context"
    a, b = int(s.cu[4]), int(s.cu[5])
    assert bool((out[a:b] == 7.0).all())
    keep = torch.ones(s.T, dtype=torch.bool, device=DEV)
    keep[a:b] = False
    assert_close(out[keep], want[keep], tol[keep])


@pytest.mark.parametrize("by", [0.0, 30.0, 300.0])
@pytest.mark.parametrize("scale", [SCALE, -SCALE])
def test_saturating_scores(by, scale):
    s = Chunks([0, 200], [300, 40], 8, 2, 16, seed=6, by=by)
    for cap in (0.0, 5.0, 50.0, 60.0, 1000.0):
        assert_close(s.call(scale=scale, softcap=cap), *s.reference(scale=scale, softcap=cap),
                     what="cap %g" % cap)


def test_rows_whose_scores_are_all_at_the_low_end_of_the_cap():
    """Every score of a row near -softcap: exponentials of the lowest arguments."""
    s = Chunks([0, 60], [130, 10], 8, 2, 16, seed=7)
    s.q = torch.full_like(s.q, -60.0)
    s.k = s.k.abs() + 1
    for cap in (30.0, 50.0, 51.9, 53.0, 200.0):
        assert_close(s.call(softcap=cap), *s.reference(softcap=cap), what="cap %g" % cap)
    s.q = -s.q  # and at the high end
    for cap in (30.0, 50.0, 51.9, 53.0, 200.0):
        assert_close(s.call(softcap=cap), *s.reference(softcap=cap), what="cap %g" % cap)


def test_scores_that_grow_along_the_row():
    """The running maximum moves in every tile."""
    s = Chunks([0], [700], 4, 1, 16, seed=8)
    s.q[:] = 1.0
    ramp = torch.arange(700, device=DEV) / 700 * 300
    k = s.rows(0, s.k)
    s.k.zero_()
    n = (700 + 15) // 16
    k = torch.cat([ramp[None, :, None].expand(1, 700, D) / (D * SCALE),
                   torch.zeros(1, n * 16 - 700, D, device=DEV)], 1).bfloat16()
    s.k[s.where[0, :n].long()] = k.view(1, n, 16, D).transpose(0, 1)
    for name in ("plain", "cap", "wide cap", "window 100", "slopes, cap"):
        ref, kw = make(name, s)
        assert_close(s.call(**kw), *s.reference(**ref), what=name)


def test_rows_that_see_nothing_and_rows_behind_the_last_chunk():
    s = Chunks([0, 40, 300], [70, 200, 5], 32, 8, 16, seed=9, tail=9)
    pos = torch.tensor([p for _, p in s.positions()], dtype=torch.int32, device=DEV)
    first = torch.zeros(s.T + 9, dtype=torch.int32, device=DEV)
    first[:s.T] = pos + 1  # every row empty
    first[5:60] = 3
    first[100:300:3] = 2 ** 31 - 1
    first[101:300:3] = -2 ** 31
    for cap in (0.0, 50.0):
        out = torch.full_like(s.q, 7.0)
        assert s.call(softcap=cap, first_key=first, out=out) is out
        assert bool((out[s.T:] == 7.0).all())
        want = s.reference(softcap=cap, first=first[:s.T])
        assert_close(out[:s.T], *want)
        lo = torch.tensor(s.ranges(first=first[:s.T].tolist()), device=DEV)
        empty = lo[:, 0] > lo[:, 1]
        assert int(empty.sum()) > 50 and bool((out[:s.T][empty] == 0).all())


@pytest.mark.parametrize("contig,bs", [(False, 16), (False, 48), (False, 128), (True, 16)])
@pytest.mark.parametrize("name", ["plain", "cap", "window 1", "window 100", "cap, window 33", "all"])
def test_nothing_in_masked_places_matters(name, contig, bs):
    """Cache rows that no token of the chunk sees hold NaN and infinities."""
    s = Chunks([0, 3, 400, 64, 700], [1, 5, 64, 165, 30], 8, 2, bs, contig, seed=10)
    ref, kw = make(name, s)
    keep, at = [], 0
    rng = s.ranges(ref.get("window", 0), None if "first" not in ref else ref["first"].tolist(),
                   ref.get("prefix"))
    for n in s.new:
        keep.append((min(a for a, b in rng[at:at + n] if a <= b),
                     max(b for a, b in rng[at:at + n] if a <= b)))
        at += n
    k, v = s.poison(keep)
    assert_close(s.call(k=k, v=v, **kw), *s.reference(**ref), what=name)


@pytest.mark.parametrize("cap", [0.0, 50.0, 200.0])
@pytest.mark.parametrize("G", [4, 7])
def test_a_poisoned_document_leaves_its_neighbours_alone(cap, G):
    """Three packed documents; the middle one's keys and values are NaN and
    infinities, in key tiles that the others' rows share with it."""
    s = Chunks([0], [300], 2 * G, 2, 16, seed=11)
    starts = [0, 90, 150]
    first = torch.tensor([max(x for x in starts if x <= p) for p in range(300)], dtype=torch.int32,
                         device=DEV)
    want, tol = s.reference(softcap=cap, first=first)
    n = (300 + 15) // 16
    for x, bad in ((s.k, float("nan")), (s.v, float("inf"))):
        rows = s.rows(0, x)
        rows[:, 90:150] = bad
        rows = torch.cat([rows, torch.zeros(2, n * 16 - 300, D, device=DEV).bfloat16()], 1)
        x[s.where[0, :n].long()] = rows.view(2, n, 16, D).transpose(0, 1)
    got = s.call(softcap=cap, first_key=first)
    other = torch.tensor([p < 90 or p >= 150 for p in range(300)], device=DEV)
    assert_close(got[other], want[other], tol[other])
    assert bool(torch.isnan(got[~other]).all())


def test_future_values_do_not_leak():
    """A NaN or infinite value at position j reaches rows at j and later only."""
    for at in (0, 77, 128, 255):
        s = Chunks([0], [256], 8, 2, 16, seed=12)
        want, tol = s.reference(softcap=50.0)
        s.v[int(s.where[0, at // 16]), :, at % 16] = float("inf")
        got = s.call(softcap=50.0)
        assert_close(got[:at], want[:at], tol[:at]) if at else None
        assert not bool(torch.isfinite(got[at:]).any())


def test_chunk_of_one_token_is_the_decode_call():
    s = Chunks([0, 16, 99, 700], [1, 1, 1, 1], 32, 8, 16, seed=13)
    first = torch.tensor([0, 4, 99, 200], dtype=torch.int32, device=DEV)
    kw = dict(softcap=30.0, window=300, alibi_slopes=slopes_of(32), first_key=first)
    want = s.reference(softcap=30.0, window=300, slopes=slopes_of(32), first=first)
    assert_close(s.call(**kw), *want)
    dec = pkv.paged_decode_attention_scored(s.q, s.k, s.v, s.where, s.ctx_t, 701, SCALE, **kw)
    assert_close(dec, *want)


def test_null_score_is_the_plain_call():
    s = Chunks([0, 100], [300, 40], 32, 8, 16, seed=14)
    plain = pkv.paged_prefill_attention(s.q, s.cu, s.k, s.v, s.where, s.ctx_t, 300, SCALE).double()
    assert_close(s.call(), plain, 2.0 ** -7 * plain.abs() + 2.0 ** -7)


@pytest.mark.parametrize("bs", [16, 48])
def test_blocks_that_no_token_sees_are_never_read(bs):
    s = Chunks([300, 0, 500], [70, 90, 3], 8, 2, bs, seed=15)
    want = s.reference(window=50, softcap=50.0)
    for i, (c, n) in enumerate(zip(s.ctx, s.new)):
        s.where[i, :max(0, c - n - 49) // bs] = -1
        s.where[i, (c + bs - 1) // bs:] = 1 << 30
    pkv.set_checked(True)
    got = s.call(window=50, softcap=50.0)
    assert pkv.get_device_error() == "none"
    assert_close(got, *want)
    s.where[0, 360 // bs] = -1  # a visible one is reported
    s.call(window=50)
    assert pkv.get_device_error() == "block_id"


def test_checked_mode_reports_a_chunk_longer_than_its_context():
    s = Chunks([5, 0], [20, 30], 8, 2, 16, seed=16)
    pkv.set_checked(True)
    s.ctx_t[0] = 10
    s.call(softcap=50.0)
    assert pkv.get_device_error() == "context"


def test_alignment_of_out():
    """out 16-byte but not 32-byte aligned, heads that do not divide a tile."""
    for hq, hkv in ((7, 1), (4, 1)):
        s = Chunks([10], [100], hq, hkv, 16, seed=17)
        out = torch.empty(100 * hq * D + 8, dtype=torch.bfloat16, device=DEV)[8:].view(100, hq, D)
        assert_close(s.call(softcap=50.0, out=out), *s.reference(softcap=50.0))


def test_graph_and_streams():
    s = Chunks([0, 300, 20], [500, 70, 1], 32, 8, 16, seed=18)
    ref, kw = make("cap, documents", s)
    want = s.reference(**ref)
    out = torch.zeros_like(s.q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        there = s.call(**kw)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            s.call(out=out, **kw)
    torch.cuda.synchronize()
    assert_close(there, *want)
    for _ in range(2):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, there)


def test_binding_refusals():
    s = Chunks([0, 4], [20, 3], 8, 2, 16, seed=19)
    i32 = dict(dtype=torch.int32, device=DEV)
    for kw, error in ((dict(softcap=-1.0), pkv.PkvError), (dict(softcap=float("inf")), pkv.PkvError),
                      (dict(window=-3), pkv.PkvError), (dict(scale=float("nan")), pkv.PkvError),
                      (dict(alibi_slopes=torch.ones(4, device=DEV)), ValueError),
                      (dict(first_key=torch.zeros(2, **i32)), ValueError),
                      (dict(prefix_lens=torch.zeros(3, **i32)), ValueError),
                      (dict(prefix_lens=torch.zeros(2, device=DEV)), TypeError),
                      (dict(prefix_lens=torch.zeros(4, **i32)[::2]), ValueError),
                      (dict(out=torch.empty_like(s.q)[1:]), ValueError)):
        with pytest.raises(error):
            s.call(**kw)
    odd = Chunks([0], [20], 8, 2, 24, seed=20)
    with pytest.raises(pkv.PkvError):
        odd.call(softcap=5.0)


def test_a_layer_prefills_and_decodes():
    """One layer as it is used: prompts turned and appended, attended under a
    cap and a window, then decode steps that grow the cache, each stage against
    the formula in 64 bits."""
    hq, hkv, bs, window, cap = 8, 2, 16, 60, 30.0
    prompts, steps = [70, 1, 33], 20
    plan = pkv.RopePlan(64, theta=1e4, scaling={"kind": "parts", "factor": 4, "original": 64})
    bm = pkv.BlockManager(40, bs)
    ids = [bm.add_sequence(n) for n in prompts]
    g = torch.Generator(device=DEV).manual_seed(21)
    kc, vc = (torch.full((40, hkv, bs, D), float("nan"), device=DEV).bfloat16() for _ in "kv")

    def project(n):
        qkv = torch.randn(n, (hq + 2 * hkv) * D, generator=g, device=DEV).bfloat16()
        return [x.unflatten(1, (-1, D)) for x in qkv.split([hq * D, hkv * D, hkv * D], 1)]

    def dev(a):
        return torch.as_tensor(np.ascontiguousarray(a), device=DEV)

    turn = np.array([int(x) for x in plan.c.turn[:32]], dtype=object)

    def check_turned(got, x, pos):
        """Rows as the library turned them: one rounding to bf16 (2^-8) and fp32
        arithmetic (under 2^-20 of the pair) from the formula in 64 bits."""
        frac = np.array([[(int(p) * t % 2 ** 64) / 2 ** 64 for t in turn] for p in pos])
        c, sn = (dev(f(2 * np.pi * frac))[:, None] * float(plan.c.gain) for f in (np.cos, np.sin))
        y, size = x.double().clone(), torch.zeros_like(x, dtype=torch.float64)
        a, b = x[..., :32].double(), x[..., 32:64].double()
        y[..., :32], y[..., 32:64] = a * c - b * sn, b * c + a * sn
        size[..., :32] = size[..., 32:64] = (a.abs() + b.abs()) * float(plan.c.gain)
        assert bool(((got.double() - y).abs() <= y.abs() * 2.0 ** -8 + size * 2.0 ** -20).all())

    history = [([], []) for _ in prompts]

    def remember(i, k, v, pos, slots):
        """The rows of new positions, as the caches hold them at their slots."""
        at = dev(slots)
        kr, vr = (x.transpose(1, 2).reshape(-1, hkv, D)[at] for x in (kc, vc))
        check_turned(kr, k, pos)
        assert torch.equal(vr, v)
        history[i][0].append(kr)
        history[i][1].append(vr)

    def check(out, qt, i, pos, what):
        k, v = (torch.cat(x).transpose(0, 1) for x in history[i])
        rng = [visible(p, 0, window, 0, p + 1) for p in pos]
        assert_close(out, *attend64(qt, k, v, pos, rng, SCALE, cap), what)

    tables, ctx = bm.export(ids, 8)
    cu = np.concatenate([[0], np.cumsum(prompts)]).astype(np.int32)
    pos = np.concatenate([np.arange(n) for n in prompts]).astype(np.int32)
    slots = np.concatenate([tables[i, np.arange(n) // bs].astype(np.int64) * bs + np.arange(n) % bs
                            for i, n in enumerate(prompts)])
    q, k, v = project(int(cu[-1]))
    qt = pkv.rope_append(dev(pos), dev(slots), q, k, v, kc, vc, plan)
    out = pkv.paged_prefill_attention_scored(qt, dev(cu), kc, vc, dev(tables), dev(ctx),
                                             max(prompts), SCALE, softcap=cap, window=window)
    check_turned(qt, q, pos)
    for i, n in enumerate(prompts):
        rows = slice(int(cu[i]), int(cu[i + 1]))
        remember(i, k[rows], v[rows], range(n), slots[rows])
        check(out[rows], qt[rows], i, list(range(n)), "prompt %d" % i)
    for step in range(steps):
        slots, pairs = bm.append(ids)
        assert len(pairs) == 0
        tables, ctx = bm.export(ids, 8)
        q, k, v = project(len(ids))
        qt = pkv.rope_append(dev((ctx - 1).astype(np.int32)), dev(slots), q, k, v, kc, vc, plan)
        out = pkv.paged_decode_attention_scored(qt, kc, vc, dev(tables), dev(ctx), int(ctx.max()),
                                                SCALE, softcap=cap, window=window)
        for i in range(len(ids)):
            p = [int(ctx[i]) - 1]
            remember(i, k[i:i + 1], v[i:i + 1], p, slots[i:i + 1])
            check(out[i:i + 1], qt[i:i + 1], i, p, "step %d of %d" % (step, i))
    bm.close()


FRESH = """
import torch, paged_kv_cache_245_gb300 as pkv
dev = torch.device("cuda:0")
k, v = (torch.randn(80, 8, 16, 128, device=dev).bfloat16() for _ in "kv")
tables = torch.arange(80, dtype=torch.int32, device=dev)[None]
q1, q2 = (torch.randn(n, 32, 128, device=dev).bfloat16() for n in (1, 40))
ctx = torch.tensor([1200], dtype=torch.int32, device=dev)
cu = torch.tensor([0, 40], dtype=torch.int32, device=dev)
work = torch.empty(max(pkv.scored_decode_workspace_size(1, 32, 8, 1200), 16), dtype=torch.uint8, device=dev)
outs = [torch.zeros_like(q1), torch.zeros_like(q2)]
graph = torch.cuda.CUDAGraph()
def calls():
    pkv.paged_decode_attention_scored(q1, k, v, tables, ctx, 1200, 0.1, softcap=30.0, out=outs[0], workspace=work)
    pkv.paged_prefill_attention_scored(q2, cu, k, v, tables, ctx, 40, 0.1, softcap=30.0, out=outs[1])
with torch.cuda.graph(graph):
    calls()
graph.replay()
torch.cuda.synchronize()
got = [x.clone() for x in outs]
calls()
assert all(torch.equal(a, b) and bool((a != 0).any()) for a, b in zip(got, outs))
print("same")
"""


def test_the_first_calls_of_a_process_may_be_captured():
    """What a call asks the device once (shared memory, room for clusters) does not
    break a capture."""
    r = subprocess.run([sys.executable, "-c", FRESH], capture_output=True, text=True, timeout=300,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0 and "same" in r.stdout, r.stdout + r.stderr
