"""Decode attention with capped, biased and masked scores against the formula
in 64 bits: head groups, block sizes, both layouts and every kernel, rows that
see nothing, poisoned masked places, freed blocks, graphs, refusals."""
import pytest
import torch

import paged_kv_cache_245_gb300 as pkv
from scored_ref import Sequences, assert_close, attend64, visible

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
D = 128
SCALE = D ** -0.5
AUTO, SPLIT, RUNS, TC = (pkv.VARIANT_AUTO, pkv.VARIANT_SPLIT, pkv.VARIANT_TC_8X3,
                         pkv.VARIANT_TC_12X2)


@pytest.fixture(autouse=True)
def _reset():
    pkv.set_checked(False)
    pkv.set_decode_variant(AUTO)
    yield
    pkv.set_checked(False)
    pkv.set_decode_variant(AUTO)
    pkv.set_split_tiles(0)
    torch.cuda.synchronize()


def slopes_of(hq):
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / hq) for h in range(hq)], device=DEV)


def ranges(s, window=0, first=None):
    return [visible(c - 1, 0 if first is None else int(first[i]), window, 0, c)
            for i, c in enumerate(s.ctx)]


def reference(s, q, window=0, first=None, softcap=0.0, slopes=None, scale=SCALE):
    out, tol = torch.zeros(q.shape, dtype=torch.float64, device=DEV), torch.zeros(
        q.shape, dtype=torch.float64, device=DEV)
    for i, (lo, hi) in enumerate(ranges(s, window, first)):
        if lo <= hi:
            out[i:i + 1], tol[i:i + 1] = attend64(q[i:i + 1], s.rows(i, s.k), s.rows(i, s.v),
                                                  [s.ctx[i] - 1], [(lo, hi)], scale, softcap, slopes)
    return out, tol


def call(s, q, k=None, v=None, scale=SCALE, **kw):
    f = pkv.contig_decode_attention_scored if s.contig else pkv.paged_decode_attention_scored
    return f(q, s.k if k is None else k, s.v if v is None else v, s.where, s.ctx_t,
             max(max(s.ctx), 1), scale, **kw)


def queries(s, hq, by=4.0):
    return (torch.randn(len(s.ctx), hq, D, generator=s.g, device=DEV) * by).bfloat16()


CTX = [1, 2, 15, 16, 17, 0, 33, 100, 257, 700, 129]
SCORES = {
    "plain": dict(),
    "cap": dict(softcap=50.0),
    "small cap": dict(softcap=0.5),
    "huge cap": dict(softcap=1e6),
    "window 1": dict(window=1),
    "window 16": dict(window=16, softcap=30.0),
    "window 100": dict(window=100),
    "window past all": dict(window=2 ** 31 - 1),
    "slopes": dict(slopes=True),
    "documents": dict(first=True),
    "all": dict(softcap=20.0, window=90, slopes=True, first=True),
}


def make(name, s, hq):
    kw = dict(SCORES[name])
    kw["slopes"] = slopes_of(hq) if kw.get("slopes") else None
    if kw.pop("first", False):
        # starts of documents inside, at the end of and past the context; a negative one
        f = [(c * (i % 5)) // 4 + (1 if i % 7 == 6 else 0) for i, c in enumerate(s.ctx)]
        f[1] = -5
        kw["first"] = torch.tensor(f, dtype=torch.int32, device=DEV)
    return kw


def both(kw):
    """(for the reference, for the call)"""
    return kw, dict(softcap=kw.get("softcap", 0.0), window=kw.get("window", 0),
                    alibi_slopes=kw.get("slopes"), first_key=kw.get("first"))


@pytest.mark.parametrize("name", list(SCORES))
@pytest.mark.parametrize("variant", [SPLIT, RUNS, TC])
@pytest.mark.parametrize("contig", [False, True])
def test_scores(name, variant, contig):
    s = Sequences(CTX, 8, 16, contig, seed=3)
    q = queries(s, 32)
    ref, kw = both(make(name, s, 32))
    pkv.set_decode_variant(variant)
    assert_close(call(s, q, **kw), *reference(s, q, **ref), what=name)


@pytest.mark.parametrize("hq,hkv", [(3, 3), (8, 4), (3, 1), (8, 2), (10, 2), (6, 1), (56, 8), (32, 4)])
@pytest.mark.parametrize("bs", [1, 7, 16, 48, 128])
def test_groups_and_block_sizes(hq, hkv, bs):
    s = Sequences([1, 40, 0, 333, 64, 17], hkv, bs, seed=hq + bs)
    q = queries(s, hq)
    ref, kw = both(make("all", s, hq))
    want = reference(s, q, **ref)
    for variant in (SPLIT, RUNS, TC) if bs % 16 == 0 else (AUTO, SPLIT):
        pkv.set_decode_variant(variant)
        assert_close(call(s, q, **kw), *want, what="variant %d" % variant)


@pytest.mark.parametrize("variant", [AUTO, SPLIT, RUNS, TC])
@pytest.mark.parametrize("window", [0, 1000])
def test_long_ragged_batch(variant, window):
    s = Sequences([8000, 1, 5000, 77, 1000, 1001, 3001, 999] * 3, 8, 16, seed=9)
    q = queries(s, 32)
    pkv.set_decode_variant(variant)
    got = call(s, q, softcap=50.0, window=window)
    assert_close(got, *reference(s, q, softcap=50.0, window=window))


@pytest.mark.parametrize("hq,hkv", [(32, 8), (56, 8), (4, 1)])
@pytest.mark.parametrize("variant", [RUNS, TC])
def test_batches_larger_and_smaller_than_the_grid(variant, hq, hkv):
    """Hundreds of short sequences (several pairs a warp), a few long ones
    (several CTAs a pair), more sequences than one launch takes."""
    g = torch.Generator().manual_seed(4)
    pkv.set_decode_variant(variant)
    for ctx in ([int(x) for x in torch.randint(0, 60, (700,), generator=g)], [20000, 3],
                [0] * 40 + [5000] + [0] * 40, [16] * 300):
        s = Sequences(ctx, hkv, 16, seed=len(ctx))
        q = queries(s, hq)
        assert_close(call(s, q, softcap=30.0), *reference(s, q, softcap=30.0))


@pytest.mark.parametrize("chunk", [4, 8])
def test_split_lengths(chunk):
    s = Sequences([2000, 3, 640, 1500], 2, 16, seed=10)
    q = queries(s, 8)
    pkv.set_decode_variant(SPLIT)
    pkv.set_split_tiles(chunk)
    for window in (0, 70, 700):
        assert_close(call(s, q, softcap=30.0, window=window),
                     *reference(s, q, softcap=30.0, window=window))


@pytest.mark.parametrize("by", [0.0, 30.0, 300.0])
@pytest.mark.parametrize("scale", [SCALE, -SCALE])
def test_saturating_scores(by, scale):
    s = Sequences([300, 20, 1], 2, 16, seed=11)
    q = queries(s, 8, by=by)
    for variant in (SPLIT, RUNS, TC):
        pkv.set_decode_variant(variant)
        for cap in (0.0, 5.0, 50.0):
            assert_close(call(s, q, scale=scale, softcap=cap),
                         *reference(s, q, softcap=cap, scale=scale), what="cap %g" % cap)


@pytest.mark.parametrize("variant", [SPLIT, RUNS, TC])
@pytest.mark.parametrize("contig,bs", [(False, 16), (False, 48), (True, 16)])
def test_nothing_in_masked_places_matters(variant, contig, bs):
    s = Sequences(CTX, 2, bs, contig, seed=12)
    q = queries(s, 8)
    pkv.set_decode_variant(variant)
    for name in ("plain", "window 1", "window 16", "window 100", "all", "documents"):
        ref, kw = both(make(name, s, 8))
        k, v = s.poison(ranges(s, ref.get("window", 0), ref.get("first")))
        assert_close(call(s, q, k=k, v=v, **kw), *reference(s, q, **ref), what=name)


@pytest.mark.parametrize("variant", [SPLIT, RUNS, TC])
def test_blocks_before_the_window_are_never_read(variant):
    """Checked mode rejects every table entry the kernel reads that is no
    block: freed entries before the window are not among them."""
    s = Sequences([200, 33, 64, 500], 2, 16, seed=13)
    q = queries(s, 8)
    want = reference(s, q, window=40)
    for i, (lo, _) in enumerate(ranges(s, 40)):
        s.where[i, :lo // 16] = -1
        s.where[i, (s.ctx[i] + 15) // 16:] = 1 << 30
    pkv.set_checked(True)
    pkv.set_decode_variant(variant)
    got = call(s, q, window=40)
    assert pkv.get_device_error() == "none"
    assert_close(got, *want)
    s.where[3, 31] = -1  # a visible one is reported
    call(s, q, window=40)
    assert pkv.get_device_error() == "block_id"


def test_a_negative_slope_and_a_steep_one():
    s = Sequences([400, 3, 90], 2, 16, seed=14)
    q = queries(s, 8)
    slopes = torch.tensor([-0.3, 0.0, 1e6, 40.0, 1e30, 2.0 ** -20, 3.0, -0.01], device=DEV)
    for variant in (SPLIT, RUNS, TC):
        pkv.set_decode_variant(variant)
        assert_close(call(s, q, alibi_slopes=slopes), *reference(s, q, slopes=slopes))


def test_null_score_is_the_plain_call():
    s = Sequences(CTX, 8, 16, seed=15)
    q = queries(s, 32)
    for variant in (SPLIT, RUNS, TC):
        pkv.set_decode_variant(variant)
        plain = pkv.paged_decode_attention(q, s.k, s.v, s.where, s.ctx_t, max(s.ctx), SCALE)
        assert_close(call(s, q), plain.double(), 2.0 ** -7 * plain.double().abs() + 2.0 ** -7)


def test_cache_beyond_32_bit_offsets():
    """Rows past 2^31 elements into the cache, both layouts."""
    hkv, bs = 8, 128
    nb = 2 ** 31 // (hkv * bs * D) + 8
    s = Sequences([300, 150], hkv, bs, seed=16)
    k, v = (torch.empty(nb, hkv, bs, D, dtype=torch.bfloat16, device=DEV) for _ in "kv")
    k[nb - s.nb:], v[nb - s.nb:] = s.k, s.v
    q = queries(s, 32)
    want = reference(s, q, softcap=30.0, window=200)
    for variant in (SPLIT, RUNS, TC):
        pkv.set_decode_variant(variant)
        got = pkv.paged_decode_attention_scored(q, k, v, s.where + (nb - s.nb), s.ctx_t, 300, SCALE,
                                                softcap=30.0, window=200)
        assert_close(got, *want)
    # a request row past 2^31 elements
    del k, v
    S = 2 ** 21
    c = Sequences([300], hkv, 16, True, seed=17)
    big = torch.empty(2, hkv, S, D, dtype=torch.bfloat16, device=DEV)
    bigv = torch.empty_like(big)
    big[1, :, :300], bigv[1, :, :300] = c.k[int(c.where[0]), :, :300], c.v[int(c.where[0]), :, :300]
    q = queries(c, 32)
    got = pkv.contig_decode_attention_scored(
        q, big, bigv, torch.ones(1, dtype=torch.int32, device=DEV), c.ctx_t, 300, SCALE, window=77)
    assert_close(got, *reference(c, q, window=77))


@pytest.mark.parametrize("variant", [RUNS, TC])
def test_graph_streams_and_shared_workspace(variant):
    pkv.set_decode_variant(variant)
    s = Sequences([900, 31, 400, 65] * 8, 8, 16, seed=18)
    q = queries(s, 32)
    size = pkv.scored_decode_workspace_size(len(s.ctx), 32, 8, 900, 300)
    ws = torch.empty(max(size, 16), dtype=torch.uint8, device=DEV)
    a = call(s, q, softcap=50.0, window=300)
    b = call(s, q, softcap=50.0)
    outs = [torch.empty_like(q) for _ in "ab"]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = []
    with torch.cuda.stream(side):
        call(s, q, softcap=50.0, window=300, workspace=ws)
        for out, window in zip(outs, (300, 0)):  # two graphs, one workspace
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                call(s, q, softcap=50.0, window=window, out=out, workspace=ws)
            graphs.append(g)
    torch.cuda.synchronize()
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], a) and torch.equal(outs[1], b)


def test_binding_refusals():
    s = Sequences([40, 3], 2, 16, seed=19)
    q = queries(s, 8)
    for kw, error in ((dict(softcap=-1.0), pkv.PkvError), (dict(softcap=float("nan")), pkv.PkvError),
                      (dict(softcap=1e7), pkv.PkvError), (dict(window=-1), pkv.PkvError),
                      (dict(alibi_slopes=torch.ones(7, device=DEV)), ValueError),
                      (dict(alibi_slopes=torch.ones(8, device=DEV).half()), TypeError),
                      (dict(alibi_slopes=torch.ones(8)), TypeError),
                      (dict(first_key=torch.zeros(3, dtype=torch.int32, device=DEV)), ValueError),
                      (dict(first_key=torch.zeros(2, dtype=torch.int64, device=DEV)), TypeError),
                      (dict(out=torch.empty_like(q)[:1]), ValueError),
                      (dict(workspace=torch.empty(15, dtype=torch.uint8, device=DEV)), pkv.PkvError)):
        with pytest.raises(error):
            pkv.set_decode_variant(TC)
            call(s, q, **kw)
    with pytest.raises(ValueError):
        pkv.paged_decode_attention_scored(q[:1].contiguous(), s.k, s.v, s.where, s.ctx_t, 40, SCALE)
    empty = torch.empty(0, 8, D, dtype=torch.bfloat16, device=DEV)
    none = torch.empty(0, dtype=torch.int32, device=DEV)
    assert pkv.paged_decode_attention_scored(empty, s.k, s.v, s.where[:0], none, 40, SCALE,
                                             softcap=5.0).shape == (0, 8, D)


def test_runs_of_more_than_a_million_units():
    """So many tiles that the schedule leaves 32-bit arithmetic (the caches' blocks
    are shared by all sequences)."""
    g = torch.Generator(device=DEV).manual_seed(3)
    hkv, bs, ctx, batch = 8, 16, 60000, 40
    k, v = (torch.randn(32, hkv, bs, D, generator=g, device=DEV).bfloat16() for _ in "kv")
    tables = torch.randint(0, 32, (1, ctx // bs), generator=g, device=DEV, dtype=torch.int32)
    q = torch.randn(1, 8, D, generator=g, device=DEV).bfloat16()
    ctx_t = torch.full((batch,), ctx, dtype=torch.int32, device=DEV)
    pkv.set_decode_variant(RUNS)
    out = pkv.paged_decode_attention_scored(q.expand(batch, -1, -1).contiguous(), k, v,
                                            tables.expand(batch, -1).contiguous(), ctx_t, ctx,
                                            SCALE, softcap=30.0)
    rows = [x[tables[0].long()].transpose(0, 1).reshape(hkv, ctx, D) for x in (k, v)]
    want, tol = attend64(q, *rows, [ctx - 1], [(0, ctx - 1)], SCALE, 30.0)
    assert_close(out, want.expand(batch, -1, -1), tol.expand(batch, -1, -1))


@pytest.mark.parametrize("hq,hkv", [(32, 8), (7, 1), (4, 4), (16, 2)])
@pytest.mark.parametrize("contig", [False, True])
def test_few_sequences_whose_splits_are_a_cluster(hq, hkv, contig):
    """Small batches around the sizes where clusters of 2 to 16 CTAs join the
    splits, with sequences that leave splits empty, and a window."""
    for ctx in ([1000], [65], [4000], [700, 0], [1000, 3, 500], [512] * 8, [100] * 16, [900] * 20):
        s = Sequences(ctx, hkv, 16, contig, seed=len(ctx) + ctx[0])
        q = queries(s, hq)
        for kw in (dict(softcap=30.0), dict(window=300, slopes=slopes_of(hq))):
            ref = reference(s, q, **kw)
            kw["alibi_slopes"] = kw.pop("slopes", None)
            assert_close(call(s, q, **kw), *ref)


def test_a_cluster_replays_beside_an_eager_call():
    s = Sequences([1000, 20], 8, 16, seed=8)
    q = queries(s, 32)
    want = reference(s, q, softcap=50.0)
    out, side = torch.empty_like(q), torch.cuda.Stream()
    other = torch.empty_like(q)
    call(s, q, softcap=50.0, out=out)
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call(s, q, softcap=50.0, out=out)
    for _ in range(5):
        out.fill_(7.0)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            call(s, q, softcap=50.0, out=other)
        graph.replay()
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(out, other)
    assert_close(out, *want)
