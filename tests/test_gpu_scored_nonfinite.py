"""NaN and infinities in places that a token sees: scored attention gives what
the formula gives, whichever kernel runs and wherever a schedule cuts the keys."""
import pytest
import torch

import paged_kv_cache_245_gb300 as pkv
from scored_ref import Sequences, assert_close, attend64
from test_gpu_scored_prefill import Chunks, make, slopes_of

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
D = 128
SCALE = D ** -0.5
# (decode variant, tiles a split): what the name says runs where the batch allows it
KERNELS = {"auto": (pkv.VARIANT_AUTO, 0), "cluster": (pkv.VARIANT_SPLIT, 0),
           "splits of 4 and combine": (pkv.VARIANT_SPLIT, 4),
           "splits of 8 and combine": (pkv.VARIANT_SPLIT, 8),
           "runs": (pkv.VARIANT_TC_8X3, 0), "pairs": (pkv.VARIANT_TC_12X2, 0)}


@pytest.fixture(autouse=True)
def _reset():
    yield
    pkv.set_decode_variant(pkv.VARIANT_AUTO)
    pkv.set_split_tiles(0)
    torch.cuda.synchronize()


def choose(kernel):
    variant, tiles = KERNELS[kernel]
    pkv.set_decode_variant(variant)
    pkv.set_split_tiles(tiles)


def decode(s, q, **kw):
    f = pkv.contig_decode_attention_scored if s.contig else pkv.paged_decode_attention_scored
    return f(q, s.k, s.v, s.where, s.ctx_t, max(s.ctx), SCALE, **kw)


def row(s, i, j):
    """Where position j of sequence i is: (block or request, offset)."""
    return (int(s.where[i]), j) if s.contig else (int(s.where[i, j // s.bs]), j % s.bs)


# batches whose pairs are one tile, several splits, and cut by many warps and CTAs
BATCHES = {"short": [1, 15, 33, 0, 100], "one of 1000": [1000], "two": [5000, 700],
           "ragged": [3000, 1, 40, 900, 129, 2000] * 4}


@pytest.mark.parametrize("kernel", list(KERNELS))
@pytest.mark.parametrize("batch", list(BATCHES))
@pytest.mark.parametrize("hq,contig", [(8, False), (14, True)])
def test_a_nan_key_makes_its_rows_nan(kernel, batch, hq, contig):
    ctx = BATCHES[batch]
    s = Sequences(ctx, 2, 16, contig, seed=len(ctx))
    q = torch.randn(len(ctx), hq, D, generator=s.g, device=DEV).bfloat16()
    choose(kernel)
    G = hq // 2
    for kw in (dict(softcap=30.0), dict(window=600)):
        want = decode(s, q, **kw)
        assert bool(torch.isfinite(want).all())
        longest = ctx.index(max(ctx))
        last = ctx[longest] - 1
        first = max(0, last - 599) if "window" in kw else 0
        for i, j in {(longest, first), (longest, (first + last) // 2), (longest, last - 17 if last > 17 else last),
                     (longest, last), (0, ctx[0] - 1)}:
            block, off = row(s, i, j)
            kept = s.k[block, 1, off].clone()
            s.k[block, 1, off, 5] = float("nan")
            got = decode(s, q, **kw)
            s.k[block, 1, off] = kept
            assert bool(torch.isnan(got[i, G:]).all()), "key %d of sequence %d" % (j, i)
            got[i, G:] = want[i, G:]
            assert torch.equal(got, want)


@pytest.mark.parametrize("kernel", list(KERNELS))
@pytest.mark.parametrize("batch", list(BATCHES))
def test_a_nan_value_makes_its_column_nan(kernel, batch):
    ctx = BATCHES[batch]
    s = Sequences(ctx, 2, 16, seed=len(ctx))
    q = torch.randn(len(ctx), 8, D, generator=s.g, device=DEV).bfloat16()
    choose(kernel)
    want = decode(s, q, softcap=30.0)
    i = ctx.index(max(ctx))
    for j in (0, ctx[i] // 2, ctx[i] - 1):
        for bad in (float("nan"), float("inf"), -float("inf")):
            block, off = row(s, i, j)
            kept = s.v[block, 0, off].clone()
            s.v[block, 0, off, 77] = bad
            got = decode(s, q, softcap=30.0)
            s.v[block, 0, off] = kept
            column = got[i, :4, 77].float()
            assert bool(torch.isnan(column).all() if bad != bad else (column == bad).all())
            got[i, :4, 77] = want[i, :4, 77]
            assert torch.equal(got, want)


@pytest.mark.parametrize("kernel", list(KERNELS))
@pytest.mark.parametrize("batch", list(BATCHES))
def test_a_nan_query_makes_its_row_nan(kernel, batch):
    ctx = BATCHES[batch]
    s = Sequences(ctx, 2, 16, seed=len(ctx))
    q = torch.randn(len(ctx), 8, D, generator=s.g, device=DEV).bfloat16()
    choose(kernel)
    for kw in (dict(softcap=30.0), dict(window=600),
               dict(alibi_slopes=torch.linspace(0.0, 1.0, 8, device=DEV))):
        want = decode(s, q, **kw)
        bad = q.clone()
        i = ctx.index(max(ctx))
        bad[i, 6, 100] = float("nan")
        got = decode(s, bad, **kw)
        assert bool(torch.isnan(got[i, 6]).all())
        got[i, 6] = want[i, 6]
        assert torch.equal(got, want)


def infinite_keys(s, q, i, keys, sign):
    """Key rows whose score is sign * infinity for every head of KV head 1."""
    q[..., 5] = 1.0
    for j in keys:
        block, off = row(s, i, j)
        s.k[block, 1, off, 5] = sign * float("inf")


def without(s, q, i, keys, kvh, softcap=0.0):
    """(out, tol) of sequence i's newest token and KV head kvh, `keys` left out."""
    G = q.shape[1] // s.hkv
    keep = torch.tensor([j for j in range(s.ctx[i]) if j not in set(keys)], device=DEV)
    k, v = (s.rows(i, x)[kvh:kvh + 1, keep] for x in (s.k, s.v))
    return attend64(q[i:i + 1, kvh * G:(kvh + 1) * G], k, v, [s.ctx[i] - 1], [(0, len(keep) - 1)],
                    SCALE, softcap)


@pytest.mark.parametrize("kernel", list(KERNELS))
@pytest.mark.parametrize("batch", ["short", "one of 1000", "two", "ragged"])
def test_a_score_of_minus_infinity_has_no_weight(kernel, batch):
    """One key, whole tiles (a warp's first among them), and the last tile's only key."""
    ctx = BATCHES[batch]
    i = ctx.index(max(ctx))
    c = ctx[i]
    for keys in ([0], range(0, 48), range(c - c % 16 or c - 16, c), range(16, c - 1)):
        s = Sequences(ctx, 2, 16, seed=len(ctx))
        q = torch.randn(len(ctx), 8, D, generator=s.g, device=DEV).bfloat16()
        infinite_keys(s, q, i, keys, -1)
        choose(kernel)
        got = decode(s, q)
        want, tol = without(s, q, i, keys, 1)
        assert_close(got[i:i + 1, 4:], want, tol, "keys %s" % keys)
        want, tol = without(s, q, i, (), 0)
        assert_close(got[i:i + 1, :4], want, tol)


@pytest.mark.parametrize("kernel", list(KERNELS))
def test_a_score_of_infinity_is_the_cap_or_nan(kernel):
    for ctx in ([700], [40, 3], [3000] * 12):
        for sign in (1, -1):
            s = Sequences(ctx, 2, 16, seed=len(ctx))
            q = torch.randn(len(ctx), 8, D, generator=s.g, device=DEV).bfloat16()
            infinite_keys(s, q, 0, (20, 33), sign)
            choose(kernel)
            if sign > 0:  # inf - inf
                assert bool(torch.isnan(decode(s, q)[0, 4:]).all())
            got = decode(s, q, softcap=5.0)
            s.k.clamp_(-1e4, 1e4)  # far beyond the cap
            assert_close(got[:1, 4:], *without(s, q, 0, (), 1, 5.0))


# ------------------------------------------------------------------ prefill

PREFILL = {"chunks": ([0, 300, 40], [500, 70, 260]), "after many": ([3000, 200], [40, 3]),
           "single": ([0, 130, 700], [1, 1, 1])}
MODES = {"masked": dict(), "capped": dict(softcap=30.0), "biased": dict(slopes=True),
         "capped and biased": dict(softcap=30.0, slopes=True), "any": dict(softcap=200.0)}
BAD = {"nan": float("nan"), "inf": float("inf"), "-inf": -float("inf")}


def expected(s, ref, bad):
    """(out, tol, kind) with values `bad` [(sequence, KV head, position, column, kind)]
    in V: kind is 0 where an output is finite (out holds it), 1 NaN, 2 inf, 3 -inf."""
    kept = s.v.clone()
    for i, h, j, column, _ in bad:
        block, off = row(s, i, j)
        s.v[block, h, off, column] = 0.0
    out, tol = s.reference(**ref)
    s.v = kept
    rng = s.ranges(ref.get("window", 0), None if "first" not in ref else ref["first"].tolist(),
                   ref.get("prefix"))
    kinds = torch.zeros(s.T, s.hq, D, dtype=torch.int64, device=DEV)
    G = s.hq // s.hkv
    met = {}
    for i, h, j, column, name in bad:
        for t, (seq, _) in enumerate(s.positions()):
            if seq == i and rng[t][0] <= j <= rng[t][1]:
                met.setdefault((t, h, column), set()).add(name)
    for (t, h, column), names in met.items():
        one = {"nan": 1, "inf": 2, "-inf": 3}[next(iter(names))] if len(names) == 1 else 1
        kinds[t, h * G:(h + 1) * G, column] = one
    return out, tol, kinds


@pytest.mark.parametrize("mode", list(MODES))
@pytest.mark.parametrize("masks", ["plain", "documents", "prefix", "window 100"])
@pytest.mark.parametrize("batch", list(PREFILL))
@pytest.mark.parametrize("hq,contig", [(8, False), (14, True)])
def test_values_that_are_not_finite_reach_the_rows_that_see_them(batch, masks, mode, hq, contig):
    """NaN and infinities scattered over V, several kinds in a column, seen by some
    rows of a work item and masked for others."""
    s = Chunks(*PREFILL[batch], hq, 2, 16, contig, seed=61, by=1.0)
    ref, kw = make(masks, s)
    m = MODES[mode]
    if m.get("slopes"):  # gentle: every weight stays above 2^-126
        ref["slopes"] = kw["alibi_slopes"] = slopes_of(hq) / 64
    ref["softcap"] = kw["softcap"] = m.get("softcap", 0.0)
    g = torch.Generator().manual_seed(62)
    bad = []
    for i, c in enumerate(s.ctx):
        for n in range(24):
            j, column, h = (int(torch.randint(0, x, (1,), generator=g)) for x in (c, D, 2))
            column = column if n % 2 else 64  # many in one column
            bad.append((i, h, j, column, list(BAD)[int(torch.randint(0, 3, (1,), generator=g))]))
    bad = list({b[:4]: b for b in bad}.values())
    for i, h, j, column, name in bad:
        block, off = row(s, i, j)
        s.v[block, h, off, column] = BAD[name]
    out, tol, kinds = expected(s, ref, bad)
    got = s.call(**kw).float()
    assert bool(torch.isnan(got[kinds == 1]).all())
    assert bool((got[kinds == 2] == float("inf")).all())
    assert bool((got[kinds == 3] == -float("inf")).all())
    finite = kinds == 0
    assert_close(got[finite], out[finite], tol[finite])


@pytest.mark.parametrize("mode", list(MODES))
@pytest.mark.parametrize("batch", list(PREFILL))
def test_a_nan_key_or_query_in_prefill(batch, mode):
    s = Chunks(*PREFILL[batch], 8, 2, 16, seed=63, by=1.0)
    m = MODES[mode]
    kw = dict(softcap=m.get("softcap", 0.0), window=250,
              alibi_slopes=slopes_of(8) if m.get("slopes") else None)
    # Rows beside it are held to the formula's bound, not to the same bits: where one row
    # of a warp needs the exponentials, its other rows take them in place of the polynomial.
    want, tol = s.reference(softcap=kw["softcap"], window=250, slopes=kw["alibi_slopes"])
    i = 1
    for j in (s.ctx[i] - 1, max(0, s.ctx[i] - 100)):
        block, off = row(s, i, j)
        kept = s.k[block, 1, off].clone()
        s.k[block, 1, off, 3] = float("nan")
        got = s.call(**kw)
        s.k[block, 1, off] = kept
        sees = torch.tensor([seq == i and lo <= j <= hi for (seq, _), (lo, hi) in
                             zip(s.positions(), s.ranges(250))], device=DEV)
        assert bool(torch.isnan(got[sees][:, 4:]).all())
        rest = torch.ones_like(got, dtype=torch.bool)
        rest[sees, 4:] = False
        assert_close(got[rest], want[rest], tol[rest])
    q = s.q.clone()
    q[0, 5, 9] = float("nan")
    got = s.call(q=q, **kw)
    assert bool(torch.isnan(got[0, 5]).all())
    rest = torch.ones_like(got, dtype=torch.bool)
    rest[0, 5] = False
    assert_close(got[rest], want[rest], tol[rest])


def timed(run):
    best = float("inf")
    for _ in range(4):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in "ab")
        a.record()
        run()
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b))
    return best


@pytest.mark.parametrize("mode", ["masked", "capped", "biased"])
def test_a_value_that_every_later_token_sees_costs_little(mode):
    """One NaN among a prompt's first values: every row after it is NaN in a column,
    which is found by a look through V, not by computing the rows again."""
    s = Chunks([0] * 4, [2048] * 4, 32, 8, 16, seed=64)
    m = MODES[mode]
    kw = dict(softcap=m.get("softcap", 0.0), alibi_slopes=slopes_of(32) if m.get("slopes") else None)
    out = torch.empty_like(s.q)
    s.call(out=out, **kw)
    clean, time = out.clone(), timed(lambda: s.call(out=out, **kw))
    for bad, at in ((float("nan"), 5), (float("inf"), 5)):
        block, off = row(s, 0, at)
        s.v[block, :, off, 40] = bad
        slow = timed(lambda: s.call(out=out, **kw))
        s.v[block, :, off, 40] = 0.5
        # a look through 2048 rows of V an item and warp at worst: about ten times; computed
        # again, the rows took over a hundred times as long
        assert slow < 20 * time, "%.3f ms, %.3f ms without" % (slow, time)
        column = out[at:2048, :, 40]
        assert not bool(torch.isfinite(column).any())
        other = torch.arange(D, device=DEV) != 40
        close = (out[:, :, other].float() - clean[:, :, other].float()).abs()
        assert bool((close <= 2.0 ** -6 * clean[:, :, other].float().abs() + 2.0 ** -7).all())


def test_rows_computed_again_over_long_contexts():
    """Half of each chunk's rows beside a masked NaN, over fifty thousand positions, in
    more work items than the device has SMs: every one is written."""
    hkv, hq, bs, ctx, new, batch = 1, 4, 16, 50000, 64, 160
    s = Chunks([ctx - new], [new], hq, hkv, bs, seed=65, by=1.0)
    first = torch.zeros(new, dtype=torch.int32, device=DEV)
    want, tol = s.reference(softcap=30.0)
    at = ctx - new // 2
    block, off = row(s, 0, at)
    s.v[block, 0, off, 9] = float("nan")
    cu = torch.arange(batch + 1, dtype=torch.int32, device=DEV) * new
    pkv.set_checked(True)
    out = pkv.paged_prefill_attention_scored(
        s.q.repeat(batch, 1, 1), cu, s.k, s.v, s.where.repeat(batch, 1), s.ctx_t.repeat(batch), new,
        SCALE, softcap=30.0, first_key=first.repeat(batch))
    error = pkv.get_device_error()
    pkv.set_checked(False)
    assert error == "none"
    out = out.view(batch, new, hq, D)
    assert bool(torch.isnan(out[:, new // 2:, :, 9]).all())
    out[:, new // 2:, :, 9] = 0
    want[new // 2:, :, 9] = 0
    assert torch.equal(out, out[:1].expand_as(out))
    assert_close(out[0], want, tol)
