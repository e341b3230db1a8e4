"""NaN and infinities in places that a token sees: scored attention gives what
the formula gives, whichever kernel runs and wherever a schedule cuts the keys."""
import pytest
import torch

import paged_kv_cache_245_gb300 as pkv
from scored_ref import Sequences, assert_close, attend64

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
