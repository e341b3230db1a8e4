"""Distance biases so steep that a row's weight is one key's: the nearest key's
under a positive slope, the farthest's under a negative one."""
import pytest
import torch

import paged_kv_cache_245_gb300 as pkv
from scored_ref import assert_close
from test_gpu_scored_prefill import Chunks, make

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
STEEP = [2.5, 11.0, 1234.5, 1e4, 1e5, 1e6, 1.1e7, 1e8, 123456789.0, 3e9, 7e10, 1e12, 3e15, 1e20, 1e30, 3e38]
# a batch of many items, of few with long contexts (several CTAs an item), of single tokens
BATCHES = {"chunks": ([0, 500, 30], [400, 33, 200]), "after many": ([3000], [40]),
           "single": ([0, 16, 99, 700], [1, 1, 1, 1]), "long": ([0, 900], [700, 1100])}


@pytest.mark.parametrize("softcap", [0.0, 5.0, 30.0, 50.0, 200.0])
@pytest.mark.parametrize("name", ["plain", "documents", "prefix", "window 100"])
@pytest.mark.parametrize("batch", list(BATCHES))
def test_a_steep_slope_leaves_the_nearest_key(batch, name, softcap):
    s = Chunks(*BATCHES[batch], 16, 2, 16, seed=51)
    ref, kw = make(name, s)
    ref["slopes"] = kw["alibi_slopes"] = torch.tensor(STEEP, device=DEV)
    ref["softcap"] = kw["softcap"] = softcap
    # (the key at distance 0 has no bias, so the bound that the formula's error has stays small)
    assert_close(s.call(**kw), *s.reference(**ref), what=name)


@pytest.mark.parametrize("softcap", [0.0, 5.0, 30.0, 50.0, 200.0])
@pytest.mark.parametrize("name", ["plain", "documents", "window 100"])
@pytest.mark.parametrize("batch", list(BATCHES))
def test_a_steep_negative_slope_leaves_the_farthest_key(batch, name, softcap):
    s = Chunks(*BATCHES[batch], 16, 2, 16, seed=52, by=0.5)
    _, kw = make(name, s)
    # scores differ by less than 32 between neighbours (|q| |k| scale under 0.5 x 128 x 3 x 0.09);
    # from a slope of 1e3 on, the weight of any key but the farthest is under 2^-1000
    kw["alibi_slopes"] = -torch.tensor([1000.0 * x for x in STEEP[:-1]] + [3e38], device=DEV)
    kw["softcap"] = softcap
    first = None if kw["first_key"] is None else kw["first_key"].tolist()
    low = torch.tensor([lo for lo, _ in s.ranges(kw["window"], first)], device=DEV)
    out, at = s.call(**kw), 0
    for i, n in enumerate(s.new):
        v = s.rows(i, s.v)[:, low[at:at + n]].transpose(0, 1).repeat_interleave(8, 1).double()
        # P = 1 and its sum are exact, the output is one value
        assert_close(out[at:at + n], v, v.abs() * 2.0 ** -8)
        at += n


@pytest.mark.parametrize("variant", [pkv.VARIANT_AUTO, pkv.VARIANT_SPLIT, pkv.VARIANT_TC_8X3,
                                     pkv.VARIANT_TC_12X2])
def test_decode_under_steep_slopes(variant):
    s = Chunks([0, 16, 99, 700, 3000], [1, 1, 1, 1, 1], 16, 2, 16, seed=53, by=0.5)
    pkv.set_decode_variant(variant)
    try:
        for softcap in (0.0, 30.0):
            for sign in (1.0, -1.0):
                slopes = sign * torch.tensor([1000.0 * x for x in STEEP[:-1]] + [3e38], device=DEV)
                out = pkv.paged_decode_attention_scored(s.q, s.k, s.v, s.where, s.ctx_t, max(s.ctx),
                                                        128 ** -0.5, softcap=softcap,
                                                        alibi_slopes=slopes)
                for i, c in enumerate(s.ctx):
                    j = c - 1 if sign > 0 else 0
                    v = s.rows(i, s.v)[:, j].repeat_interleave(8, 0).double()
                    assert_close(out[i], v, v.abs() * 2.0 ** -8)
    finally:
        pkv.set_decode_variant(pkv.VARIANT_AUTO)
