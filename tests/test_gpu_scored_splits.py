"""Scored decode by splits whose partials a second kernel combines: a split length
that is set by hand leaves no cluster to join them (pkv_set_split_tiles)."""
import pytest
import torch

import paged_kv_cache_245_gb300 as pkv
from scored_ref import Sequences, assert_close
from test_gpu_scored_decode import CTX, SCALE, SCORES, both, call, make, queries, ranges, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, params=[4, 8])
def _splits(request):
    pkv.set_decode_variant(pkv.VARIANT_SPLIT)
    pkv.set_split_tiles(request.param)
    yield
    pkv.set_split_tiles(0)
    pkv.set_decode_variant(pkv.VARIANT_AUTO)
    torch.cuda.synchronize()


@pytest.mark.parametrize("name", list(SCORES))
@pytest.mark.parametrize("contig", [False, True])
def test_scores(name, contig):
    s = Sequences(CTX, 8, 16, contig, seed=3)
    q = queries(s, 32)
    ref, kw = both(make(name, s, 32))
    assert_close(call(s, q, **kw), *reference(s, q, **ref), what=name)


@pytest.mark.parametrize("hq,hkv", [(3, 3), (8, 4), (3, 1), (8, 2), (10, 2), (6, 1), (56, 8), (32, 4)])
@pytest.mark.parametrize("bs", [1, 7, 16, 48, 128])
def test_groups_and_block_sizes(hq, hkv, bs):
    s = Sequences([1, 40, 0, 333, 64, 17, 1000], hkv, bs, seed=hq + bs)
    q = queries(s, hq)
    ref, kw = both(make("all", s, hq))
    assert_close(call(s, q, **kw), *reference(s, q, **ref))


@pytest.mark.parametrize("contig,bs", [(False, 16), (False, 48), (True, 16)])
def test_nothing_in_masked_places_matters(contig, bs):
    s = Sequences(CTX, 2, bs, contig, seed=12)
    q = queries(s, 8)
    for name in ("plain", "window 1", "window 16", "window 100", "all", "documents"):
        ref, kw = both(make(name, s, 8))
        k, v = s.poison(ranges(s, ref.get("window", 0), ref.get("first")))
        assert_close(call(s, q, k=k, v=v, **kw), *reference(s, q, **ref), what=name)


@pytest.mark.parametrize("by", [0.0, 30.0, 300.0])
@pytest.mark.parametrize("scale", [SCALE, -SCALE])
def test_saturating_scores(by, scale):
    s = Sequences([300, 20, 1, 700], 2, 16, seed=11)
    q = queries(s, 8, by=by)
    for cap in (0.0, 5.0, 50.0):
        assert_close(call(s, q, scale=scale, softcap=cap),
                     *reference(s, q, softcap=cap, scale=scale), what="cap %g" % cap)
