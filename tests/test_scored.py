"""Host-side checks of the scored attention calls.  No GPU."""
import ctypes

import pytest

import paged_kv_cache_245_gb300 as pkv
from paged_kv_cache_245_gb300 import binding
from paged_kv_cache_245_gb300.build import build

FAKE = ctypes.c_void_p(0x10000)        # never dereferenced: validation fails first
MISALIGNED = ctypes.c_void_p(0x10008)


@pytest.fixture(scope="module")
def L():
    build()
    return pkv.lib()


def _h(hq=8, hkv=2, d=128):
    return binding.Heads(hq, hkv, d)


def score(**kw):
    return binding.Score(kw.get("softcap", 0.0), kw.get("window", 0), kw.get("slopes"),
                         kw.get("first"), kw.get("prefix"))


def calls(L):
    def decode(sc, h=_h(), q=FAKE, ctx=FAKE, B=2, mc=64, bs=16, scale=0.1, mb=4):
        return L.pkv_paged_decode_attention_scored(q, FAKE, FAKE, FAKE, mb, 10, ctx, B, mc, bs,
                                                   scale, sc, h, FAKE, None, 0, None)

    def contig(sc, h=_h(), q=FAKE, ctx=FAKE, B=2, mc=64, bs=64, scale=0.1, mb=4):
        return L.pkv_contig_decode_attention_scored(q, FAKE, FAKE, FAKE, mb, ctx, B, mc, bs,
                                                    scale, sc, h, FAKE, None, 0, None)

    def prefill(sc, h=_h(), q=FAKE, ctx=FAKE, B=2, mc=64, bs=16, scale=0.1, mb=4):
        return L.pkv_paged_prefill_attention_scored(q, FAKE, 8, FAKE, FAKE, FAKE, mb, 10, ctx, B,
                                                    mc, bs, scale, sc, h, FAKE, None)

    def contig_prefill(sc, h=_h(), q=FAKE, ctx=FAKE, B=2, mc=64, bs=64, scale=0.1, mb=4):
        return L.pkv_contig_prefill_attention_scored(q, FAKE, 8, FAKE, FAKE, FAKE, mb, ctx, B, mc,
                                                     bs, scale, sc, h, FAKE, None)

    return decode, contig, prefill, contig_prefill


@pytest.mark.parametrize("which", range(4))
def test_score_refusals(L, which):
    f = calls(L)[which]
    for bad in (dict(softcap=-0.5), dict(softcap=float("nan")), dict(softcap=float("inf")),
                dict(window=-1), dict(slopes=0x10002), dict(first=0x10001), dict(prefix=0x10003)):
        assert f(ctypes.byref(score(**bad))) == 1, bad
        assert L.pkv_last_error() != b""
    for bad in (dict(softcap=1e-7), dict(softcap=2e6)):
        assert f(ctypes.byref(score(**bad))) == 2 and b"softcap" in L.pkv_last_error()


@pytest.mark.parametrize("which", range(4))
@pytest.mark.parametrize("given", [True, False])
def test_the_plain_calls_refusals_hold(L, which, given):
    f, sc = calls(L)[which], ctypes.byref(score(softcap=50.0)) if given else None
    assert f(sc, h=_h(d=64)) == 2
    assert f(sc, h=_h(32, 2)) == 2
    assert f(sc, h=_h(9, 2)) == 1
    assert f(sc, q=None) == 1
    assert f(sc, q=MISALIGNED) == 1 and b"aligned" in L.pkv_last_error()
    assert f(sc, ctx=None) == 1
    assert f(sc, ctx=ctypes.c_void_p(0x10002)) == 1
    assert f(sc, scale=float("inf")) == 1
    assert f(sc, mb=0) == 1
    assert f(sc, B=-1) == 1
    assert f(sc, B=70000) == 2
    assert f(sc, bs=0) in (1, 2)
    assert f(sc, B=0) == 0


def test_contexts_beyond_the_layout(L):
    decode, contig, prefill, contig_prefill = calls(L)
    sc = ctypes.byref(score(window=10))
    assert decode(sc, mc=65) == 1 and b"max_blocks" in L.pkv_last_error()
    assert contig(sc, mc=65) == 1 and b"S" in L.pkv_last_error()
    assert prefill(sc, bs=24) == 2 and contig_prefill(sc, bs=1000) == 2


def test_workspace_size_of_bad_arguments(L):
    assert pkv.scored_decode_workspace_size(4, 9, 2, 100) == 0
    assert pkv.scored_decode_workspace_size(-4, 8, 2, 100) == 0
    assert pkv.scored_decode_workspace_size(4, 8, 2, 100, window=-1) == 0
