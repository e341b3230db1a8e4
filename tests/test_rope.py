"""Rotary plans (pkv_rope_init, pkv_rope_init_frequencies) against their
formulas, and the host-side checks of pkv_rope_append.  No GPU."""
import ctypes
import math

import numpy as np
import pytest

import paged_kv_cache_245_gb300 as pkv
from paged_kv_cache_245_gb300 import binding
from paged_kv_cache_245_gb300.build import build


@pytest.fixture(scope="module")
def L():
    build()
    return pkv.lib()


def turns(plan):
    """Turns per position of each pair, from the plan's 64-bit fractions."""
    return np.array([int(x) for x in plan.c.turn[:plan.c.rotary_dim // 2]], dtype=object) / 2 ** 64


def close(plan, radians):
    # two roundings of 2^-53: 1 / (2 pi) and the product; the reference's own: two more
    want = np.asarray(radians, np.float64) / (2 * math.pi)
    got = turns(plan).astype(np.float64)
    assert np.all(np.abs(got - want) <= 8 * 2.0 ** -53 * want + 2.0 ** -64), (got, want)


def base(rd, theta):
    return np.array([theta ** (-2.0 * i / rd) for i in range(rd // 2)])


@pytest.mark.parametrize("rd", [2, 6, 50, 64, 128])
def test_plain_frequencies(L, rd):
    p = pkv.RopePlan(rd, theta=10000.0)
    close(p, base(rd, 10000.0))
    assert p.c.gain == 1.0 and p.c.rotary_dim == rd and p.c.interleaved == 0
    assert pkv.RopePlan(rd, interleaved=True).c.interleaved == 1
    assert all(x == 0 for x in p.c.turn[rd // 2:])


def test_linear_and_base_scaling(L):
    close(pkv.RopePlan(64, theta=5e5, scaling={"kind": "linear", "factor": 8}), base(64, 5e5) / 8)
    theta = 1e4 * 4.0 ** (128 / 126)
    close(pkv.RopePlan(128, theta=1e4, scaling={"kind": "base", "factor": 4}), base(128, theta))
    # the defining property: the slowest pair ends up divided by the factor
    p = turns(pkv.RopePlan(128, theta=1e4, scaling={"kind": "base", "factor": 4}))
    q = turns(pkv.RopePlan(128, theta=1e4))
    assert abs(float(q[63] / p[63]) - 4.0) < 1e-12 and p[0] == q[0]


def test_smooth_scaling(L):
    s = {"kind": "smooth", "factor": 8, "original": 8192, "low": 1, "high": 4}
    got = turns(pkv.RopePlan(128, theta=5e5, scaling=s)).astype(np.float64)
    w = base(128, 5e5)
    n = 8192 * w / (2 * math.pi)
    keep = np.clip((n - 1) / 3, 0, 1)
    close(pkv.RopePlan(128, theta=5e5, scaling=s), w / 8 * (1 - keep) + w * keep)
    assert (keep == 0).any() and (keep == 1).any() and ((keep > 0) & (keep < 1)).any()
    assert np.allclose(got[n >= 4] * 2 * math.pi, w[n >= 4], rtol=1e-14)
    assert np.allclose(got[n <= 1] * 2 * math.pi, w[n <= 1] / 8, rtol=1e-14)


def test_scaling_by_parts(L):
    s = {"kind": "parts", "factor": 16, "original": 4096}
    p = pkv.RopePlan(128, theta=1e4, scaling=s)
    w = base(128, 1e4)
    at = lambda t: 128 * math.log(4096 / (t * 2 * math.pi)) / (2 * math.log(1e4))  # noqa: E731
    low, high = math.floor(at(32)), math.ceil(at(1))
    slow = np.clip((np.arange(64) - low) / (high - low), 0, 1)
    close(p, w / 16 * slow + w * (1 - slow))
    assert p.c.gain == np.float32(0.1 * math.log(16) + 1)
    assert pkv.RopePlan(128, scaling=dict(s, gain=2.5)).c.gain == 2.5
    # every pair faster than beta_fast turns keeps its frequency, every slower than beta_slow does not
    n = 4096 * w / (2 * math.pi)
    got = turns(p).astype(np.float64) * 2 * math.pi
    assert np.allclose(got[n >= 40], w[n >= 40], rtol=1e-14)
    assert np.allclose(got[n <= 0.9], w[n <= 0.9] / 16, rtol=1e-14)


def test_frequencies_of_the_caller(L):
    w = [0.5, 2 * math.pi + 0.25, 0.0, -1e-3]
    p = pkv.RopePlan(8, inv_freq=w, gain=1.25)
    got = turns(p).astype(np.float64)
    # whole turns drop out; a negative frequency is its fraction from below
    want = np.array([0.5, 0.25, 0.0, 2 * math.pi - 1e-3]) / (2 * math.pi)
    assert np.allclose(got, want, rtol=0, atol=2.0 ** -50) and p.c.gain == 1.25
    # so small a negative one that its fraction rounds to a whole turn: none
    assert pkv.RopePlan(2, inv_freq=[-1e-30]).c.turn[0] == 0


@pytest.mark.parametrize("kw", [
    dict(rotary_dim=0), dict(rotary_dim=7), dict(rotary_dim=130), dict(theta=0.5),
    dict(theta=float("nan")), dict(scaling={"kind": "linear", "factor": 0.5}),
    dict(scaling={"kind": "linear", "factor": float("inf")}),
    dict(rotary_dim=2, scaling={"kind": "base", "factor": 2}),
    dict(scaling={"kind": "parts", "factor": 2, "original": 0}),
    dict(scaling={"kind": "smooth", "factor": 2, "original": 100, "low": 4, "high": 4}),
    dict(scaling={"kind": "parts", "factor": 2, "original": 100, "gain": -1}),
    dict(rotary_dim=4, inv_freq=[1.0, float("nan")]), dict(rotary_dim=4, inv_freq=[1.0, 1e7]),
    dict(rotary_dim=4, inv_freq=[1.0, 0.1], gain=float("inf"))])
def test_plans_refused_by_the_library(L, kw):
    with pytest.raises(pkv.PkvError) as e:
        pkv.RopePlan(**kw)
    assert e.value.status == 1


@pytest.mark.parametrize("kw", [
    dict(scaling={"kind": "other", "factor": 2}), dict(gain=2.0),
    dict(scaling={"kind": "linear", "factor": 2, "original": 5}),
    dict(rotary_dim=8, inv_freq=[1.0]),
    dict(rotary_dim=2, inv_freq=[1.0], scaling={"kind": "linear", "factor": 2})])
def test_plans_refused_by_the_binding(L, kw):
    with pytest.raises(ValueError):
        pkv.RopePlan(**kw)


FAKE = 0x100000
FAR = [FAKE + (i << 24) for i in range(8)]  # never dereferenced: validation fails first


def call(L, rope, **kw):
    a = dict(pos=FAR[0], slots=FAR[1], n=4, q=FAR[2], qs=1024, k=FAR[3], ks=256, v=FAR[4], vs=256,
             out=FAR[5], kc=FAR[6], vc=FAR[7], num_slots=64, bs=16, h=binding.Heads(8, 2, 128))
    a.update(kw)
    return L.pkv_rope_append(a["pos"], a["slots"], a["n"], a["q"], a["qs"], a["k"], a["ks"],
                             a["v"], a["vs"], a["out"], a["kc"], a["vc"], a["num_slots"], a["bs"],
                             a["h"], ctypes.byref(rope) if rope is not None else None, None)


def test_append_refusals(L):
    r = pkv.RopePlan(64).c
    assert call(L, r, n=0, pos=None, q=None) == 0  # nothing to do
    for bad in (dict(n=-1), dict(pos=None), dict(slots=None), dict(q=None), dict(k=None),
                dict(v=None), dict(out=None), dict(kc=None), dict(vc=None), dict(bs=0),
                dict(pos=FAKE + 2), dict(slots=FAKE + 4), dict(q=FAR[2] + 8), dict(k=FAR[3] + 2),
                dict(out=FAR[5] + 8), dict(vc=FAR[7] + 8), dict(qs=-8), dict(ks=252),
                dict(vs=1 << 40), dict(num_slots=-1), dict(h=binding.Heads(9, 2, 128))):
        assert call(L, r, **bad) == 1, bad
        assert L.pkv_last_error() != b""
    assert call(L, r, h=binding.Heads(8, 2, 64)) == 2
    assert call(L, r, h=binding.Heads(32, 2, 128)) == 2
    assert call(L, r, n=1 << 31) == 2
    assert call(L, None) == 1
    broken = pkv.RopePlan(64).c
    broken.rotary_dim = 63
    assert call(L, broken) == 1
    broken.rotary_dim, broken.interleaved = 64, 2
    assert call(L, broken) == 1


def test_append_refuses_overlaps(L):
    r = pkv.RopePlan(64).c
    # q inside a wider row, written in place: rows would land on other tokens
    assert call(L, r, out=FAR[2], qs=2048) == 1 and b"overlaps q" in L.pkv_last_error()
    assert call(L, r, out=FAR[2] + 16) == 1
    assert call(L, r, out=FAR[3]) == 1 and b"k or v" in L.pkv_last_error()
    assert call(L, r, out=FAR[4] + 512) == 1
