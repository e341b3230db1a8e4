"""The rotary append to the 8-bit cache: rows that it does not write, NaN and infinities
among the turned elements, checked mode."""
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_245_gb300 as pkv
import q8_ref
from test_gpu_q8_append import D, DEV, Cache, turned

pytestmark = pytest.mark.gpu

LAYOUTS = [(128, True), (50, True), (128, False), (64, False), (50, False), (126, False)]


@pytest.fixture(autouse=True)
def _reset():
    pkv.set_checked(False)
    yield
    pkv.set_checked(False)
    torch.cuda.synchronize()


def rows(T, hq, hkv, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return [torch.randn(T, n, D, generator=g, device=DEV).bfloat16() for n in (hq, hkv, hkv)]


def whole(c):
    return [x.cpu().view(torch.int8) if x.dtype != torch.float32 else x.cpu() for x in c.dev]


@pytest.mark.parametrize("dtype", q8_ref.FORMATS)
@pytest.mark.parametrize("rotary,interleaved", LAYOUTS)
@pytest.mark.parametrize("T,spread", [(1, 300), (40, 1000), (1100, 9000)])
def test_other_groups_stay(dtype, rotary, interleaved, T, spread):
    """Codes and scales of groups that the call does not write to, bit for bit; K and V."""
    hq, hkv, bs = 4, 2, 48
    plan = pkv.RopePlan(rotary, theta=500000.0, interleaved=interleaved)
    c = Cache(spread // bs + 2, hkv, bs, dtype, seed=T)
    slots = torch.randperm(spread, generator=torch.Generator().manual_seed(T))[:T]
    if T > 1:
        slots[T // 2] = -1
    pos = torch.arange(T, dtype=torch.int32, device=DEV) + 31
    before = whole(c)
    pkv.rope_append_q8(pos, slots.to(DEV), *rows(T, hq, hkv), *c.dev, plan)
    after = whole(c)
    groups = torch.unique(slots[slots >= 0] // 16)
    per = bs // 16
    touched = torch.zeros(before[0].shape[0] * per, dtype=torch.bool)
    touched[groups] = True
    touched = touched.view(-1, 1, per)
    for a, b in zip(before, after):
        same = (a == b) if a.dim() == 3 else (a == b).unflatten(2, (per, 16)).all(-1).all(-1)
        assert bool((same | touched).all())
        assert not bool(same[touched.expand_as(same)].all())  # the others are written


@pytest.mark.parametrize("dtype", q8_ref.FORMATS)
@pytest.mark.parametrize("rotary,interleaved", LAYOUTS)
@pytest.mark.parametrize("T", [40, 1040])
def test_non_finite_pairs(dtype, rotary, interleaved, T):
    """NaN and infinities among the turned elements: both of the pair follow the turn, and
    no other code and no scale changes."""
    hq, hkv = 4, 2
    half = rotary // 2
    plan = pkv.RopePlan(rotary, interleaved=interleaved)
    q, k, v = rows(T, hq, hkv, seed=rotary)
    pos = torch.arange(T, dtype=torch.int32) + 77
    slots = torch.arange(T, device=DEV)
    # (token, head, pair, which of the pair): one in each place of a lane's chunks
    odd = {(3, 0, 0, 0): math.nan, (3, 1, half - 1, 1): math.inf, (20, 0, half // 2, 0): -math.inf,
           (21, 0, 1, 1): -math.inf, (38, 1, half // 3, 0): math.inf, (39, 1, half - 2, 1): math.nan}

    def element(pair, which):
        return 2 * pair + which if interleaved else pair + which * half

    bad = torch.zeros(T, hkv, D, dtype=torch.bool)
    for (t, h, i, w) in odd:
        bad[t, h, element(i, 0)] = bad[t, h, element(i, 1)] = True
    base = k.clone()
    k[bad.to(DEV)] = 0.0  # turned: zeros
    caches = [Cache(T // 16 + 1, hkv, 16, dtype) for _ in range(2)]
    pkv.rope_append_q8(pos.to(DEV), slots, q, k, v, *caches[0].dev, plan)
    k = base
    for (t, h, i, w), x in odd.items():
        k[t, h, element(i, w)] = x
    pkv.rope_append_q8(pos.to(DEV), slots, q, k, v, *caches[1].dev, plan)
    clean, got = whole(caches[0]), whole(caches[1])
    with np.errstate(invalid="ignore"):
        want, _ = turned(k.double().cpu().numpy(), pos, plan)
    code = caches[1].dev[0].float().cpu()
    top = float(q8_ref.QMAX[dtype])
    for t, h, e in bad.nonzero().tolist():
        x = float(want[t, h, e])
        assert not math.isfinite(x)
        y = float(code[t // 16, h, t % 16, e])
        if math.isnan(x):
            assert y == 0.0 if dtype == torch.int8 else math.isnan(y)
        else:
            assert y == math.copysign(top, x)
    spot = torch.zeros(clean[0].shape, dtype=torch.bool)
    at = torch.arange(T)
    spot[at // 16, :, at % 16] = bad
    assert bool(((clean[0] == got[0]) | spot).all())
    for a, b in zip(clean[1:], got[1:]):
        assert torch.equal(a, b)


@pytest.mark.parametrize("T", [5, 1040])
def test_rope_checked(T):
    """Slots past the cache are reported and skipped; queries and other rows are as ever."""
    hq, hkv = 4, 2
    plan = pkv.RopePlan(128)
    q, k, v = rows(T, hq, hkv)
    pos = torch.arange(T, dtype=torch.int32, device=DEV)
    good = torch.arange(T, device=DEV)
    good[3] = -1
    wrong = good.clone()
    caches = [Cache(T // 16 + 1, hkv, 16, torch.int8) for _ in range(2)]
    wrong[3] = caches[0].dev[0].shape[0] * 16
    want = pkv.rope_append_q8(pos, good, q, k, v, *caches[0].dev, plan)
    pkv.set_checked(True)
    got = pkv.rope_append_q8(pos, wrong, q, k, v, *caches[1].dev, plan)
    assert pkv.get_device_error() == "slot"
    assert pkv.get_device_error() == "none"
    assert torch.equal(got, want)
    for a, b in zip(*(whole(c) for c in caches)):
        assert torch.equal(a, b)
