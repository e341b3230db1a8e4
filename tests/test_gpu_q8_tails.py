"""Attention over the 8-bit cache where one key has nearly all of the softmax and values of
zero, so that the output is what thousands of keys of tiny probability give; contexts of
100000 and more.

Bounds, relative to sum_j w_j |v_j|: a probability's rounding (half a step of fp16 or bf16);
the fp32 sums of c keys, of which a lane adds up c / 8 and an output c / 16 tiles'
products, 2^-24 each (2^-26 c together); exponentials and products 2^-18.  Decode rounds
probabilities times 2^15 to fp16: below 2^-29 of the largest one they are off by half of
fp16's smallest step, 2^-25 2^-15 = 2^-40.  The output's rounding to bf16 is 2^-8."""
import math

import pytest
import torch

import paged_kv_cache_245_gb300 as pkv
import q8_ref
from test_gpu_q8_attention import DEV, VARIANTS, Batch

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _reset():
    pkv.set_checked(False)
    yield
    pkv.set_decode_variant(pkv.VARIANT_AUTO)
    torch.cuda.synchronize()


def sinks(dtype, ctx, new, at, low, v_up, hq=8, hkv=2, layout="paged"):
    """Keys whose score is their code's first element: 16 for position `at` (from the end
    if negative) of each sequence, whose value is zero, and 16 - low nats for the others;
    low None: 13 to 18 nats below, by turns.  Values of one sign, 2^v_up apart in scale."""
    b = Batch(dtype, layout, hq, hkv, ctx, new, bs=128)
    b.q.zero_()
    b.q[..., 0] = 1.0
    b.ks.masked_fill_(~b.ks.isnan(), 1.0)
    g = torch.Generator(device=DEV).manual_seed(4)
    up = torch.randint(0, v_up + 1, b.vs.shape, generator=g, device=DEV)
    b.vs.copy_(torch.where(b.vs.isnan(), b.vs, torch.exp2(up.float() - 6)))
    for i, c in enumerate(ctx):
        pos = torch.arange(c, device=DEV)
        blocks = torch.tensor(b.blocks(i), device=DEV)[pos // b.bs]
        code = 16 - (low if low is not None else 13 + pos % 6)
        code = torch.as_tensor(code, device=DEV).expand(c).float()
        value = torch.randint(3, 16, (c, hkv, 128), generator=g, device=DEV).float()
        first = at if at >= 0 else c + at
        code = torch.where(pos == first, 16.0, code)
        value[first] = 0.0
        row = torch.zeros(c, hkv, 128, device=DEV)
        row[:, :, 0] = code[:, None]
        for cache, x in ((b.k, row), (b.v, value)):
            cache.view(torch.int8)[blocks, :, pos % b.bs] = x.to(dtype).view(torch.int8)
    return b


def check(b, got, half_step, floor):
    at = 0
    for i, (c, n) in enumerate(zip(b.lens, b.new)):
        k, v = b.rows(i)
        group = b.q.shape[1] // b.hkv
        pos = torch.arange(c - n, c, device=DEV)
        seen = torch.arange(c, device=DEV) <= pos[:, None]
        for h in range(b.q.shape[1]):
            z = (b.q[at:at + n, h].double() @ k[h // group].T).masked_fill(~seen, -math.inf)
            w = torch.exp(z - z.amax(-1, keepdim=True))
            total = w.sum(-1, keepdim=True)
            low = seen.double() * floor / total
            w = w / total
            want, size = w @ v[h // group], w @ v[h // group].abs()
            tol = (half_step + c * 2.0 ** -26 + 2.0 ** -18) * size + low @ v[h // group].abs() \
                + want.abs() * 2.0 ** -8
            q8_ref.assert_close(got[at:at + n, h], want, tol, "sequence %d head %d" % (i, h))
        at += n


DECODE_FLOOR = 2.0 ** -40


@pytest.mark.parametrize("dtype", q8_ref.FORMATS)
@pytest.mark.parametrize("variant", VARIANTS)
@pytest.mark.parametrize("at", [0, 700, -1])
@pytest.mark.parametrize("low", [13, 16, 17, 18, None])
def test_decode_tail(dtype, variant, at, low):
    pkv.set_decode_variant(variant)
    b = sinks(dtype, [8000, 1111], None, at, low, 0)
    check(b, b.decode(scale=1.0), q8_ref.DECODE, DECODE_FLOOR)


@pytest.mark.parametrize("dtype", q8_ref.FORMATS)
@pytest.mark.parametrize("variant", VARIANTS)
def test_decode_tail_of_uneven_scales(dtype, variant):
    """Groups of values 2^12 apart: the largest values stand at small probabilities."""
    pkv.set_decode_variant(variant)
    b = sinks(dtype, [5000, 300], None, 3, None, 12)
    check(b, b.decode(scale=1.0), q8_ref.DECODE, DECODE_FLOOR)


@pytest.mark.parametrize("dtype", q8_ref.FORMATS)
@pytest.mark.parametrize("at", [0, 700])
@pytest.mark.parametrize("low", [13, 16, 17, 18, None])
def test_short_chunk_tail(dtype, at, low):
    b = sinks(dtype, [3000, 1500] * 4, [4, 3] * 4, at, low, 0, hq=16, hkv=4)  # 32 pairs: by runs
    check(b, b.prefill(scale=1.0), q8_ref.DECODE, DECODE_FLOOR)


@pytest.mark.parametrize("dtype", q8_ref.FORMATS)
@pytest.mark.parametrize("at", [0, 700])
@pytest.mark.parametrize("low", [13, 16, 17, 18, None])
@pytest.mark.parametrize("new", [[40, 3], [300, 200]])
def test_prefill_tail(dtype, at, low, new):
    b = sinks(dtype, [6000, 1500], new, at, low, 0)
    check(b, b.prefill(scale=1.0), q8_ref.PREFILL, 0.0)


@pytest.mark.parametrize("dtype", q8_ref.FORMATS)
def test_prefill_tail_of_uneven_scales(dtype):
    b = sinks(dtype, [5000, 900], [100, 50], 3, None, 12)
    check(b, b.prefill(scale=1.0), q8_ref.PREFILL, 0.0)


@pytest.mark.parametrize("dtype", q8_ref.FORMATS)
@pytest.mark.parametrize("variant", VARIANTS)
@pytest.mark.parametrize("layout", ["paged", "contig"])
def test_decode_long(dtype, variant, layout):
    """One key far above 100000 equal ones, and a short sequence beside it."""
    pkv.set_decode_variant(variant)
    b = sinks(dtype, [100001, 77], None, 0, 17, 0, hq=4, hkv=1, layout=layout)
    check(b, b.decode(scale=1.0), q8_ref.DECODE, DECODE_FLOOR)


@pytest.mark.parametrize("dtype", q8_ref.FORMATS)
@pytest.mark.parametrize("new", [[3, 2], [70, 1]])
def test_prefill_long(dtype, new):
    b = sinks(dtype, [131072, 40], new, 0, 17, 0, hq=4, hkv=1)
    check(b, b.prefill(scale=1.0), q8_ref.PREFILL, 0.0)


@pytest.mark.parametrize("dtype", q8_ref.FORMATS)
@pytest.mark.parametrize("variant", VARIANTS)
def test_long_contexts(dtype, variant):
    """Contexts of 32K to 128K of keys like any others', one token each and chunks."""
    pkv.set_decode_variant(variant)
    b = Batch(dtype, "paged", 8, 1, [32768, 65537, 130001], bs=64)
    b.check(b.decode())
    b = Batch(dtype, "paged", 8, 1, [40000, 70000], [33, 5], bs=64)
    b.check(b.prefill(), half_step=q8_ref.PREFILL)
