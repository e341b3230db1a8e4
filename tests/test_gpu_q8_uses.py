"""Calls over the 8-bit cache as a server makes them: captured and replayed, several at once
on streams of their own, more tiles than 32-bit shares take."""
import pytest
import torch

import paged_kv_cache_245_gb300 as pkv
import q8_ref
from test_gpu_q8_append import Cache
from test_gpu_q8_attention import DEV, SCALE, Batch

pytestmark = pytest.mark.gpu

D = 128


@pytest.fixture(autouse=True)
def _reset():
    pkv.set_checked(False)
    yield
    pkv.set_decode_variant(pkv.VARIANT_AUTO)
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", q8_ref.FORMATS)
@pytest.mark.parametrize("rotary,interleaved", [(128, False), (50, False), (64, True)])
@pytest.mark.parametrize("T", [1, 40, 1040])  # queries in the same launch, and in one before it
def test_rope_append_captured(dtype, rotary, interleaved, T):
    """Replayed over other rows, positions and slots: as the call itself gives."""
    hq, hkv, blocks = 6, 2, 90
    plan = pkv.RopePlan(rotary, interleaved=interleaved)
    caches = [Cache(blocks, hkv, 16, dtype) for _ in range(2)]
    qkv = torch.randn(T, (hq + 2 * hkv) * D, device=DEV).bfloat16()
    q, k, v = (x.unflatten(1, (-1, D)) for x in qkv.split([hq * D, hkv * D, hkv * D], 1))
    pos = torch.arange(T, dtype=torch.int32, device=DEV)
    slots = torch.arange(T, device=DEV)
    out = torch.empty(T, hq, D, dtype=torch.bfloat16, device=DEV)
    for c in caches:
        pkv.rope_append_q8(pos, slots, q, k, v, *c.dev, plan, out=out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pkv.rope_append_q8(pos, slots, q, k, v, *caches[0].dev, plan, out=out)
    for i in range(4):
        gen = torch.Generator(device=DEV).manual_seed(i)
        qkv.copy_(torch.randn(qkv.shape, generator=gen, device=DEV) * (1 + i))
        pos.copy_(torch.randint(0, 1 << 17, (T,), generator=gen, device=DEV))
        slots.copy_(torch.randperm(blocks * 16, generator=gen, device=DEV)[:T])
        slots[i % T] = -1
        out.fill_(7.0)
        g.replay()
        want = pkv.rope_append_q8(pos, slots, q, k, v, *caches[1].dev, plan)
        assert torch.equal(out, want)
        for a, b in zip(*(c.dev for c in caches)):
            assert torch.equal(a.view(torch.int8), b.view(torch.int8))


@pytest.mark.parametrize("dtype", q8_ref.FORMATS)
def test_calls_at_once(dtype):
    """Every kernel on a stream of its own, each call with its workspace, give what they give
    alone."""
    batches = [
        (Batch(dtype, "paged", 32, 8, [1000]), "decode"),                       # a cluster a pair
        (Batch(dtype, "paged", 32, 8, [37 * i + 1 for i in range(64)], seed=1), "decode"),
        (Batch(dtype, "contig", 14, 2, [3000, 17, 900], seed=2), "decode"),
        (Batch(dtype, "paged", 32, 8, [600 + i for i in range(16)], [4] * 16, seed=3), "prefill"),
        (Batch(dtype, "paged", 8, 2, [4064, 700], [64, 33], seed=4), "prefill"),   # cut items
        (Batch(dtype, "paged", 32, 8, [520] * 24, [500] * 24, seed=5), "prefill")]  # whole items
    wants = [getattr(b, call)().clone() for b, call in batches]
    streams = [torch.cuda.Stream() for _ in batches]
    torch.cuda.synchronize()
    for _ in range(15):
        outs = []
        for s, (b, call) in zip(streams, batches):
            with torch.cuda.stream(s):
                outs.append(getattr(b, call)())
        torch.cuda.synchronize()
        for got, want, (b, call) in zip(outs, wants, batches):
            assert torch.equal(got, want), call


@pytest.mark.parametrize("dtype", q8_ref.FORMATS)
def test_more_tiles_than_32_bit_shares(dtype):
    """24 sequences of 8 heads that share one prefix of 100000: more than 2^20 tiles."""
    one = Batch(dtype, "paged", 8, 8, [100003], bs=128)
    n = 24
    b = Batch.__new__(Batch)
    b.__dict__.update(one.__dict__)
    b.lens = [100003 - 1000 * i for i in range(n)]
    b.new = [1] * n
    b.where = one.where.expand(n, -1).contiguous()
    b.ctx = torch.tensor(b.lens, dtype=torch.int32, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(9)
    b.q = (torch.randn(n, 8, D, generator=g, device=DEV) * 4).bfloat16()
    assert sum((c + 15) // 16 + 4 for c in b.lens) * 8 > 1 << 20
    pkv.set_decode_variant(pkv.VARIANT_TC_12X2)
    got = b.decode()
    pkv.set_decode_variant(pkv.VARIANT_AUTO)
    for i in (0, 11, 23):
        k, v = b.rows(i)
        want, tol = q8_ref.attend64(b.q[i:i + 1], k, v, [b.lens[i] - 1], SCALE)
        q8_ref.assert_close(got[i:i + 1], want, tol, "sequence %d" % i)
