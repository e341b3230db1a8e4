"""Attention over the 8-bit cache (pkv_*_attention_q8) against the formula in 64
bits: formats, layouts, groups, block sizes, lengths, scales, unread rows."""
import math

import pytest
import torch

import paged_kv_cache_245_gb300 as pkv
import q8_ref

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
D = 128
SCALE = D ** -0.5


@pytest.fixture(autouse=True)
def _reset():
    pkv.set_checked(False)
    yield
    pkv.set_checked(False)
    pkv.set_decode_variant(pkv.VARIANT_AUTO)
    torch.cuda.synchronize()


# decode's kernels: the call's own choice, by clusters, by warp runs
VARIANTS = [pkv.VARIANT_AUTO, pkv.VARIANT_SPLIT, pkv.VARIANT_TC_12X2]


@pytest.fixture(params=VARIANTS)
def variant(request):
    pkv.set_decode_variant(request.param)
    return request.param


class Batch:
    """Sequences of given contexts (and new tokens) over an 8-bit cache whose other
    rows, groups and blocks hold NaN."""

    def __init__(self, dtype, layout, hq, hkv, ctx, new=None, bs=16, seed=0, by=4.0):
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.dtype, self.contig, self.hkv, self.bs = dtype, layout == "contig", hkv, bs
        self.lens, self.new = ctx, new or [1] * len(ctx)
        B, top = len(ctx), max(max(ctx), 1)
        self.top = top
        if self.contig:
            self.bs = bs = (top + 15) // 16 * 16
            order = torch.randperm(B + 2, generator=g, device=DEV)[:B]
            self.where, n, need = order.to(torch.int32), B + 2, [1] * B
        else:
            need = [(c + bs - 1) // bs for c in ctx]
            n = sum(need) + 2
            pool = torch.randperm(n, generator=g, device=DEV).tolist()
            self.where = torch.full((B, max(max(need), 1)), -7, dtype=torch.int32)
            at = 0
            for i, m in enumerate(need):
                self.where[i, :m] = torch.tensor(pool[at:at + m], dtype=torch.int32)
                at += m
            self.where = self.where.to(DEV)
        shape, per = (n, hkv, bs, D), (n, hkv, bs // 16)
        self.k, self.v = (q8_ref.random_codes(shape, dtype, g, DEV) for _ in range(2))
        self.ks, self.vs = (q8_ref.random_scales(per, dtype, g, DEV) for _ in range(2))
        self.q = (torch.randn(sum(self.new), hq, D, generator=g, device=DEV) * by).bfloat16()
        self.ctx = torch.tensor(ctx, dtype=torch.int32, device=DEV)
        self.cu = torch.tensor([0] + self.new, dtype=torch.int32).cumsum(0).to(torch.int32).to(DEV)
        self.spoil()

    def blocks(self, i):
        if self.contig:
            return [int(self.where[i])]
        return self.where[i, :(self.lens[i] + self.bs - 1) // self.bs].tolist()

    def spoil(self):
        """NaN into everything that no sequence sees."""
        seen = torch.zeros(self.k.shape[0], self.bs, dtype=torch.bool, device=DEV)
        for i, c in enumerate(self.lens):
            for j, b in enumerate(self.blocks(i) if c else []):
                seen[b, :max(0, min(self.bs, c - j * self.bs))] = True
        for x in (self.k, self.v):
            bytes_ = x.view(torch.int8)
            bytes_.masked_fill_(~seen[:, None, :, None], 127 if self.dtype == torch.float8_e4m3fn
                                else -128)
        unread = ~seen.view(seen.shape[0], -1, 16).any(2)
        for s in (self.ks, self.vs):
            s.masked_fill_(unread[:, None], math.nan)

    def rows(self, i):
        c, out = self.lens[i], []
        for x, s in ((self.k, self.ks), (self.v, self.vs)):
            b = torch.tensor(self.blocks(i), device=DEV)
            x = x.view(torch.int8)[b].view(self.dtype)
            out.append(torch.cat(list(q8_ref.values(x, s[b])), 1)[:, :c])
        return out

    def check(self, got, scale=SCALE, half_step=q8_ref.DECODE):
        at = 0
        for i, (c, n) in enumerate(zip(self.lens, self.new)):
            mine = got[at:at + n]
            if c == 0:
                assert bool((mine == 0).all())
            elif n:
                k, v = self.rows(i)
                want, tol = q8_ref.attend64(self.q[at:at + n], k, v, range(c - n, c), scale,
                                            half_step)
                q8_ref.assert_close(mine, want, tol, "sequence %d (context %d)" % (i, c))
            at += n

    def decode(self, max_context=None, scale=SCALE, **more):
        call = pkv.contig_decode_attention_q8 if self.contig else pkv.paged_decode_attention_q8
        return call(self.q, self.k, self.v, self.ks, self.vs, self.where, self.ctx,
                    self.top if max_context is None else max_context, scale, **more)

    def prefill(self, max_new=None, scale=SCALE, **more):
        call = pkv.contig_prefill_attention_q8 if self.contig else pkv.paged_prefill_attention_q8
        return call(self.q, self.cu, self.k, self.v, self.ks, self.vs, self.where, self.ctx,
                    max(self.new) if max_new is None else max_new, scale, **more)


HEADS = [(4, 4), (10, 2), (20, 4), (32, 8), (6, 1), (14, 2), (8, 1)]


# ------------------------------------------------------------------ one token a sequence

@pytest.mark.parametrize("dtype", q8_ref.FORMATS)
@pytest.mark.parametrize("layout", ["paged", "contig"])
@pytest.mark.parametrize("hq,hkv", HEADS)
def test_decode_heads(variant, dtype, layout, hq, hkv):
    b = Batch(dtype, layout, hq, hkv, [1, 15, 16, 17, 0, 100, 257, 640])
    b.check(b.decode())


@pytest.mark.parametrize("dtype", q8_ref.FORMATS)
@pytest.mark.parametrize("bs", [16, 32, 48, 64, 128, 272])
def test_decode_block_sizes(variant, dtype, bs):
    b = Batch(dtype, "paged", 8, 2, [bs - 1, bs, bs + 1, 3 * bs + 5, 1], bs=bs)
    b.check(b.decode())


@pytest.mark.parametrize("dtype", q8_ref.FORMATS)
@pytest.mark.parametrize("ctx", [[1], [16], [1000], [4000], [9001], [300] * 4, [700] * 40,
                                 [1, 8192] + [50] * 30, [2500] * 64, [5] * 600, [300] * 19 + [1] * 19, [200] * 90])
def test_decode_lengths(variant, dtype, ctx):
    b = Batch(dtype, "paged", 8, 2, ctx, bs=32)
    b.check(b.decode())


def test_decode_wide_bound(variant):
    """A max_context far above the contexts."""
    b = Batch(torch.int8, "paged", 8, 2, [40, 3, 900], bs=16)
    b.where = torch.cat([b.where, torch.full((3, 3000), -7, dtype=torch.int32, device=DEV)], 1)
    b.check(b.decode(max_context=40000))


@pytest.mark.parametrize("dtype", q8_ref.FORMATS)
@pytest.mark.parametrize("scale", [0.0, -0.2, 1.0, 1e-6])
def test_decode_scales(variant, dtype, scale):
    b = Batch(dtype, "paged", 8, 2, [70, 1, 333], by=1.0)
    b.check(b.decode(scale=scale), scale=scale)


def spread_scales(b, low, high):
    """Scales from 2^low to 2^high, some zero."""
    g = torch.Generator(device=DEV).manual_seed(3)
    for s in (b.ks, b.vs):
        e = torch.randint(low, high + 1, s.shape, generator=g, device=DEV)
        new = torch.exp2(e.float()) * (e % 5 != 0)
        s.copy_(torch.where(s.isnan(), s, new))


@pytest.mark.parametrize("dtype", q8_ref.FORMATS)
def test_decode_uneven_groups(variant, dtype):
    """Neighbouring groups whose scales differ by orders of magnitude, zeros among them."""
    b = Batch(dtype, "paged", 8, 2, [500, 37, 2100], by=0.01)
    spread_scales(b, -24, 4)
    b.check(b.decode())


def test_decode_large_queries(variant):
    b = Batch(torch.int8, "paged", 8, 2, [200, 17], by=2.0 ** 18)
    b.check(b.decode(scale=2.0 ** -24), scale=2.0 ** -24)
    b = Batch(torch.int8, "paged", 8, 2, [200, 17], by=2.0 ** -40)
    b.check(b.decode(scale=2.0 ** 37), scale=2.0 ** 37)


def test_decode_streams_and_capture(variant):
    b = Batch(torch.float8_e4m3fn, "paged", 8, 2, [900, 40, 1, 2000])
    b.check(b.decode())
    out = torch.empty_like(b.q)
    size = pkv.q8_decode_workspace_size(4, 8, 2, b.top)
    ws = torch.empty(max(size, 16), dtype=torch.uint8, device=DEV)
    ws.fill_(0xff)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.decode(out=out, workspace=ws)
    full = list(b.lens)
    for lens in (full, [1, 40, 0, 1500], [899, 13, 1, 16], full):  # replayed over other lengths
        b.lens = lens
        b.ctx.copy_(torch.tensor(lens, dtype=torch.int32))
        out.fill_(7.0)
        g.replay()
        b.check(out)


def test_decode_checked(variant):
    b = Batch(torch.int8, "paged", 8, 2, [100, 60])
    pkv.set_checked(True)
    b.check(b.decode())
    assert pkv.get_device_error() == "none"
    b.where[0, 2] = 10 ** 6
    b.decode()
    assert pkv.get_device_error() == "block_id"
    b.decode(max_context=90)
    assert pkv.get_device_error() in ("context", "block_id")
    b.where[0, 2] = 0
    b.decode(max_context=90)
    assert pkv.get_device_error() == "context"
    c = Batch(torch.int8, "contig", 8, 2, [100, 60])
    c.where[1] = 99
    c.decode()
    assert pkv.get_device_error() == "req_id"


def odd_rows(b, run, half_step):
    """Queries with NaN and infinities make their own row and head NaN, no other."""
    clean = run().clone()
    b.check(clean, half_step=half_step)
    q, bad = b.q.clone(), torch.zeros(b.q.shape[:2], dtype=torch.bool, device=DEV)
    for (t, h, e), x in (((0, 1, 3), math.nan), ((2, 0, 127), math.inf), ((2, 5, 64), -math.inf),
                         ((b.q.shape[0] - 1, 7, 0), math.nan)):
        b.q[t, h, e], bad[t, h] = x, True
    got = run()
    assert bool(got[bad].isnan().all())
    b.q = q
    b.check(torch.where(bad[..., None], clean, got), half_step=half_step)


def odd_cache(b, run, half_step):
    """A visible NaN code or scale makes its sequence's and KV head's rows NaN, no others."""
    clean = run().clone()
    at = b.blocks(1)[0]
    if b.dtype == torch.float8_e4m3fn:
        spot, odd = b.k.view(torch.int8)[at, 1, 0, 100:101], 127
    else:
        spot, odd = b.ks[at, 1, :1], math.nan
    was = spot.clone()
    spot.fill_(odd)
    got = run()
    spot.copy_(was)
    first, group = sum(b.new[:1]), b.q.shape[1] // b.hkv
    bad = torch.zeros(b.q.shape[:2], dtype=torch.bool, device=DEV)
    bad[first:first + b.new[1], group:2 * group] = True
    assert bool(got[bad].isnan().all())
    b.check(torch.where(bad[..., None], clean, got), half_step=half_step)


@pytest.mark.parametrize("dtype", q8_ref.FORMATS)
def test_decode_non_finite(variant, dtype):
    b = Batch(dtype, "paged", 8, 2, [900, 40, 17, 300])
    odd_rows(b, b.decode, q8_ref.DECODE)
    odd_cache(b, b.decode, q8_ref.DECODE)


def test_decode_two_graphs_one_workspace(variant):
    """Replayed one after another, graphs may share what they work in."""
    bs = [Batch(torch.int8, "paged", 8, 2, lens, seed=i)
          for i, lens in enumerate(([3000, 40], [10, 2000, 700]))]
    ws = torch.empty(max(pkv.q8_decode_workspace_size(len(b.lens), 8, 2, b.top) for b in bs),
                     dtype=torch.uint8, device=DEV)
    graphs, outs = [], [torch.empty_like(b.q) for b in bs]
    for b, out in zip(bs, outs):
        b.decode(out=out, workspace=ws)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            b.decode(out=out, workspace=ws)
        graphs.append(g)
    for _ in range(3):
        for g, b, out in zip(graphs, bs, outs):
            out.fill_(7.0)
            g.replay()
            b.check(out)


@pytest.mark.parametrize("layout", ["paged", "contig"])
def test_decode_many_sequences(variant, layout):
    """More sequences than one launch of the warp runs takes."""
    lens = [(37 * i) % 90 for i in range(1100)]
    b = Batch(torch.int8, layout, 4, 1, lens)
    b.check(b.decode())


def test_blocks_past_32_bits():
    """Codes beyond 2^32 bytes from the cache's start give what they give near it."""
    hkv, bs, blocks = 8, 16, 300000
    assert blocks * hkv * bs * D > 2 ** 32
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB of device memory")
    k, v = (torch.zeros(blocks, hkv, bs, D, dtype=torch.int8, device=DEV) for _ in range(2))
    ks, vs = (torch.zeros(blocks, hkv, 1, device=DEV) for _ in range(2))
    T = 100
    g = torch.Generator(device=DEV).manual_seed(3)
    rows = [torch.randn(T, hkv, D, generator=g, device=DEV).bfloat16() for _ in range(2)]
    q = torch.randn(T, 32, D, generator=g, device=DEV).bfloat16()
    outs = []
    for first in (0, blocks - 7):
        table = torch.arange(first, first + 7, dtype=torch.int32, device=DEV)[None]
        pkv.kv_append_q8(torch.arange(T, device=DEV) + first * bs, *rows, k, v, ks, vs)
        where = (k, v, ks, vs, table.contiguous(), torch.tensor([T], dtype=torch.int32, device=DEV))
        got = [k[first:first + 7].clone(), ks[first:first + 7].clone()]
        for n in (T, 3):
            cu = torch.tensor([0, n], dtype=torch.int32, device=DEV)
            got.append(pkv.paged_prefill_attention_q8(q[:n], cu, *where, n, SCALE))
        # enough chunks for the warp runs
        many = (where[4].expand(4, 7).contiguous(), where[5].expand(4).contiguous())
        cu = torch.arange(0, 10, 2, dtype=torch.int32, device=DEV)
        got.append(pkv.paged_prefill_attention_q8(q[:8], cu, *where[:4], *many, 2, SCALE))
        for choice in VARIANTS:
            pkv.set_decode_variant(choice)
            got.append(pkv.paged_decode_attention_q8(q[:1], *where, T, SCALE))
        pkv.set_decode_variant(pkv.VARIANT_AUTO)
        outs.append(got)
    for a, b in zip(*outs):
        assert torch.equal(a, b)
    assert all(bool((x != 0).any()) for x in outs[0])


# ------------------------------------------------------------------ chunks

@pytest.mark.parametrize("dtype", q8_ref.FORMATS)
@pytest.mark.parametrize("layout", ["paged", "contig"])
@pytest.mark.parametrize("hq,hkv", HEADS)
def test_prefill_heads(dtype, layout, hq, hkv):
    new = [1, 5, 17, 64, 130, 33]
    b = Batch(dtype, layout, hq, hkv, [n + c for n, c in zip(new, [0, 20, 0, 127, 300, 1])], new)
    b.check(b.prefill(), half_step=q8_ref.PREFILL)


@pytest.mark.parametrize("dtype", q8_ref.FORMATS)
@pytest.mark.parametrize("bs", [16, 32, 48, 64, 128, 272])
def test_prefill_block_sizes(dtype, bs):
    b = Batch(dtype, "paged", 8, 2, [bs - 1, 2 * bs + 3, 3 * bs, 500 + bs], [bs - 1, bs + 3, 1, 77],
              bs=bs)
    b.check(b.prefill(), half_step=q8_ref.PREFILL)


@pytest.mark.parametrize("dtype", q8_ref.FORMATS)
@pytest.mark.parametrize("new,cached", [([1], [0]), ([1], [5000]), ([700], [0]), ([64], [4000]),
                                        ([3] * 20, list(range(0, 2000, 100))), ([128] * 3, [128] * 3),
                                        ([1500, 2, 1], [7, 2500, 0]), ([300] * 40, [10] * 40)])
def test_prefill_lengths(dtype, new, cached):
    b = Batch(dtype, "paged", 8, 2, [n + c for n, c in zip(new, cached)], new, bs=32)
    b.check(b.prefill(), half_step=q8_ref.PREFILL)


@pytest.mark.parametrize("dtype", q8_ref.FORMATS)
@pytest.mark.parametrize("scale", [0.0, -0.2, 1.0, 1e-6])
def test_prefill_scales(dtype, scale):
    b = Batch(dtype, "paged", 8, 2, [70, 1, 333], [70, 1, 140], by=1.0)
    b.check(b.prefill(scale=scale), scale=scale, half_step=q8_ref.PREFILL)


@pytest.mark.parametrize("dtype", q8_ref.FORMATS)
def test_prefill_uneven_groups(dtype):
    b = Batch(dtype, "paged", 8, 2, [500, 37, 2100], [500, 20, 60], by=0.01)
    spread_scales(b, -24, 4)
    b.check(b.prefill(), half_step=q8_ref.PREFILL)


def test_prefill_large_queries():
    b = Batch(torch.int8, "paged", 8, 2, [200, 17], [150, 17], by=2.0 ** 18)
    b.check(b.prefill(scale=2.0 ** -24), scale=2.0 ** -24, half_step=q8_ref.PREFILL)
    b = Batch(torch.int8, "paged", 8, 2, [200, 17], [150, 17], by=2.0 ** -40)
    b.check(b.prefill(scale=2.0 ** 37), scale=2.0 ** 37, half_step=q8_ref.PREFILL)


def test_prefill_rows_behind_the_last_chunk():
    b = Batch(torch.int8, "paged", 8, 2, [40, 70], [40, 30])
    tail = torch.full((9, 8, D), math.nan, device=DEV).bfloat16()
    b.q = torch.cat([b.q, tail])
    out = torch.full_like(b.q, 3.0)
    b.prefill(max_new=2 ** 31 - 1, out=out)
    assert bool((out[70:] == 3.0).all())
    b.check(out, half_step=q8_ref.PREFILL)


@pytest.mark.parametrize("dtype", q8_ref.FORMATS)
@pytest.mark.parametrize("new,cached", [([300] * 40, [10] * 40), ([8] * 60, [700] * 60),
                                        ([20] * 5, [3000] * 5), ([33] * 80, [500] * 80)])
def test_prefill_again(dtype, new, cached):
    """Nothing depends on timing: every call gives the same bits."""
    b = Batch(dtype, "paged", 8, 2, [n + c for n, c in zip(new, cached)], new, bs=32)
    first = b.prefill().clone()
    b.check(first, half_step=q8_ref.PREFILL)
    for _ in range(20):
        assert torch.equal(b.prefill(), first)


def test_prefill_empty_chunks():
    b = Batch(torch.int8, "paged", 8, 2, [40, 70, 0, 5], [0, 30, 0, 5])
    b.check(b.prefill(), half_step=q8_ref.PREFILL)


@pytest.mark.parametrize("dtype", q8_ref.FORMATS)
@pytest.mark.parametrize("layout", ["paged", "contig"])
@pytest.mark.parametrize("hq,hkv", HEADS)
def test_short_chunks(dtype, layout, hq, hkv):
    """Chunks of few tokens take decode's arithmetic, 16 rows at a time."""
    most = 2 * (16 // (hq // hkv))
    new = [most, 1, most - 1, 0, most // 2, most // 2 + 1, 2, 1] * 4
    cached = [0, 0, 14, 0, 100, 1000, 31, 257, 1, 20, 0, 7, 999, 15, 16, 17] * 2
    b = Batch(dtype, layout, hq, hkv, [n + c for n, c in zip(new, cached)], new)
    b.check(b.prefill())
    new = [1 + (most // 2 - 1) * (i % 2) for i in range(32)]
    b = Batch(dtype, layout, hq, hkv, [n + c for n, c in zip(new, cached)], new)
    b.check(b.prefill())


@pytest.mark.parametrize("dtype", q8_ref.FORMATS)
@pytest.mark.parametrize("new,cached", [([2], [9000]), ([1] * 300, [50] * 300), ([8, 1] * 120, [90] * 240),
                                        ([8, 1, 5] * 6, [30000, 0, 1] * 6), ([4] * 16, [300] * 16),
                                        ([4, 1, 2] * 400, [i % 77 for i in range(1200)]),
                                        ([8, 1, 0] * 200, [i % 77 for i in range(600)]),
                                        ([3, 8] * 20, list(range(0, 2000, 50)))])
def test_short_chunk_lengths(dtype, new, cached):
    b = Batch(dtype, "paged", 8, 2, [n + c for n, c in zip(new, cached)], new, bs=32)
    first = b.prefill().clone()
    b.check(first)
    for _ in range(10):
        assert torch.equal(b.prefill(), first)


def test_short_chunks_captured():
    b = Batch(torch.float8_e4m3fn, "paged", 48, 12, [300, 700, 20], [4, 2, 2])
    tail = torch.full((5, 48, D), math.nan, device=DEV).bfloat16()
    b.q = torch.cat([b.q, tail])  # 13 rows for 3 chunks
    out = torch.full_like(b.q, 3.0)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.prefill(max_new=8, out=out)
    for lens, new in (([300, 700, 20], [4, 2, 2]), ([290, 650, 0], [1, 7, 0]), ([140, 0, 3], [5, 0, 3])):
        b.lens, b.new = lens, new
        b.ctx.copy_(torch.tensor(lens, dtype=torch.int32))
        b.cu.copy_(torch.tensor([0] + new, dtype=torch.int32).cumsum(0).to(torch.int32))
        for _ in range(2):
            out.fill_(3.0)
            g.replay()
            b.check(out)
            assert bool((out[sum(new):] == 3.0).all())


def test_short_chunks_checked():
    b = Batch(torch.int8, "paged", 64, 16, [100, 60], [5, 6])
    pkv.set_checked(True)
    b.check(b.prefill())
    assert pkv.get_device_error() == "none"
    b.prefill(max_new=5)
    assert pkv.get_device_error() == "context"
    b.where[0, 2] = 10 ** 6
    b.prefill()
    assert pkv.get_device_error() == "block_id"


@pytest.mark.parametrize("dtype", q8_ref.FORMATS)
@pytest.mark.parametrize("new,cached", [([3, 4, 2, 1] * 3, [200, 30, 14, 900] * 3),
                                        ([200, 30, 14, 65], [800, 9, 0, 3])])
def test_prefill_non_finite(dtype, new, cached):
    b = Batch(dtype, "paged", 8, 2, [n + c for n, c in zip(new, cached)], new)
    odd_rows(b, b.prefill, q8_ref.PREFILL)
    odd_cache(b, b.prefill, q8_ref.PREFILL)


@pytest.mark.parametrize("new,cached,heads", [
    ([2100] * 12, [0] * 12, (32, 8)),                     # more items than are cut by tiles
    ([70] * 600, [20] * 600, (8, 2)),                     # more pairs than are sorted
    ([40] * 560, list(range(560)), (8, 2)), ([1000] * 6, [3, 100, 2000, 0, 64, 640], (14, 2))])
def test_prefill_schedules(new, cached, heads):
    b = Batch(torch.float8_e4m3fn, "paged", *heads, [n + c for n, c in zip(new, cached)], new, bs=32)
    b.check(b.prefill(), half_step=q8_ref.PREFILL)


@pytest.mark.parametrize("new,cached", [([64], [4000]), ([3, 4] * 6, [900] * 12)])
def test_prefill_workspace_and_streams(new, cached):
    b = Batch(torch.int8, "paged", 8, 2, [n + c for n, c in zip(new, cached)], new)
    size = pkv.q8_prefill_workspace_size(sum(new), len(new), max(new), 8, 2)
    assert size > 0
    ws = torch.empty(size + 32, dtype=torch.uint8, device=DEV)
    assert ws.data_ptr() % 32 == 0
    with pytest.raises(pkv.PkvError):
        b.prefill(workspace=ws[:size - 1])
    with pytest.raises(pkv.PkvError):
        b.prefill(workspace=ws[16:16 + size])
    ws.fill_(0xff)
    out = torch.empty_like(b.q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b.prefill(workspace=ws[:size], out=out)
    s.synchronize()
    b.check(out, half_step=q8_ref.PREFILL)
    # two graphs over one workspace, replayed one after another
    other = Batch(torch.int8, "paged", 8, 2, [c + n for n, c in zip(new, cached)], new, seed=5)
    runs = []
    for x in (b, other):
        o = torch.empty_like(x.q)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            x.prefill(workspace=ws[:size], out=o)
        runs.append((x, g, o))
    for _ in range(3):
        for x, g, o in runs:
            o.fill_(7.0)
            g.replay()
            x.check(o, half_step=q8_ref.PREFILL)


def test_prefill_captured():
    b = Batch(torch.float8_e4m3fn, "paged", 8, 2, [300, 700], [100, 40])
    b.check(b.prefill(), half_step=q8_ref.PREFILL)
    out = torch.empty_like(b.q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.prefill(max_new=140, out=out)
    for lens, new in (([300, 700], [100, 40]), ([290, 650], [10, 130]), ([140, 0], [140, 0])):
        b.lens, b.new = lens, new
        b.ctx.copy_(torch.tensor(lens, dtype=torch.int32))
        b.cu.copy_(torch.tensor([0, new[0], new[0] + new[1]], dtype=torch.int32))
        g.replay()
        b.check(out, half_step=q8_ref.PREFILL)


def test_prefill_checked():
    b = Batch(torch.int8, "paged", 8, 2, [100, 60], [50, 60])
    pkv.set_checked(True)
    b.check(b.prefill(), half_step=q8_ref.PREFILL)
    assert pkv.get_device_error() == "none"
    b.prefill(max_new=55)
    assert pkv.get_device_error() == "context"
    b.where[0, 2] = 10 ** 6
    b.prefill()
    assert pkv.get_device_error() == "block_id"


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("dtype", q8_ref.FORMATS)
def test_append_and_attend(dtype):
    """Prompts appended and attended as chunks, then decode steps, against the same
    attention over the values that the cache holds."""
    hq, hkv, bs = 8, 2, 16
    bm = pkv.BlockManager(40, bs)
    lens = [37, 5]
    seqs = [bm.add_sequence(n) for n in lens]
    shape = (40, hkv, bs, D)
    k, v = (torch.zeros(shape, device=DEV).to(dtype) for _ in range(2))
    ks, vs = (torch.zeros(40, hkv, bs // 16, device=DEV) for _ in range(2))
    plan = pkv.RopePlan(128)
    g = torch.Generator(device=DEV).manual_seed(8)
    b = Batch.__new__(Batch)
    b.dtype, b.contig, b.hkv, b.bs, b.k, b.v, b.ks, b.vs = dtype, False, hkv, bs, k, v, ks, vs

    def step(new, slots, positions):
        T = sum(new)
        q, kn, vn = (torch.randn(T, n, D, generator=g, device=DEV).bfloat16() for n in (hq, hkv, hkv))
        b.q = pkv.rope_append_q8(torch.tensor(positions, dtype=torch.int32, device=DEV),
                                 torch.tensor(slots, device=DEV), q * 4, kn, vn, k, v, ks, vs, plan)
        tables, ctx = bm.export(seqs, 8)
        b.where, b.ctx = torch.from_numpy(tables).to(DEV), torch.from_numpy(ctx).to(DEV)
        b.lens, b.new, b.top = ctx.tolist(), new, int(ctx.max())
        b.cu = torch.tensor([0] + new, dtype=torch.int32).cumsum(0).to(torch.int32).to(DEV)

    slots, positions = [], []
    for s, n in zip(seqs, lens):
        table = bm.block_table(s)
        slots += [int(table[p // bs]) * bs + p % bs for p in range(n)]
        positions += range(n)
    step(lens, slots, positions)
    b.check(b.prefill(), half_step=q8_ref.PREFILL)
    for _ in range(15):
        at = [bm.length(s) for s in seqs]
        slots, _ = bm.append(seqs)
        step([1, 1], slots.tolist(), at)
        b.check(b.decode())
