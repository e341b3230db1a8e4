"""What the 8-bit cache's calls refuse, and the plain append's own values."""
import ctypes

import numpy as np
import pytest
import torch

import q8_ref
from paged_kv_cache_245_gb300 import binding
from paged_kv_cache_245_gb300.build import build

FAKE = 0x10000  # aligned, never dereferenced: every call here fails before a launch
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3


@pytest.fixture(scope="module")
def L():
    build()
    return binding.lib()


def cache(**over):
    c = dict(k=FAKE, v=FAKE, k_scale=FAKE, v_scale=FAKE, format=1, reserved=0)
    c.update(over)
    return binding.Q8Cache(*(c[n] for n, _ in binding.Q8Cache._fields_))


H = binding.Heads(8, 2, 128)

BAD_CACHES = [(dict(k=None), INVALID), (dict(v_scale=None), INVALID), (dict(v=FAKE + 8), INVALID),
              (dict(k_scale=FAKE + 2), INVALID), (dict(format=0), INVALID), (dict(format=3), INVALID)]


def append(L, slots=FAKE, n=1, k=FAKE, ks=256, v=FAKE, vs=256, c=None, num_slots=64, bs=16, h=H):
    return L.pkv_kv_append_q8(slots, n, k, ks, v, vs, cache() if c is None else c, num_slots, bs, h,
                              None)


@pytest.mark.parametrize("over,code", BAD_CACHES)
def test_bad_caches(L, over, code):
    bad = cache(**over)
    assert append(L, c=bad) == code
    assert decode(L, c=bad) == code
    assert prefill(L, c=bad) == code
    assert L.pkv_last_error()


@pytest.mark.parametrize("over,code", [
    (dict(n=-1), INVALID), (dict(num_slots=-1), INVALID), (dict(n=2 ** 30 + 1), UNSUPPORTED),
    (dict(slots=None), INVALID), (dict(slots=FAKE + 4), INVALID), (dict(k=None), INVALID),
    (dict(v=FAKE + 8), INVALID), (dict(ks=4), INVALID), (dict(vs=-8), INVALID),
    (dict(bs=0), INVALID), (dict(bs=24), UNSUPPORTED), (dict(bs=8), UNSUPPORTED),
    (dict(h=binding.Heads(8, 2, 64)), UNSUPPORTED), (dict(h=binding.Heads(8, 0, 128)), INVALID)])
def test_append_refuses(L, over, code):
    assert append(L, **over) == code


def test_nothing_to_do(L):
    assert append(L, n=0, slots=None, k=None, v=None) == 0
    assert decode(L, B=0) == 0
    assert prefill(L, B=0) == 0
    assert prefill(L, T=0) == 0
    assert prefill(L, max_q=0) == 0


@pytest.mark.parametrize("over,code", [
    (dict(pos=None), INVALID), (dict(pos=FAKE + 2), INVALID), (dict(q=None), INVALID),
    (dict(qs=4), INVALID), (dict(out=None), INVALID), (dict(out=FAKE + 4096 + 256), INVALID),
    (dict(out=2 * FAKE), INVALID), (dict(rope=None), INVALID),
    (dict(h=binding.Heads(18, 2, 128)), UNSUPPORTED)])
def test_rope_append_refuses(L, over, code):
    plan = binding.Rope()
    assert L.pkv_rope_init(ctypes.byref(plan), 128, 0, 10000.0, None) == 0
    a = dict(pos=FAKE, q=FAKE + 4096, qs=1024, k=2 * FAKE, v=3 * FAKE, out=4 * FAKE, rope=plan, h=H)
    a.update(over)
    assert L.pkv_rope_append_q8(a["pos"], FAKE, 4, a["q"], a["qs"], a["k"], 256, a["v"], 256,
                                a["out"], cache(), 64, 16, a["h"], a["rope"], None) == code


def decode(L, q=FAKE, c=None, tables=FAKE, maxb=4, nb=8, ctx=FAKE, B=2, top=64, bs=16, scale=0.1,
           h=H, out=FAKE):
    return L.pkv_paged_decode_attention_q8(q, cache() if c is None else c, tables, maxb, nb, ctx, B,
                                           top, bs, scale, h, out, None, 0, None)


def prefill(L, q=FAKE, cu=FAKE, T=4, c=None, tables=FAKE, maxb=4, nb=8, ctx=FAKE, B=2, max_q=2,
            bs=16, scale=0.1, h=H, out=FAKE):
    return L.pkv_paged_prefill_attention_q8(q, cu, T, cache() if c is None else c, tables, maxb, nb,
                                            ctx, B, max_q, bs, scale, h, out, None, 0, None)


COMMON = [(dict(q=None), INVALID), (dict(q=FAKE + 8), INVALID), (dict(tables=None), INVALID),
          (dict(tables=FAKE + 2), INVALID), (dict(ctx=None), INVALID), (dict(ctx=FAKE + 1), INVALID),
          (dict(out=None), INVALID), (dict(out=FAKE + 4), INVALID), (dict(B=-1), INVALID),
          (dict(B=65536), UNSUPPORTED), (dict(scale=float("nan")), INVALID),
          (dict(scale=float("inf")), INVALID), (dict(bs=24), UNSUPPORTED), (dict(bs=0), INVALID),
          (dict(maxb=0), INVALID), (dict(nb=0), INVALID),
          (dict(nb=2 ** 31 - 1, bs=2 ** 20, maxb=1), UNSUPPORTED),
          (dict(h=binding.Heads(9, 1, 128)), UNSUPPORTED), (dict(h=binding.Heads(8, 3, 128)), INVALID),
          (dict(h=binding.Heads(8, 2, 64)), UNSUPPORTED)]


@pytest.mark.parametrize("over,code", COMMON + [(dict(top=65), INVALID), (dict(top=-1), INVALID)])
def test_decode_refuses(L, over, code):
    assert decode(L, **over) == code


@pytest.mark.parametrize("over,code", COMMON + [
    (dict(cu=None), INVALID), (dict(cu=FAKE + 2), INVALID), (dict(T=-1), INVALID),
    (dict(max_q=-1), INVALID), (dict(maxb=2 ** 28), UNSUPPORTED)])
def test_prefill_refuses(L, over, code):
    assert prefill(L, **over) == code


def test_append_refuses_too_many_tokens(L):
    """Each CTA passes over all of a call's slots."""
    assert L.pkv_kv_append_q8(FAKE, 2 ** 22 + 1, 2 * FAKE, 256, 3 * FAKE, 256, cache(), 64, 16, H,
                              None) == UNSUPPORTED


def test_contig_refuses(L):
    c = cache()
    assert L.pkv_contig_decode_attention_q8(FAKE, c, FAKE, 4, FAKE, 2, 65, 64, 0.1, H, FAKE, None, 0,
                                            None) == INVALID
    assert L.pkv_contig_decode_attention_q8(FAKE, c, FAKE, 4, FAKE, 2, 30, 40, 0.1, H, FAKE, None, 0,
                                            None) == UNSUPPORTED
    assert L.pkv_contig_prefill_attention_q8(FAKE, FAKE, 4, c, FAKE, 0, FAKE, 2, 2, 64, 0.1, H, FAKE,
                                             None, 0, None) == INVALID
    assert L.pkv_contig_prefill_attention_q8(FAKE, FAKE, 4, c, FAKE, 4, FAKE, 2, 2, 2 ** 31, 0.1, H,
                                             FAKE, None, 0, None) == UNSUPPORTED


def test_binding_refuses():
    x = torch.zeros(1, 2, 16, 128)
    with pytest.raises(TypeError):
        binding._q8_cache(0, x, x, x, x)
    with pytest.raises(TypeError):
        binding._q8_cache(0, x.to(torch.int8), x.to(torch.int8), x, x)
    with pytest.raises(TypeError):
        binding.kv_append_q8(torch.zeros(1), x, x, x, x, x, x)


@pytest.mark.parametrize("dtype", q8_ref.FORMATS)
def test_plain_append(dtype):
    """Each value within half a step of what was appended; a smaller row leaves the rest."""
    c, s = torch.zeros(2, 1, 16, 128).to(dtype), torch.zeros(2, 1, 1)
    x = torch.randn(12, 1, 128, generator=torch.Generator().manual_seed(2))
    q8_ref.append(c, s, torch.arange(12), x)
    assert float(s[0, 0, 0]) == float(x.abs().max().numpy() * (np.float32(1) / q8_ref.QMAX[dtype]))
    got = q8_ref.values(c, s)[0, 0, :12]
    want = x[:, 0].double()
    step = float(s[0, 0, 0])
    half = step / 2 if dtype == torch.int8 else torch.maximum(want.abs() / 16,
                                                              torch.tensor(step / 1024))
    assert bool(((got - want).abs() <= half * (1 + 1e-6)).all())
    before = c.clone()
    q8_ref.append(c, s, torch.tensor([12]), x[:1] * 0.01)
    assert torch.equal(c.view(torch.int8)[0, 0, :12], before.view(torch.int8)[0, 0, :12])
    q8_ref.append(c, s, torch.tensor([13]), x[:1] * 100)
    assert float(q8_ref.values(c, s)[0, 0, 5].abs().max()) < 5
