"""Scored attention captured once and replayed over other lengths, contexts and
masks in the same arrays; several streams at once; rows of odd length."""
import numpy as np
import pytest
import torch

import paged_kv_cache_245_gb300 as pkv
from scored_ref import Sequences, assert_close, attend64
from test_gpu_scored_decode import call, queries, reference
from test_gpu_scored_prefill import Chunks

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
D = 128
SCALE = D ** -0.5
VARIANTS = [pkv.VARIANT_AUTO, pkv.VARIANT_SPLIT, pkv.VARIANT_TC_8X3, pkv.VARIANT_TC_12X2]


@pytest.fixture(autouse=True)
def _reset():
    yield
    pkv.set_decode_variant(pkv.VARIANT_AUTO)
    torch.cuda.synchronize()


def close(got, want, tol):
    """The sum takes the rounded probabilities p (1 + d), |d| <= 2^-8: out is off by
    sum w d (v - out), so the bound has |out| 2^-8 for it beside the output's rounding."""
    assert_close(got, want, tol + want.abs() * 2.0 ** -8)


def captured(run):
    run()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        run()
    return graph


def test_a_captured_prefill_takes_other_lengths_and_masks():
    s = Chunks([0, 300, 20, 0], [400, 70, 1, 129], 32, 8, 16, seed=5)
    first = torch.zeros(s.T, dtype=torch.int32, device=DEV)
    prefix = torch.zeros(4, dtype=torch.int32, device=DEV)
    out = torch.zeros_like(s.q)
    graph = captured(lambda: pkv.paged_prefill_attention_scored(
        s.q, s.cu, s.k, s.v, s.where, s.ctx_t, 600, SCALE, softcap=30.0, window=500,
        first_key=first, prefix_lens=prefix, out=out))
    for new in ([400, 70, 1, 129], [129, 71, 0, 129], [0, 0, 0, 0], [1, 1, 1, 1], [100, 100, 20, 129]):
        s.new, s.T = new, sum(new)
        s.cu.copy_(torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32))
        out.fill_(7.0)
        graph.replay()
        if s.T:
            close(out[:s.T], *s.reference(window=500, first=first[:s.T], prefix=prefix, softcap=30.0))
        assert bool((out[s.T:] == 7.0).all())
        prefix.copy_(torch.tensor([5, 900, 0, 60], dtype=torch.int32))
        first[:50] = torch.arange(50, device=DEV, dtype=torch.int32)


@pytest.mark.parametrize("variant", VARIANTS)
def test_a_captured_decode_takes_other_contexts(variant):
    pkv.set_decode_variant(variant)
    s = Sequences([900, 31, 400, 65] * 3, 8, 16, seed=18)
    q = queries(s, 32)
    first = torch.zeros(12, dtype=torch.int32, device=DEV)
    out = torch.empty_like(q)
    graph = captured(lambda: call(s, q, softcap=20.0, first_key=first, out=out))
    base = list(s.ctx)
    for k in range(4):
        s.ctx = [max(0, c - 37 * k * (i % 3)) for i, c in enumerate(base)]
        s.ctx_t.copy_(torch.tensor(s.ctx, dtype=torch.int32))
        first.copy_(torch.tensor([c // (k + 1) if k else 0 for c in s.ctx], dtype=torch.int32))
        graph.replay()
        close(out, *reference(s, q, first=first, softcap=20.0))


@pytest.mark.parametrize("variant", VARIANTS)
@pytest.mark.parametrize("S", [1007, 333, 17, 1])
def test_request_rows_of_odd_length(variant, S):
    """Tiles reach past a request's rows, where NaN stands."""
    pkv.set_decode_variant(variant)
    g = torch.Generator(device=DEV).manual_seed(S)
    k = torch.full((4, 2, S, D), float("nan"), device=DEV).bfloat16()
    v = k.clone()
    ids, ctx = [2, 0, 3], [S, max(1, S - 5), 1]
    for i, c in zip(ids, ctx):
        k[i, :, :c], v[i, :, :c] = (torch.randn(2, c, D, generator=g, device=DEV).bfloat16()
                                  for _ in "kv")
    q = torch.randn(3, 8, D, generator=g, device=DEV).bfloat16()
    got = pkv.contig_decode_attention_scored(
        q, k, v, torch.tensor(ids, dtype=torch.int32, device=DEV),
        torch.tensor(ctx, dtype=torch.int32, device=DEV), S, SCALE, softcap=9.0, window=300)
    for r, (i, c) in enumerate(zip(ids, ctx)):
        close(got[r:r + 1], *attend64(q[r:r + 1], k[i, :, :c], v[i, :, :c], [c - 1],
                                      [(max(0, c - 300), c - 1)], SCALE, 9.0))


def test_three_streams_at_once():
    s = Sequences([3000, 100] * 10, 8, 16, seed=3)
    q = queries(s, 32)
    want = call(s, q, softcap=30.0)
    streams = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(10):
        outs = []
        for x in streams:
            x.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(x):
                outs.append(call(s, q, softcap=30.0))
        for x in streams:
            torch.cuda.current_stream().wait_stream(x)
        assert all(torch.equal(o, want) for o in outs)
