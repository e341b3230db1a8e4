"""Prefill under a max_q_tokens far above any chunk, up to the largest int32."""
import pytest
import torch

import paged_kv_cache_245_gb300 as pkv
from test_gpu_scored_prefill import Chunks

pytestmark = pytest.mark.gpu

SCALE = 128 ** -0.5


@pytest.mark.parametrize("hq,hkv", [(8, 2), (2, 2), (7, 1)])
@pytest.mark.parametrize("bound", [301, 5000, 2 ** 20, 2 ** 28, 2 ** 29, 2 ** 31 - 1])
@pytest.mark.parametrize("contig", [False, True])
def test_a_generous_bound_changes_nothing(hq, hkv, bound, contig):
    s = Chunks([0, 300], [200, 101], hq, hkv, 16, contig, seed=71)
    for kw in (None, dict(), dict(softcap=30.0, window=50)):
        if kw is None:
            f = pkv.contig_prefill_attention if contig else pkv.paged_prefill_attention
        else:
            f = (pkv.contig_prefill_attention_scored if contig
                 else pkv.paged_prefill_attention_scored)
        args = (s.q, s.cu, s.k, s.v, s.where, s.ctx_t)
        want = f(*args, 200, SCALE, **(kw or {}))
        out = torch.full_like(s.q, 7.0)
        f(*args, bound, SCALE, out=out, **(kw or {}))
        # (other key splits may round differently: the largest value is under 8)
        assert float((out.float() - want.float()).abs().max()) <= 2.0 ** -5
        pkv.set_checked(True)
        f(*args, bound, SCALE, out=out, **(kw or {}))
        error = pkv.get_device_error()
        pkv.set_checked(False)
        assert error == "none"
