"""Calls over the 8-bit cache whose host bound is below what the device holds: nothing is
written but the rows that the bound covers."""
import pytest
import torch

import paged_kv_cache_245_gb300 as pkv
import q8_ref
from test_gpu_q8_attention import DEV, Batch

pytestmark = pytest.mark.gpu

GUARD = 1 << 20


@pytest.fixture(autouse=True)
def _reset():
    pkv.set_checked(False)
    yield
    pkv.set_checked(False)
    torch.cuda.synchronize()


def run(b, bound, half_step):
    """A call with max_q_tokens `bound`: tokens past it are left alone, the others right."""
    size = pkv.q8_prefill_workspace_size(b.q.shape[0], len(b.new), bound, b.q.shape[1], b.hkv)
    ws = torch.full((size + GUARD,), 0xa5, dtype=torch.uint8, device=DEV)
    out = torch.full_like(b.q, 3.0)
    b.prefill(max_new=bound, out=out, workspace=ws[:size] if size else None)
    assert bool((ws[size:] == 0xa5).all())
    at = 0
    for i, (c, n) in enumerate(zip(b.lens, b.new)):
        k, v = b.rows(i)
        mine, most = out[at:at + n], min(n, bound)
        assert bool((mine[most:] == 3.0).all()), "sequence %d" % i
        want, tol = q8_ref.attend64(b.q[at:at + most], k, v, range(c - n, c - n + most),
                                    128 ** -0.5, half_step)
        q8_ref.assert_close(mine[:most], want, tol, "sequence %d" % i)
        at += n
    return size


@pytest.mark.parametrize("dtype", q8_ref.FORMATS)
@pytest.mark.parametrize("layout", ["paged", "contig"])
@pytest.mark.parametrize("new,cached,bound", [
    ([64, 10, 3], [2000, 500, 0], 10),   # items cut by key tiles: records of 40 rows
    ([64], [3000], 1), ([200, 70], [1000, 0], 33), ([300, 64], [900, 40], 64),
    ([33, 32, 31], [700, 0, 64], 32)])
def test_chunk_past_the_bound_in_pieces(dtype, layout, new, cached, bound):
    b = Batch(dtype, layout, 8, 2, [n + c for n, c in zip(new, cached)], new)
    assert run(b, bound, q8_ref.PREFILL) > 0


@pytest.mark.parametrize("heads", [(8, 2), (14, 2)])
def test_chunk_past_the_bound_of_whole_items(heads):
    new = [70] * 600
    new[17], new[599] = 150, 200
    b = Batch(torch.int8, "paged", *heads, [n + 20 for n in new], new, bs=32)
    assert run(b, 70, q8_ref.PREFILL) == 0


def test_chunk_past_the_bound_of_sorted_items():
    new = [300] * 160
    new[3], new[159] = 400, 700
    b = Batch(torch.float8_e4m3fn, "paged", 8, 2, [n + 20 for n in new], new, bs=32)
    assert run(b, 300, q8_ref.PREFILL) == 0


@pytest.mark.parametrize("dtype", q8_ref.FORMATS)
@pytest.mark.parametrize("layout", ["paged", "contig"])
@pytest.mark.parametrize("bound", [1, 3, 4, 6, 8])
def test_short_chunk_past_the_bound(dtype, layout, bound):
    new = [min(n, bound) for n in (1, 2, 3, 4) * 8]
    new[5], new[30] = bound + 1, 40
    b = Batch(dtype, layout, 16, 4, [n + 30 * i for i, n in enumerate(new)], new)
    run(b, bound, q8_ref.PREFILL)


def test_checked_leaves_the_chunk():
    b = Batch(torch.int8, "paged", 8, 2, [2064, 510], [64, 10])
    pkv.set_checked(True)
    out = torch.full_like(b.q, 3.0)
    b.prefill(max_new=10, out=out)
    assert pkv.get_device_error() == "context"
    assert bool((out[:64] == 3.0).all()) and bool((out[64:] != 3.0).any())
