"""Attention over the 8-bit cache gives the same bits on every call: no operand is taken
before it has landed or overwritten before it was read."""
import pytest
import torch

import q8_ref
from test_gpu_q8_attention import Batch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", q8_ref.FORMATS)
@pytest.mark.parametrize("layout", ["paged", "contig"])
@pytest.mark.parametrize("heads,new,cached,times", [
    ((8, 2), [300] * 40, [10] * 40, 300),             # masked tiles, cut items
    ((8, 2), [129] * 120, [127] * 120, 300),          # one whole tile, one with a row in it
    ((32, 8), [2048] * 8, [0] * 8, 40),               # whole items
    ((56, 8), [100, 1500, 700, 333, 1000, 64], [3000, 0, 128, 77, 2000, 1], 60),
    ((14, 2), [18] * 200, list(range(200)), 200)])    # items of one row tile
def test_prefill_repeats(dtype, layout, heads, new, cached, times):
    b = Batch(dtype, layout, *heads, [n + c for n, c in zip(new, cached)], new, bs=32)
    first = b.prefill().clone()
    if sum(new) < 16000:
        b.check(first, half_step=q8_ref.PREFILL)
    for i in range(times):
        assert torch.equal(b.prefill(), first), "call %d" % i
