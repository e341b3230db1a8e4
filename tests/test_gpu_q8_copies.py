"""Block copies and swaps of an 8-bit cache's scales, of any number of heads: blocks of
4 bytes and more, pools that begin anywhere."""
import pytest
import torch

import paged_kv_cache_245_gb300 as pkv
import q8_ref
from test_gpu_q8_attention import DEV, Batch

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _reset():
    pkv.set_checked(False)
    yield
    pkv.set_checked(False)
    torch.cuda.synchronize()


def pool(blocks, hkv, per, first=0, device=DEV):
    """Scales [blocks, hkv, per] that begin `first` words after an aligned address."""
    flat = torch.randn(first + blocks * hkv * per + 7, device=device)
    return flat, flat[first:first + blocks * hkv * per].view(blocks, hkv, per)


SHAPES = [(1, 1), (2, 1), (3, 1), (4, 1), (6, 1), (1, 3), (2, 8), (8, 8), (5, 70), (16, 1000)]


@pytest.mark.parametrize("hkv,per", SHAPES)
@pytest.mark.parametrize("first", [0, 1])
@pytest.mark.parametrize("layers", [1, 67])
def test_copy(hkv, per, first, layers):
    if layers > 1 and hkv * per > 1000:
        layers = 2
    sides = [[pool(9, hkv, per, first if i == layers - 1 else 0) for i in range(layers)]
             for _ in range(2)]
    pairs = torch.tensor([[0, 8], [3, 1], [5, 4]], device=DEV)
    wants = [[flat.clone() for flat, _ in side] for side in sides]
    for side, want in zip(sides, wants):
        for (flat, x), w in zip(side, want):
            off = x.storage_offset()
            y = w[off:off + x.numel()].view(x.shape)
            for src, dst in pairs.tolist():
                y[dst] = y[src].clone()
    pkv.block_copy(pairs, [x for _, x in sides[0]], [x for _, x in sides[1]])
    for side, want in zip(sides, wants):
        for (flat, _), w in zip(side, want):
            assert torch.equal(flat, w)  # (what stands around the pool too)


@pytest.mark.parametrize("hkv,per", SHAPES)
@pytest.mark.parametrize("first", [0, 3])
def test_swap(hkv, per, first):
    dev = [pool(9, hkv, per, first) for _ in range(2)]
    host = [torch.zeros(6, hkv, per).pin_memory() for _ in range(2)]
    was = [flat.clone() for flat, _ in dev]
    out = torch.tensor([[2, 5], [7, 0]], device=DEV)
    pkv.block_swap(out, [dev[0][1]], [dev[1][1]], [host[0]], [host[1]])
    torch.cuda.synchronize()
    for (flat, x), h in zip(dev, host):
        for src, dst in out.tolist():
            assert torch.equal(h[dst], x[src].cpu())
        assert bool((h[[1, 2, 3, 4]] == 0).all())
    back = torch.tensor([[5, 1], [0, 4]]).pin_memory()
    pkv.block_swap(back, [host[0]], [host[1]], [dev[0][1]], [dev[1][1]])
    torch.cuda.synchronize()
    for (flat, x), w in zip(dev, was):
        y = w[first:first + x.numel()].view(x.shape)
        y[1], y[4] = y[2].clone(), y[7].clone()
        assert torch.equal(flat, w)


def test_checked():
    (flat, x), (_, y) = pool(4, 3, 1), pool(4, 3, 1)
    was = x.clone()
    pkv.set_checked(True)
    pkv.block_copy(torch.tensor([[0, 4], [-1, 2], [1, 3]], device=DEV), [x], [y])
    assert pkv.get_device_error() == "copy_pair"
    was[3] = was[1].clone()
    assert torch.equal(x, was)


@pytest.mark.parametrize("dtype", q8_ref.FORMATS)
@pytest.mark.parametrize("hkv", [1, 2, 3])
def test_shared_block_is_copied(dtype, hkv):
    """A sequence whose tail block is copied attends as the one that it came from."""
    b = Batch(dtype, "paged", 4 * hkv, hkv, [40])
    want = b.decode().clone()
    free = next(i for i in range(b.k.shape[0]) if i not in b.blocks(0))
    tail = int(b.where[0, 2])
    pairs = torch.tensor([[tail, free]], device=DEV)
    pkv.block_copy(pairs, [b.k], [b.v])
    pkv.block_copy(pairs, [b.ks], [b.vs])
    b.where[0, 2] = free
    for x in (b.k.view(torch.int8), b.v.view(torch.int8)):
        x[tail] = 0
    assert torch.equal(b.decode(), want)
