"""The 8-bit KV cache: its append as a plain loop, exact, and attention over it
in 64 bits with the bound that the kernels' error has by arithmetic."""
import math

import numpy as np
import torch

QMAX = {torch.int8: np.float32(127), torch.float8_e4m3fn: np.float32(448)}
FORMATS = [torch.int8, torch.float8_e4m3fn]
TINY = np.float32(2.0 ** -100)


def to_codes(y, dtype):
    """fp32 values in units of the scale as codes."""
    y = torch.as_tensor(y)
    if dtype == torch.int8:
        return torch.nan_to_num(y, nan=0.0).round().clamp(-127, 127).to(torch.int8)
    return torch.where(y.isnan(), y, y.clamp(-448, 448)).to(torch.float8_e4m3fn)


def append(cache, scale, slots, x):
    """Rows x [T, Hkv, D] (fp32, CPU) into cache [blocks, Hkv, bs, D] and scale
    [blocks, Hkv, bs / 16], in place, group by group."""
    nb, hkv, bs, D = cache.shape
    qmax = QMAX[cache.dtype]
    groups = {}
    for t, slot in enumerate(slots.tolist()):
        if slot >= 0:
            groups.setdefault(slot // 16, []).append((slot % 16, t))
    for g, rows in groups.items():
        block, part = (16 * g) // bs, (16 * g) % bs // 16
        last = {r: t for r, t in rows}  # a row's last token
        for h in range(hkv):
            old = np.float32(0) if 0 in last else np.float32(scale[block, h, part])
            new = x[list(last.values()), h].numpy()
            size = np.abs(new)
            top = np.max(size[np.isfinite(size)], initial=np.float32(0))
            s = np.maximum(old, top * (np.float32(1) / qmax))
            inv = np.float32(1) / s if s >= TINY else np.float32(0)
            held = cache[block, h, 16 * part:16 * part + 16]
            if 0 in last:
                held.copy_(to_codes(torch.zeros(16, D), cache.dtype))
            elif s != old:
                held.copy_(to_codes(held.float().numpy() * old * inv, cache.dtype))
            for r, t in last.items():
                with np.errstate(invalid="ignore"):
                    held[r] = to_codes(x[t, h].numpy() * inv, cache.dtype)
            scale[block, h, part] = float(s)


def values(cache, scale):
    """What the codes stand for, fp64."""
    return cache.to(torch.float32).double() * scale.double().repeat_interleave(16, 2)[..., None]


# What a probability is rounded to on its way into the product with V, half a step: the
# decode kernels round it to fp16, the prefill kernel rounds it times its group's scale
# to bf16 (whose range holds every scale).  Neither rounds keys or values: a code has at
# most 8 significant bits, which fp16 (11) and bf16 (8) hold exactly.
DECODE, PREFILL = 2.0 ** -11, 2.0 ** -8


def attend64(q, k, v, pos, scale, half_step=DECODE):
    """q [n, Hq, D], k and v [Hkv, c, D] fp64, pos [n] -> (out, tol) [n, Hq, D]."""
    n, hq, D = q.shape
    hkv, c, _ = k.shape
    q, k, v = q.double(), k.repeat_interleave(hq // hkv, 0), v.repeat_interleave(hq // hkv, 0)
    z = torch.einsum("nhd,hcd->hnc", q, k) * scale
    # fp32 dot products of 128 terms (at most 128 roundings of 2^-24 of the sum of
    # sizes, the group's scale and the softmax's factor among them)
    ez = torch.einsum("nhd,hcd->hnc", q.abs(), k.abs()) * (abs(scale) * 2.0 ** -16)
    seen = torch.arange(c, device=q.device) <= torch.as_tensor(pos, device=q.device)[:, None]
    z = z.masked_fill(~seen, -math.inf)
    top = z.amax(-1, keepdim=True)
    w = torch.exp(z - top)
    total = w.sum(-1, keepdim=True)
    small = seen.double() / total  # a probability below fp16's normal range: off by 2^-25
    w = w / total
    out = torch.einsum("hnc,hcd->nhd", w, v)
    size = torch.einsum("hnc,hcd->nhd", w, v.abs())
    err = torch.einsum("hnc,hcd->nhd", w * (2 * ez) + small * 2.0 ** -25, v.abs())
    werr = (w * 2 * ez).sum(-1).transpose(0, 1)[..., None]
    # a probability's rounding, its exponential and the sums (2^-18), and the output's
    # rounding to bf16
    tol = (half_step + 2.0 ** -18) * size + err + werr * size \
        + out.abs() * 2.0 ** -8 + 1e-30
    return out, tol


def assert_close(got, want, tol, what=""):
    g = got.detach().double()
    assert g.shape == want.shape
    assert bool(torch.isfinite(g).all()), "%s: non-finite output" % what
    off = (g - want).abs() - tol
    worst = int(off.argmax())
    assert float(off.max()) <= 0, "%s: element %d got %.6g want %.6g, allowed %.3g off" % (
        what, worst, g.flatten()[worst], want.flatten()[worst], tol.flatten()[worst])


def random_codes(shape, dtype, gen, device):
    x = torch.randn(shape, generator=gen, device=device)
    if dtype == torch.int8:
        return (x * 42).round().clamp(-127, 127).to(torch.int8)
    return (x * 150).clamp(-448, 448).to(torch.float8_e4m3fn)


def random_scales(shape, dtype, gen, device):
    return torch.randn(shape, generator=gen, device=device).mul_(0.7).exp_().mul_(
        3.0 / float(QMAX[dtype]))
