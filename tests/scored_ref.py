"""Attention with capped, biased and masked scores in 64 bits, with the bound
that a bf16 / fp32 kernel's error has by arithmetic."""
import math

import torch


def visible(pos, first, window, prefix, ctx):
    """(first key, last key) that a token at `pos` sees; none if first > last."""
    lo = max(first, 0)
    if window:
        lo = max(lo, pos - window + 1)
    return lo, min(max(pos, min(prefix, ctx) - 1), ctx - 1)


def attend64(q, k, v, pos, rng, scale, softcap=0.0, slopes=None):
    """q [n, Hq, D], k and v [Hkv, c, D], pos [n], rng [(lo, hi)] * n ->
    (out [n, Hq, D], tol [n, Hq, D]), fp64."""
    n, hq, D = q.shape
    hkv, c, _ = k.shape
    G = hq // hkv
    dev = q.device
    q, k, v = q.double(), k.double(), v.double()
    k, v = k.repeat_interleave(G, 0), v.repeat_interleave(G, 0)
    z = torch.einsum("nhd,hcd->hnc", q, k) * scale
    # fp32 dot products of 128 terms: at most 128 roundings of 2^-24 of the sum of sizes
    ez = torch.einsum("nhd,hcd->hnc", q.abs(), k.abs()) * (abs(scale) * 2.0 ** -17)
    if softcap:
        z = softcap * torch.tanh(z / softcap)  # slope at most 1: the error does not grow
        ez = ez + z.abs() * 2.0 ** -16         # the tanh's own: 2^-17 relative, and its products
    p = torch.as_tensor(pos, device=dev)
    key = torch.arange(c, device=dev)
    if slopes is not None:
        b = slopes.double()[:, None, None] * (p[:, None] - key).abs()
        z = z - b
        ez = ez + (b.abs() + z.abs()) * 2.0 ** -22  # a product, a sum, log2 e
    r = torch.as_tensor(rng, device=dev)
    seen = (key >= r[:, :1]) & (key <= r[:, 1:])
    z = z.masked_fill(~seen, -math.inf)
    top = z.amax(-1, keepdim=True)
    w = torch.exp(z - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = w.sum(-1, keepdim=True)
    w = w / torch.where(total == 0, torch.ones_like(total), total)
    out = torch.einsum("hnc,hcd->nhd", w, v)
    # every probability: rounded to bf16 once (2^-8), exp2 and the score's error
    # (twice: numerator and sum); the output rounded to bf16 once more
    size = torch.einsum("hnc,hcd->nhd", w, v.abs())
    err = torch.einsum("hnc,hcd->nhd", w * (2 * ez), v.abs())
    werr = (w * 2 * ez).sum(-1).transpose(0, 1)[..., None]
    tol = (2.0 ** -8 + 2.0 ** -18) * size + err + werr * size + out.abs() * 2.0 ** -8 + 1e-30
    return out, tol


def assert_close(got, want, tol, what=""):
    g = got.detach().double()
    assert g.shape == want.shape
    assert bool(torch.isfinite(g).all()), "%s: non-finite output" % what
    off = (g - want).abs() - tol
    worst = int(off.argmax())
    assert float(off.max()) <= 0, "%s: element %d got %.6g want %.6g, allowed %.3g off" % (
        what, worst, float(g.flatten()[worst]), float(want.flatten()[worst]),
        float(tol.flatten()[worst]))


class Sequences:
    """Seeded caches of a batch, paged or contiguous, with every position that
    no token sees (and every unused row) holding NaN or infinities if poison."""

    def __init__(self, ctx, hkv, bs, contig=False, seed=1, dev="cuda:0", spare=3, D=128):
        self.ctx, self.hkv, self.bs, self.contig, self.dev = list(ctx), hkv, bs, contig, dev
        g = torch.Generator(device=dev).manual_seed(seed)
        self.g = g
        B, top = len(self.ctx), max(max(self.ctx), 1)
        if contig:
            self.S = (top + 15) // 16 * 16 + 16
            shape = (B + 1, hkv, self.S, D)
            self.where = torch.randperm(B + 1, generator=g, device=dev)[:B].to(torch.int32)
        else:
            need = [(c + bs - 1) // bs for c in self.ctx]
            self.nb = sum(need) + spare
            shape = (self.nb, hkv, bs, D)
            pool = torch.randperm(self.nb, generator=g, device=dev).to(torch.int32)
            # entries past a sequence's blocks: the last spare block
            self.where = torch.full((B, max(max(need), 1)), int(pool[-1]), dtype=torch.int32,
                                    device=dev)
            at = 0
            for i, n in enumerate(need):
                self.where[i, :n] = pool[at:at + n]
                at += n
            self.spare = pool[at:]
        self.k = torch.randn(shape, generator=g, device=dev).bfloat16()
        self.v = torch.randn(shape, generator=g, device=dev).bfloat16()
        self.ctx_t = torch.tensor(self.ctx, dtype=torch.int32, device=dev)

    def rows(self, i, x):
        """[Hkv, ctx, D] of sequence i (a copy)."""
        c = self.ctx[i]
        if self.contig:
            return x[int(self.where[i]), :, :c].clone()
        n = (c + self.bs - 1) // self.bs
        return x[self.where[i, :n].long()].transpose(0, 1).reshape(self.hkv, -1, x.shape[-1])[:, :c]

    def poison(self, keep):
        """NaN and infinities in every cache row but those keep[i] = (lo, hi) of
        sequence i; returns the poisoned (k, v)."""
        mask = torch.zeros(self.k.shape[0], self.k.shape[2], dtype=torch.bool, device=self.dev)
        for i, (lo, hi) in enumerate(keep):
            for j in range(max(lo, 0), hi + 1):
                if self.contig:
                    mask[int(self.where[i]), j] = True
                else:
                    mask[int(self.where[i, j // self.bs]), j % self.bs] = True
        bad = torch.tensor([float("nan"), float("inf"), -float("inf")], device=self.dev).bfloat16()
        fill = bad[torch.arange(self.k.shape[2], device=self.dev) % 3][None, None, :, None]
        m = mask[:, None, :, None]
        return (torch.where(m, self.k, fill).contiguous(),
                torch.where(m, self.v, fill.roll(1, 2)).contiguous())
