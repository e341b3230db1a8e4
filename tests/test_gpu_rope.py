"""Rotary append (pkv_rope_append) against the formula in 64 bits: layouts,
parts of heads, far positions, strides, padding, in place, captured, the
contiguous layout, checked mode."""
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_245_gb300 as pkv

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
D = 128


@pytest.fixture(autouse=True)
def _reset():
    pkv.set_checked(False)
    yield
    pkv.set_checked(False)
    torch.cuda.synchronize()


def radians(plan):
    return np.array([int(x) for x in plan.c.turn[:plan.c.rotary_dim // 2]],
                    dtype=object) / 2 ** 64 * (2 * math.pi)


def turned(x, pos, plan):
    """(value, bound of its error) in 64 bits of x [T, H, D] (fp64)."""
    rd, half = plan.c.rotary_dim, plan.c.rotary_dim // 2
    # the fraction of a turn in exact integers, for any position
    turn = [int(t) for t in plan.c.turn[:half]]
    frac = np.array([[((int(p) * t) % 2 ** 64) / 2 ** 64 for t in turn] for p in pos])
    c, s = (f(2 * math.pi * frac)[:, None] * float(plan.c.gain) for f in (np.cos, np.sin))
    even, odd = (slice(0, rd, 2), slice(1, rd, 2)) if plan.c.interleaved else (
        slice(0, half), slice(half, rd))
    y, tol = x.copy(), np.zeros_like(x)
    a, b = x[..., even], x[..., odd]
    y[..., even], y[..., odd] = a * c - b * s, b * c + a * s
    # one rounding to bf16 (2^-8), and in fp32: the angle (a fraction of a turn
    # rounded to 2^-25 of it: 2 pi 2^-25), sine and cosine (2 steps), times
    # gain, two products and a sum: under 2^-20 of |a| + |b|
    size = (np.abs(a) + np.abs(b)) * abs(float(plan.c.gain)) * 2.0 ** -20
    tol[..., even] = tol[..., odd] = size
    return y, tol + np.where(tol > 0, np.abs(y) * 2.0 ** -8, 0.0)


def host(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def check(got, x, pos, plan):
    want, tol = turned(host(x), pos, plan)
    off = np.abs(host(got) - want)
    assert np.all(off <= tol), (np.max(off - tol), np.argmax(off - tol))


def inputs(T, hq, hkv, bs, seed, far=1 << 20, fused=True):
    g = torch.Generator(device=DEV).manual_seed(seed)
    qkv = torch.randn(T, (hq + 2 * hkv) * D, generator=g, device=DEV).bfloat16()
    q, k, v = (x.unflatten(1, (-1, D)) for x in qkv.split([hq * D, hkv * D, hkv * D], 1))
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    nb = (T + bs - 1) // bs + 2
    kc, vc = (torch.randn(nb, hkv, bs, D, generator=g, device=DEV).bfloat16() for _ in "kv")
    slots = torch.randperm(nb * bs, generator=g, device=DEV)[:T].contiguous()
    pos = torch.randint(0, far, (T,), generator=g, device=DEV, dtype=torch.int32)
    return q, k, v, kc, vc, slots, pos


def flat(c):
    """Cache rows by slot: [slots, Hkv, D]."""
    return c.transpose(1, 2).reshape(-1, c.shape[1], D)


def run_and_check(q, k, v, kc, vc, slots, pos, plan, **kw):
    k0, v0 = flat(kc).clone(), flat(vc).clone()
    q0, kept = q.clone(), slots >= 0
    out = pkv.rope_append(pos, slots, q, k, v, kc, vc, plan, **kw)
    check(out, q0, pos.tolist(), plan)
    rows = slots[kept]
    check(flat(kc)[rows], k[kept], pos[kept].tolist(), plan)
    v0[rows] = v[kept]
    assert torch.equal(flat(vc).view(torch.int16), v0.view(torch.int16))
    rest = torch.ones(k0.shape[0], dtype=torch.bool, device=DEV)
    rest[rows] = False
    assert torch.equal(flat(kc)[rest], k0[rest])  # no other row was touched
    return out


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rd", [2, 16, 30, 50, 64, 96, 126, 128])
@pytest.mark.parametrize("T,hq,hkv,bs", [(1, 32, 8, 16), (37, 56, 8, 48), (515, 6, 1, 16),
                                         (2051, 4, 2, 16)])
def test_layouts_and_parts_of_heads(rd, interleaved, T, hq, hkv, bs):
    plan = pkv.RopePlan(rd, theta=5e5, interleaved=interleaved)
    run_and_check(*inputs(T, hq, hkv, bs, seed=rd + T), plan)


@pytest.mark.parametrize("scaling", [
    {"kind": "linear", "factor": 4}, {"kind": "base", "factor": 3},
    {"kind": "parts", "factor": 16, "original": 4096},
    {"kind": "smooth", "factor": 8, "original": 8192}])
def test_scalings(scaling):
    run_and_check(*inputs(70, 8, 2, 16, seed=5), pkv.RopePlan(128, theta=1e4, scaling=scaling))


def test_elements_past_the_rotated_part_are_the_same_bits():
    q, k, v, kc, vc, slots, pos = inputs(33, 8, 2, 16, seed=6)
    q[..., 64:] = float("nan")
    k[..., 65] = float("inf")
    for inter in (False, True):
        out = pkv.rope_append(pos, slots, q, k, v, kc, vc, pkv.RopePlan(64, interleaved=inter))
        assert torch.equal(out[..., 64:].view(torch.int16), q[..., 64:].contiguous().view(torch.int16))
        assert bool(torch.isfinite(out[..., :64]).all())
        assert torch.equal(flat(kc)[slots][..., 64:], k[..., 64:])


@pytest.mark.parametrize("rd,inter", [(128, False), (50, False), (64, True)])
def test_far_negative_and_extreme_positions(rd, inter):
    q, k, v, kc, vc, slots, _ = inputs(8, 8, 2, 16, seed=7)
    pos = torch.tensor([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 10 ** 9, 2 ** 24 + 1, 2 ** 30],
                       dtype=torch.int32, device=DEV)
    run_and_check(q, k, v, kc, vc, slots, pos, pkv.RopePlan(rd, interleaved=inter))


def test_position_zero_turns_nothing():
    q, k, v, kc, vc, slots, pos = inputs(5, 8, 2, 16, seed=8)
    out = pkv.rope_append(torch.zeros_like(pos), slots, q, k, v, kc, vc, pkv.RopePlan(128))
    assert torch.equal(out, q) and torch.equal(flat(kc)[slots], k)


def test_scores_depend_on_distance_only():
    """The point of rotary positions: q_p . k_j is a function of p - j."""
    q, k, v, kc, vc, slots, _ = inputs(2, 1, 1, 16, seed=9)
    q, k = q[:1].expand(2, -1, -1), k[:1].expand(2, -1, -1)  # token stride 0
    plan = pkv.RopePlan(128, theta=5e5)
    scores = []
    for at in (0, 1000, 500000):
        p = torch.tensor([at + 7, at], dtype=torch.int32, device=DEV)
        out = pkv.rope_append(p, slots, q, k, v, kc, vc, plan)
        scores.append(float(host(out[0, 0]) @ host(flat(kc)[slots[1]][0])))
    n = float(np.linalg.norm(host(q[0, 0])) * np.linalg.norm(host(k[0, 0])))
    # both sides rounded to bf16 once: 2 * 2^-8 of the norms' product at most
    assert max(scores) - min(scores) <= 2 * 2 * 2.0 ** -8 * n


@pytest.mark.parametrize("rd", [128, 50])
def test_padding_tokens(rd):
    q, k, v, kc, vc, slots, pos = inputs(20, 32, 8, 16, seed=10)
    slots[3] = -1
    slots[15:] = -7
    run_and_check(q, k, v, kc, vc, slots, pos, pkv.RopePlan(rd))


@pytest.mark.parametrize("rd,inter", [(128, False), (96, False), (50, False), (50, True)])
@pytest.mark.parametrize("T", [3, 600, 2301])
def test_in_place(rd, inter, T):
    q, k, v, kc, vc, slots, pos = inputs(T, 32, 8, 16, seed=11, fused=False)
    out = run_and_check(q, k, v, kc, vc, slots, pos, pkv.RopePlan(rd, interleaved=inter), out=q)
    assert out.data_ptr() == q.data_ptr()


def test_contiguous_layout_and_out():
    """block_size = S, slot = reqId * S + position; a caller's out tensor."""
    S, reqs, hkv = 40, 5, 2
    q, k, v, _, _, _, _ = inputs(4, 8, hkv, 16, seed=12)
    kc, vc = (torch.zeros(reqs, hkv, S, D, dtype=torch.bfloat16, device=DEV) for _ in "kv")
    pos = torch.tensor([0, 39, 7, 20], dtype=torch.int32, device=DEV)
    req = torch.tensor([4, 0, 2, 1], device=DEV)
    out = torch.empty(4, 8, D, dtype=torch.bfloat16, device=DEV)
    plan = pkv.RopePlan(128)
    assert pkv.rope_append(pos, req * S + pos, q, k, v, kc, vc, plan, out=out) is out
    check(kc[req, :, pos.long()], k, pos.tolist(), plan)
    assert torch.equal(vc[req, :, pos.long()], v)


def test_matches_kv_append_where_nothing_turns():
    q, k, v, kc, vc, slots, pos = inputs(50, 8, 2, 16, seed=13, fused=False)
    kc2, vc2 = kc.clone(), vc.clone()
    pkv.rope_append(pos, slots, q, k, v, kc, vc, pkv.RopePlan(2, inv_freq=[0.0]))
    pkv.kv_append(slots, k, v, kc2, vc2)
    assert torch.equal(kc, kc2) and torch.equal(vc, vc2)


def test_graph_replay_and_another_stream():
    q, k, v, kc, vc, slots, pos = inputs(64, 32, 8, 16, seed=14)
    plan, out = pkv.RopePlan(128), torch.empty(64, 32, D, dtype=torch.bfloat16, device=DEV)
    want = pkv.rope_append(pos, slots, q, k, v, kc, vc, plan)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        there = pkv.rope_append(pos, slots, q, k, v, kc, vc, plan)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            pkv.rope_append(pos, slots, q, k, v, kc, vc, plan, out=out)
    torch.cuda.synchronize()
    assert torch.equal(there, want)
    pos += 5  # a replay reads the positions it finds
    g.replay()
    torch.cuda.synchronize()
    check(out, q, pos.tolist(), plan)


def test_checked_mode_reports_a_bad_slot_and_skips_it():
    pkv.set_checked(True)
    q, k, v, kc, vc, slots, pos = inputs(9, 8, 2, 16, seed=15)
    slots[4] = kc.shape[0] * kc.shape[2]  # one past the last
    k0 = kc.clone()
    out = pkv.rope_append(pos, slots, q, k, v, kc, vc, pkv.RopePlan(128))
    assert pkv.get_device_error() == "slot"
    good = torch.arange(9, device=DEV) != 4
    check(out, q, pos.tolist(), pkv.RopePlan(128))
    check(flat(kc)[slots[good]], k[good], pos[good].tolist(), pkv.RopePlan(128))
    rest = torch.ones(flat(kc).shape[0], dtype=torch.bool, device=DEV)
    rest[slots[good]] = False
    assert torch.equal(flat(kc)[rest], flat(k0)[rest])


def test_binding_refusals():
    q, k, v, kc, vc, slots, pos = inputs(4, 8, 2, 16, seed=16)
    plan = pkv.RopePlan(128)
    ok = [pos, slots, q, k, v, kc, vc, plan]

    def bad(i, x, error):
        a = list(ok)
        a[i] = x
        with pytest.raises(error):
            pkv.rope_append(*a)

    bad(0, pos.long(), TypeError)
    bad(0, pos[:3], ValueError)
    bad(1, slots.int(), TypeError)
    bad(2, q.float(), TypeError)
    bad(2, q.transpose(0, 1), ValueError)
    bad(2, q[..., ::2], ValueError)
    bad(2, q.cpu(), TypeError)
    bad(3, k[:, :1], ValueError)
    bad(5, kc[:, :, :8], ValueError)
    bad(7, plan.c, TypeError)
    with pytest.raises(ValueError):
        pkv.rope_append(*ok, out=torch.empty(4, 7, D, dtype=torch.bfloat16, device=DEV))
    with pytest.raises(pkv.PkvError):  # in place inside the wider projection rows
        pkv.rope_append(pos, slots, q, k, v, kc, vc, plan, out=q._base.view(-1)[:4 * 8 * D].view(4, 8, D))
    assert pkv.rope_append(pos[:0], slots[:0], q[:0], k[:0], v[:0], kc, vc, plan).shape == (0, 8, D)
