"""Rotary positions on the GPU against the 64-bit oracle (needs an sm_103a GPU).

Tolerance per element, from the arithmetic: y is one bf16 rounding (half a step: 2^-8 |y|) of an
fp32 value. Its two products and sum, the factors' rounding and mscale's are a few 2^-24; the
angle is rounded to 24 bits (at most pi 2^-24 radians) and sincospi errs by at most 2 steps:
together under 2^-20 (|x1| + |x2|) mscale.
"""
import numpy as np
import pytest
import torch

import context_parallelism_gb300 as up
from oracle import rope_ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _words(phases):
    return [int(w) % (1 << 64) for w in phases.tolist()]


def _np(t):
    return t.detach().double().cpu().numpy()


def _check(y, x, pos, phases, m, inter, back=False):
    rot = 2 * phases.numel()
    ref = rope_ref(x, pos, _words(phases), m, inter, back)
    xa = np.abs(_np(x))
    pair = np.zeros_like(xa)
    if inter:
        s = xa[..., 0:rot:2] + xa[..., 1:rot:2]
        pair[..., 0:rot:2], pair[..., 1:rot:2] = s, s
    else:
        s = xa[..., :rot // 2] + xa[..., rot // 2:rot]
        pair[..., :rot // 2], pair[..., rot // 2:rot] = s, s
    tol = 2.0 ** -8 * np.abs(ref) + 2.0 ** -20 * pair * m
    err = np.abs(_np(y) - ref)
    assert (err <= tol).all(), float((err - tol).max())
    assert torch.equal(y[..., rot:], x[..., rot:])


def _bf(*shape, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(shape, generator=g, device=DEV).to(torch.bfloat16)


SHAPES = [  # B, S, Hq, Hkv, D, rot
    (1, 1, 1, 1, 64, 64), (1, 1, 32, 8, 128, 128), (2, 7, 5, 1, 128, 64), (1, 130, 28, 4, 128, 128),
    (3, 5, 10, 2, 80, 80), (1, 33, 4, 4, 192, 96), (2, 3, 3, 3, 256, 16), (1, 65, 40, 8, 64, 32),
    (1, 2, 9, 2, 72, 48), (1, 3, 2, 1, 1024, 1024),
]


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("shape", SHAPES)
def test_forward_and_backward(shape, inter):
    B, S, Hq, Hkv, D, rot = shape
    q, k = _bf(B, S, Hq, D, seed=1), _bf(B, S, Hkv, D, seed=2)
    ph, m = up.rope_phases(rot, theta=500000.0)
    y, z = up.rope_forward(q, k, ph, m, inter, start=1000)
    pos = np.tile(1000 + np.arange(S), (B, 1))
    _check(y, q, pos, ph, m, inter)
    _check(z, k, pos, ph, m, inter)
    y, z = up.rope_backward(q, k, ph, m, inter, start=1000)
    _check(y, q, pos, ph, m, inter, back=True)
    _check(z, k, pos, ph, m, inter, back=True)


@pytest.mark.parametrize("kind", [up.UPIPE_ROPE_LINEAR, up.UPIPE_ROPE_NTK, up.UPIPE_ROPE_BY_PARTS])
def test_scaled_frequencies_and_given_positions(kind):
    B, S = 2, 19
    q, k = _bf(B, S, 4, 128, seed=3), _bf(B, S, 2, 128, seed=4)
    ph, m = up.rope_phases(128, theta=10000.0, scaling=kind, factor=8.0, trained_len=8192)
    g = torch.Generator().manual_seed(5)
    pos = torch.randint(0, 1 << 20, (B, S), generator=g)
    y, z = up.rope_forward(q, k, ph, m, positions=pos.to(DEV))
    _check(y, q, pos.numpy(), ph, m, False)
    _check(z, k, pos.numpy(), ph, m, False)
    y, z = up.rope_backward(q, k, ph, m, positions=pos.to(DEV))
    _check(y, q, pos.numpy(), ph, m, False, back=True)


def test_far_and_negative_positions():
    """Angles stay exact where a 32-bit (or 64-bit floating-point) product would have lost them."""
    pos = torch.tensor([[0, -1, 1 << 24, (1 << 31) + 1, 1 << 40, (1 << 62) + 12345, -(1 << 50)]])
    q = _bf(1, 7, 2, 64, seed=6)
    ph, m = up.rope_phases(64)
    y, _ = up.rope_forward(q, None, ph, m, positions=pos.to(DEV))
    _check(y, q, pos.numpy(), ph, m, False)
    assert torch.equal(y[:, 0], q[:, 0])  # position 0: the identity


def test_own_frequencies():
    f = [1.0, 0.25, 0.0, 3.0, 100.0, 1e-3, 1e-6, -0.5]
    q = _bf(1, 5, 2, 16, seed=7)
    ph, m = up.rope_phases(16, inv_freq=f)
    y, _ = up.rope_forward(q, None, ph, start=77)
    _check(y, q, np.array([77 + np.arange(5)]), ph, m, False)
    a = torch.arange(77, 82, dtype=torch.float64)[:, None] * torch.tensor(f, dtype=torch.float64)
    x = q[0].double().cpu()
    want = x[..., :8] * a.cos()[:, None] - x[..., 8:] * a.sin()[:, None]
    assert (y[0, ..., :8].double().cpu() - want).abs().max() <= 2.0 ** -8 * want.abs().max() + 1e-5


@pytest.mark.parametrize("inter", [False, True])
def test_gradient_against_differences(inter):
    """<dy, R x> is linear in x: its difference over a step of +-1 at one feature is the gradient,
    up to the roundings of R x (bf16, summed over the outputs that the feature reaches)."""
    ph, m = up.rope_phases(16)
    x, dy = _bf(1, 2, 1, 16, seed=8), _bf(1, 2, 1, 16, seed=9)
    dx, _ = up.rope_backward(dy, None, ph, m, inter, start=3)
    for s in range(2):
        for d in range(16):
            vals = []
            for step in (1.0, -1.0):
                e = torch.zeros_like(x)
                e[0, s, 0, d] = step
                y, _ = up.rope_forward(e, None, ph, m, inter, start=3)
                vals.append((y.double() * dy.double()).sum())
            num = float(vals[0] - vals[1]) / 2
            # two outputs of size at most 1, each off by 2^-8 of itself, and dx's own rounding
            tol = 2.0 ** -8 * (2 * float(dy.abs().max()) + abs(num)) + 1e-5
            assert abs(float(dx[0, s, 0, d]) - num) <= tol


def test_strided_inputs_and_head_major():
    B, S, Hq, Hkv, D = 2, 9, 6, 2, 128
    x = _bf(B, S, (Hq + 2 * Hkv) * D, seed=10)
    q = x[..., :Hq * D].unflatten(-1, (Hq, D))
    k = x[..., Hq * D:(Hq + Hkv) * D].unflatten(-1, (Hkv, D))
    ph, m = up.rope_phases(D)
    a = up.rope_forward(q, k, ph, m)
    b = up.rope_forward(q.contiguous(), k.contiguous(), ph, m)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    hm = q.transpose(1, 2).contiguous().transpose(1, 2)  # [B, H, S, D] in memory
    c = up.rope_forward(hm, None, ph, m)
    assert torch.equal(c[0], a[0])
    wide = q[:1, :1].expand(B, S, Hq, D)  # a broadcast input
    d = up.rope_forward(wide, None, ph, m)
    assert torch.equal(d[0], up.rope_forward(wide.contiguous(), None, ph, m)[0])


@pytest.mark.parametrize("rot", [128, 48])
def test_in_place_inside_a_fused_projection(rot):
    B, S, Hq, Hkv, D = 1, 17, 6, 2, 128
    x = _bf(B, S, (Hq + 2 * Hkv) * D, seed=11)
    q = x[..., :Hq * D].unflatten(-1, (Hq, D))
    k = x[..., Hq * D:(Hq + Hkv) * D].unflatten(-1, (Hkv, D))
    v = x[..., (Hq + Hkv) * D:].clone()
    ph, m = up.rope_phases(rot)
    want = up.rope_forward(q, k, ph, m, start=5)
    got = up.rope_forward(q, k, ph, m, start=5, inplace=True)
    assert got[0].data_ptr() == q.data_ptr()
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert torch.equal(x[..., (Hq + Hkv) * D:], v)


def test_infinities_and_nan_stay_in_their_pairs():
    q = _bf(1, 2, 2, 32, seed=12)
    q[0, 0, 0, 3], q[0, 1, 1, 20] = float("inf"), float("nan")
    ph, m = up.rope_phases(32)
    y, _ = up.rope_forward(q, None, ph, m, start=9)
    bad = ~torch.isfinite(y)
    want = torch.zeros_like(bad)
    want[0, 0, 0, [3, 19]] = True
    want[0, 1, 1, [4, 20]] = True
    assert torch.equal(bad, want)


def test_empty_and_captured_and_other_stream():
    ph, m = up.rope_phases(64)
    e, _ = up.rope_forward(torch.empty((2, 0, 4, 64), dtype=torch.bfloat16, device=DEV), None, ph)
    assert e.shape == (2, 0, 4, 64)
    q = _bf(1, 33, 4, 64, seed=13)
    want, _ = up.rope_forward(q, None, ph, m)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got, _ = up.rope_forward(q, None, ph, m, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    pos = torch.arange(33, device=DEV)[None].contiguous()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y, _ = up.rope_forward(q, None, ph, m, positions=pos)
        back, _ = up.rope_backward(y, None, ph, m, positions=pos)
    q.copy_(_bf(1, 33, 4, 64, seed=14))
    pos.add_(100)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, up.rope_forward(q, None, ph, m, positions=pos)[0])
    assert torch.equal(back, up.rope_backward(y, None, ph, m, positions=pos)[0])


def test_attention_depends_on_relative_positions_only():
    """With the framework's attention: shifting every position leaves o (rotation moves q and k by
    the same angle), up to roundings, here in the 2-norm: an element of the rotated q and k is off
    by at most 2^-8 of itself, so by less than 2^-8 / sqrt(3) in the root mean square, and a score
    (a sum of 64 such products over 8, of standard deviation 1) by 2^-8 sqrt(2 / 3) < 2^-8. Every
    weight moves by that relative amount, o by at most as much of the values' size again, twice
    (both runs), and o, lying below the values' size by the root of the row's effective number of
    keys like its error, is rounded twice: under 2^-8 (2 + 2) = 2^-6 of o's norm."""
    q, k, v = _bf(1, 200, 4, 64, seed=15), _bf(1, 200, 2, 64, seed=16), _bf(1, 200, 2, 64, seed=17)
    ph, m = up.rope_phases(64)
    o0, _ = up.attention_forward(*up.rope_forward(q, k, ph, m), v)
    o1, _ = up.attention_forward(*up.rope_forward(q, k, ph, m, start=123457), v)
    up.upipe_sync_status()
    plain, _ = up.attention_forward(q, k, v)
    moved = (o0.float() - o1.float()).norm() / o0.float().norm()
    turned = (o0.float() - plain.float()).norm() / o0.float().norm()
    assert moved < 2.0 ** -6 and turned > 10 * moved
