"""Head norms with the rotation on the GPU against the 64-bit oracle (needs an sm_103a GPU).

Tolerances per element, from the arithmetic. Forward: y is one bf16 rounding (2^-8 |y|) of an fp32
value; the sum of D <= 512 squares is off by at most 32 roundings of 2^-24 (16 in a lane, 5 joins,
the products), the root by half that and 2 steps, the products with r and w, the rotation's factors
and sums by a few more: together under 2^-18 of the normed pair's magnitudes. Backward: the same
2^-18 of the terms of dx (size) besides its one rounding; dw is a sum in fp32 whose order has at most
32 steps a thread in these tests, 2 heads each, then up to 256 sets, 76 blocks and 8 runs: under 448
roundings of 2^-24, with the terms' own errors under 2^-15 of the sum of the magnitudes.
"""
import numpy as np
import pytest
import torch

import context_parallelism_gb300 as up
from oracle import norm_rope_bwd_ref, norm_rope_ref
from tests.test_gpu_paged import Batch

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


def _words(ph):
    return None if ph is None else [int(w) % (1 << 64) for w in ph.tolist()]


def _np(t):
    return t.detach().double().cpu().numpy()


def _bf(*shape, seed=0, scale=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(BF)


def _weights(D, wide, seed, offset=0.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    w = 1 - offset + 0.3 * torch.randn(D, generator=g, device=DEV)
    return w if wide else w.to(BF)


def _pairs(n, rot, inter):
    """Sum of the magnitudes of each feature's pair."""
    a = np.abs(n)
    s = a.copy()
    p = (a[..., 0:rot:2] + a[..., 1:rot:2]) if inter else (a[..., :rot // 2] + a[..., rot // 2:rot])
    if inter:
        s[..., 0:rot:2] = s[..., 1:rot:2] = p
    else:
        s[..., :rot // 2] = s[..., rot // 2:rot] = p
    return s


def _check(y, x, w, pos, ph, m=1.0, inter=False, eps=1e-6, offset=0.0):
    ref = norm_rope_ref(x, w, pos, _words(ph), m, inter, eps, offset)
    flat = norm_rope_ref(x, w, None, None, eps=eps, offset=offset)
    size = np.abs(flat) if ph is None else _pairs(flat, 2 * ph.numel(), inter) * m
    tol = 2.0 ** -8 * np.abs(ref) + 2.0 ** -18 * size
    err = np.abs(_np(y) - ref)
    assert (err <= tol).all(), float((err - tol).max())


def _check_back(dx, dw, dy, x, w, pos, ph, m=1.0, inter=False, eps=1e-6, offset=0.0):
    rx, rw, size, w_size = norm_rope_bwd_ref(dy, x, w, pos, _words(ph), m, inter, eps, offset)
    err = np.abs(_np(dx) - rx) - 2.0 ** -8 * np.abs(rx) - 2.0 ** -18 * size
    assert (err <= 0).all(), float(err.max())
    if w is None:
        assert dw is None
        return
    assert dw.dtype is torch.float32
    err = np.abs(_np(dw) - rw) - 2.0 ** -15 * w_size
    assert (err <= 0).all(), float(err.max())


SHAPES = [  # B, S, Hq, Hkv, D, rot
    (1, 1, 1, 1, 64, 64), (1, 1, 32, 8, 128, 128), (2, 7, 5, 1, 128, 64), (1, 130, 28, 4, 128, 128),
    (3, 5, 10, 2, 80, 80), (1, 33, 4, 4, 192, 96), (2, 3, 3, 3, 256, 16), (1, 65, 40, 8, 64, 32),
    (1, 2, 9, 2, 72, 48), (1, 3, 2, 1, 512, 512), (1, 4, 3, 1, 16, 16), (2, 2, 1, 2, 24, 16),
    (1, 5, 6, 1, 8, 0), (1, 9, 7, 3, 128, 0),
]


@pytest.mark.parametrize("wide,offset", [(False, 0.0), (True, 1.0)])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("shape", SHAPES)
def test_forward_and_backward(shape, inter, wide, offset):
    B, S, Hq, Hkv, D, rot = shape
    q, k = _bf(B, S, Hq, D, seed=1), _bf(B, S, Hkv, D, seed=2, scale=8.0)
    qw, kw = _weights(D, wide, 3, offset), _weights(D, wide, 4, offset)
    ph, m = up.rope_phases(rot, theta=500000.0) if rot else (None, 1.0)
    how = dict(phases=ph, mscale=1.25, interleaved=inter, start=1000, offset=offset)
    pos = np.tile(1000 + np.arange(S), (B, 1))
    y, z = up.norm_rope_forward(q, k, qw, kw, **how)
    ref = (pos, ph, 1.25, inter, 1e-6, offset)
    _check(y, q, qw, *ref)
    _check(z, k, kw, *ref)
    dy, dz = _bf(B, S, Hq, D, seed=5), _bf(B, S, Hkv, D, seed=6)
    dq, dk, dqw, dkw = up.norm_rope_backward(dy, dz, q, k, qw, kw, **how)
    _check_back(dq, dqw, dy, q, qw, *ref)
    _check_back(dk, dkw, dz, k, kw, *ref)


def test_without_weights_or_one_tensor():
    q, k, dy = _bf(2, 9, 6, 128, seed=1), _bf(2, 9, 2, 128, seed=2), _bf(2, 9, 6, 128, seed=3)
    kw, dz = _weights(128, True, 4), _bf(2, 9, 2, 128, seed=5)
    ph, _ = up.rope_phases(128)
    pos = np.tile(np.arange(9), (2, 1))
    y, z = up.norm_rope_forward(q, k, None, kw, ph, eps=1e-3, offset=1.0)
    _check(y, q, None, pos, ph, eps=1e-3)
    _check(z, k, kw, pos, ph, eps=1e-3, offset=1.0)
    dq, dk, dqw, dkw = up.norm_rope_backward(dy, dz, q, k, None, kw, ph, eps=1e-3, offset=1.0)
    _check_back(dq, dqw, dy, q, None, pos, ph, eps=1e-3)
    _check_back(dk, dkw, dz, k, kw, pos, ph, eps=1e-3, offset=1.0)
    none, z2 = up.norm_rope_forward(None, k, None, kw, ph, eps=1e-3, offset=1.0)
    assert none is None and torch.equal(z, z2)
    _, dk2, _, dkw2 = up.norm_rope_backward(None, dz, None, k, None, kw, ph, eps=1e-3, offset=1.0)
    assert torch.equal(dk, dk2)
    _check_back(dk2, dkw2, dz, k, kw, pos, ph, eps=1e-3, offset=1.0)
    dq3, none, dqw3, _ = up.norm_rope_backward(dy, None, q, None, None, None, ph, eps=1e-3)
    assert torch.equal(dq, dq3) and none is None and dqw3 is None


def test_layouts_and_in_place():
    """Rows of a fused projection, head-major tensors, broadcast gradients; outputs keep the inputs'
    layout; in place gives the same bits."""
    B, S, Hq, Hkv, D = 2, 37, 8, 2, 128
    x = _bf(B, S, (Hq + 2 * Hkv) * D, seed=1)
    q = x[..., :Hq * D].unflatten(-1, (Hq, D))
    k = x[..., Hq * D:(Hq + Hkv) * D].unflatten(-1, (Hkv, D))
    qw, kw = _weights(D, False, 2), _weights(D, False, 3)
    ph, m = up.rope_phases(D)
    y, z = up.norm_rope_forward(q, k, qw, kw, ph, start=5)
    want = up.norm_rope_forward(q.contiguous(), k.contiguous(), qw, kw, ph, start=5)
    assert torch.equal(y, want[0]) and torch.equal(z, want[1])
    qh = q.transpose(1, 2).contiguous().transpose(1, 2)
    yh, _ = up.norm_rope_forward(qh, None, qw, None, ph, start=5)
    assert torch.equal(yh, y) and yh.stride() == qh.stride()
    dy = _bf(B, 1, 1, D, seed=4).expand(B, S, Hq, D)  # one gradient for all tokens and heads
    dz = _bf(B, S, Hkv, D, seed=5)
    d = up.norm_rope_backward(dy, dz, q, k, qw, kw, ph, start=5)
    e = up.norm_rope_backward(dy.contiguous(), dz, q.contiguous(), k.contiguous(), qw, kw, ph, start=5)
    assert all(torch.equal(a, b) for a, b in zip(d, e))
    rest = x[..., (Hq + Hkv) * D:].clone()
    y2, z2 = up.norm_rope_forward(q, k, qw, kw, ph, start=5, inplace=True)
    assert y2 is q and torch.equal(q, y) and torch.equal(k, z)
    assert torch.equal(x[..., (Hq + Hkv) * D:], rest)
    a, b = dy.contiguous(), dz.clone()
    x0 = want  # any forward input: here the normed tensors
    f = up.norm_rope_backward(a.clone(), b.clone(), *x0, qw, kw, ph, start=5)
    g = up.norm_rope_backward(a, b, *x0, qw, kw, ph, start=5, inplace=True)
    assert g[0] is a and all(torch.equal(s, t) for s, t in zip(f, g))


def test_given_and_far_positions():
    pos = torch.tensor([[0, -1, 1 << 24, (1 << 31) + 1, 1 << 40, (1 << 62) + 12345, -(1 << 50)]])
    q, w = _bf(1, 7, 3, 64, seed=6), _weights(64, True, 7)
    ph, _ = up.rope_phases(64)
    y, _ = up.norm_rope_forward(q, None, w, None, ph, positions=pos.to(DEV))
    _check(y, q, w, pos.numpy(), ph)
    dq, _, dw, _ = up.norm_rope_backward(y, None, q, None, w, None, ph, positions=pos.to(DEV))
    _check_back(dq, dw, y, q, w, pos.numpy(), ph)


def test_large_small_and_special_heads():
    """Squares beyond fp32's range (above and below), zeros, infinities and NaN; a head does not see
    its neighbours."""
    x = _bf(1, 1, 8, 128, seed=1)
    x[0, 0, 0] *= 2.0 ** 100
    x[0, 0, 1] *= 2.0 ** -120
    x[0, 0, 2] = 0
    x[0, 0, 3, 17] = float("inf")
    x[0, 0, 4, 100] = float("nan")
    x[0, 0, 5] = 2.0 ** 127
    dy, w = _bf(1, 1, 8, 128, seed=2), _weights(128, True, 3)
    ph, _ = up.rope_phases(128)
    pos, good = np.array([[9]]), [0, 1, 2, 5, 6, 7]
    y, _ = up.norm_rope_forward(x, None, w, None, ph, start=9)
    _check(y[:, :, good], x[:, :, good], w, pos, ph)
    assert (y[0, 0, 2] == 0).all() and not y[0, 0, 3:5].isfinite().all()
    dx, _, _, _ = up.norm_rope_backward(dy, None, x, None, w, None, ph, start=9)
    rx = norm_rope_bwd_ref(dy, x.nan_to_num(nan=1.0, posinf=1.0), w, pos, _words(ph))
    for h in good:
        err = np.abs(_np(dx)[0, 0, h] - rx[0][0, 0, h])
        # results below bf16's smallest normal number may be lost
        assert (err <= 2.0 ** -8 * np.abs(rx[0][0, 0, h]) + 2.0 ** -18 * rx[2][0, 0, h] + 2.0 ** -126).all(), h


def test_eps_zero_and_large():
    x, w = _bf(1, 3, 2, 64, seed=1, scale=1e-3), _weights(64, False, 2)
    for eps in (0.0, 1e-5, 10.0):
        y, _ = up.norm_rope_forward(x, None, w, None, eps=eps)
        _check(y, x, w, None, None, eps=eps)


def test_gradient_against_differences():
    """The change of <dy, y> in 64 bits over a step of x, from the oracle's forward alone."""
    x, dy, w = _bf(1, 2, 2, 32, seed=1), _bf(1, 2, 2, 32, seed=2), _weights(32, True, 3)
    ph, _ = up.rope_phases(16)
    pos = np.array([[3, 4]])
    dx, _, dw, _ = up.norm_rope_backward(dy, None, x, None, w, None, ph, start=3)
    d, xn, wn = _np(dy), _np(x), _np(w)

    def f(x, w):
        return (d * norm_rope_ref(x, w, pos, _words(ph))).sum()

    h = 1e-5  # the difference is off by about h^2 times a third derivative of order one
    for at in np.ndindex(xn.shape):
        e = np.zeros_like(xn)
        e[at] = h
        want = (f(xn + e, wn) - f(xn - e, wn)) / (2 * h)
        assert abs(float(dx[at]) - want) <= 2.0 ** -8 * abs(want) + 1e-4
    for i in range(32):
        e = np.zeros(32)
        e[i] = h
        want = (f(xn, wn + e) - f(xn, wn - e)) / (2 * h)
        assert abs(float(dw[i]) - want) <= 1e-4


def test_many_tokens_and_repeats():
    """More tokens than walkers: sums over many steps, the same bits twice, the weights' gradient equal
    to the sum over halves within its rounding."""
    B, S, Hq, Hkv, D = 2, 3001, 8, 2, 128
    q, k = _bf(B, S, Hq, D, seed=1), _bf(B, S, Hkv, D, seed=2)
    dy, dz = _bf(B, S, Hq, D, seed=3), _bf(B, S, Hkv, D, seed=4)
    qw, kw = _weights(D, False, 5), _weights(D, False, 6)
    ph, _ = up.rope_phases(D)
    a = up.norm_rope_backward(dy, dz, q, k, qw, kw, ph)
    b = up.norm_rope_backward(dy, dz, q, k, qw, kw, ph)
    assert all(torch.equal(s, t) for s, t in zip(a, b))
    for i, (x, d, w) in enumerate(((q, dy, qw), (k, dz, kw))):
        f, w64 = x.double().requires_grad_(), w.double().requires_grad_()
        n = f * (f.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * w64
        ang = torch.arange(S, device=DEV)[:, None] * 10000.0 ** (
            -torch.arange(0, D, 2, device=DEV, dtype=torch.float64) / D)
        c, s = ang.cos()[:, None], ang.sin()[:, None]
        y = torch.cat((n[..., :64] * c - n[..., 64:] * s, n[..., 64:] * c + n[..., :64] * s), -1)
        gx, gw = torch.autograd.grad(y, (f, w64), d.double())
        err = (a[i].double() - gx).abs()
        assert (err <= 2.0 ** -8 * gx.abs() + 1e-4).all()
        # terms of order one: their sum in any order of fp32 is off by far less than a term
        assert ((a[2 + i].double() - gw).abs() <= 1e-2).all()


def test_no_tokens():
    q, w = torch.zeros((2, 0, 4, 64), dtype=BF, device=DEV), _weights(64, False, 1)
    y, _ = up.norm_rope_forward(q, None, w, None)
    assert y.shape == q.shape
    dq, _, dw, _ = up.norm_rope_backward(q, None, q, None, w, None)
    assert dq.shape == q.shape and (dw == 0).all()


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("wide", [False, True])
def test_append(packed, wide):
    """The cache and q hold what norm_rope_forward gives for the tokens' positions; v as it is."""
    counts = [2, 0, 1, 3] if packed else [2] * 4
    b = Batch(counts, [40, 7, 130, 3], 8, 2, 128, 16, 0, seed=3, packed=packed)
    lead = b.q.shape[:-2]
    k, v = _bf(*lead, 2, 128, seed=4), _bf(*lead, 2, 128, seed=5)
    qw, kw = _weights(128, wide, 6), _weights(128, wide, 7)
    ph, m = up.rope_phases(64)
    kp, vp = b.kp.clone(), b.vp.clone()
    how = dict(phases=ph, mscale=1.5, start=50, offset=0.5)
    qo = torch.full_like(b.q, 7.0)
    out = up.kv_append(k, v, kp, vp, b.table, b.seq_len, q=b.q, q_out=qo, cu_seqlens=b.cu,
                       q_weight=qw, k_weight=kw, eps=1e-5, **how)
    assert out is qo
    # the same through the plain append of tokens that were normed and turned before
    lens, flat = b.seq_len.tolist(), (lambda t: t.reshape(1, -1, *t.shape[-2:]))
    pos, row = torch.zeros(flat(k).shape[:2], dtype=torch.int64), 0
    for n, ln in zip(counts, lens):
        for i in range(n):
            pos[0, row] = 50 + ln - n + i
            row += 1
    how = dict(phases=ph, mscale=1.5, offset=0.5, eps=1e-5, positions=pos.to(DEV))
    qn, kn = up.norm_rope_forward(flat(b.q), flat(k), qw, kw, **how)
    kp2, vp2 = b.kp.clone(), b.vp.clone()
    up.kv_append(kn.view(k.shape), v, kp2, vp2, b.table, b.seq_len, cu_seqlens=b.cu)
    bits = lambda t: t.contiguous().view(torch.int16)  # noqa: E731
    assert torch.equal(bits(kp), bits(kp2)) and torch.equal(bits(vp), bits(vp2))
    assert torch.equal(flat(qo)[0, :row], qn[0, :row])
    assert (flat(qo)[0, row:] == 7.0).all()  # rows of no sequence stay


def test_append_reports_missing_pages():
    kp, vp = _bf(2, 16, 2, 64), _bf(2, 16, 2, 64)
    k, w = _bf(2, 1, 2, 64, seed=1), _weights(64, False, 2)
    table = torch.tensor([[5], [1]], dtype=torch.int32, device=DEV)
    lens = torch.tensor([3, 17], dtype=torch.int32, device=DEV)
    up.upipe_sync_status()
    before = kp.clone(), vp.clone()
    up.kv_append(k, k, kp, vp, table, lens, k_weight=w, eps=1e-6)
    with pytest.raises(up.UpipeError) as e:
        up.upipe_sync_status()
    assert e.value.status == up.UPIPE_ERR_PAGE
    assert torch.equal(kp, before[0]) and torch.equal(vp, before[1])
    up.upipe_sync_status()


def test_streams_and_graphs():
    q, k = _bf(1, 300, 8, 128, seed=1), _bf(1, 300, 2, 128, seed=2)
    dy, dz = _bf(1, 300, 8, 128, seed=3), _bf(1, 300, 2, 128, seed=4)
    qw, kw = _weights(128, False, 5), _weights(128, False, 6)
    ph, _ = up.rope_phases(128)
    want = up.norm_rope_forward(q, k, qw, kw, ph), up.norm_rope_backward(dy, dz, q, k, qw, kw, ph)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = (up.norm_rope_forward(q, k, qw, kw, ph, stream=s),
           up.norm_rope_backward(dy, dz, q, k, qw, kw, ph, stream=s))
    s.synchronize()
    for a, b in zip(want[0] + want[1], got[0] + got[1]):
        assert torch.equal(a, b)
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(up.norm_rope_forward(q, k, qw, kw, ph) +
                        up.norm_rope_backward(dy, dz, q, k, qw, kw, ph))
        graphs.append(g)
    for new in (11, 12):
        q.copy_(_bf(1, 300, 8, 128, seed=new))
        want = up.norm_rope_forward(q, k, qw, kw, ph) + up.norm_rope_backward(dy, dz, q, k, qw, kw, ph)
        t = torch.cuda.Stream()
        t.wait_stream(torch.cuda.current_stream())
        graphs[0].replay()
        with torch.cuda.stream(t):
            graphs[1].replay()
        torch.cuda.synchronize()
        for o in outs:
            assert all(torch.equal(a, b) for a, b in zip(o, want))


def test_raw_entries():
    def h(t):
        st = t.stride()
        return up.Heads(t.data_ptr(), st[0], st[1], st[2], t.shape[2])

    q, dy, w = _bf(2, 5, 3, 64, seed=1), _bf(2, 5, 3, 64, seed=2), _weights(64, True, 3)
    ph, _ = up.rope_phases(32)
    norm = up.Norm(w.data_ptr(), None, 0.0, 1e-6, 1)
    y, dx, dw = torch.zeros_like(q), torch.zeros_like(q), torch.zeros(64, device=DEV)
    up.upipe_norm_rope_fwd(h(q), None, h(y), None, norm, None, 7, ph, 1.0, 2, 5, 64, 32, False)
    n = up.upipe_norm_rope_workspace_bytes(2, 5, 3, 0, 64)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    args = (h(dy), None, h(q), None, h(dx), None, dw, None, norm, None, 7, ph, 1.0, 2, 5, 64, 32,
            False, ws)
    up.upipe_norm_rope_bwd(*args)
    assert torch.equal(y, up.norm_rope_forward(q, None, w, None, ph, start=7)[0])
    want = up.norm_rope_backward(dy, None, q, None, w, None, ph, start=7)
    assert torch.equal(dx, want[0]) and torch.equal(dw, want[2])
    with pytest.raises(up.UpipeError) as e:
        up.upipe_norm_rope_bwd(*args, workspace_bytes=n - 1)
    assert e.value.status == up.UPIPE_ERR_WORKSPACE_TOO_SMALL


@pytest.mark.parametrize("B,S,Hq,Hkv,D", [(1, 1, 1, 1, 8), (2, 300, 28, 4, 128), (1, 5000, 5, 1, 80)])
def test_workspace_bounds(B, S, Hq, Hkv, D):
    """Exactly the declared bytes, between bands that stay as they are; what they held before does not
    matter; outputs stay within theirs."""
    q, k, dy, dz = (_bf(B, S, h, D, seed=i) for i, h in enumerate((Hq, Hkv, Hq, Hkv)))
    qw, kw = _weights(D, True, 5), _weights(D, True, 6)
    want = up.norm_rope_backward(dy, dz, q, k, qw, kw)
    size, band = up.upipe_norm_rope_workspace_bytes(B, S, Hq, Hkv, D), 1 << 16
    for fill in (0, 255):
        big = torch.full((size + 2 * band,), fill, dtype=torch.uint8, device=DEV)
        got = up.norm_rope_backward(dy, dz, q, k, qw, kw, workspace=big[band:band + size])
        assert all(torch.equal(a, b) for a, b in zip(want, got))
        assert (big[:band] == fill).all() and (big[band + size:] == fill).all()
    # rows beside the outputs: every second token of a larger tensor
    x = torch.full((B, 2 * S, Hq, D), 7.0, dtype=BF, device=DEV)
    x[:, ::2] = q
    y, _ = up.norm_rope_forward(x[:, ::2], None, qw, None, inplace=True)
    assert torch.equal(y, up.norm_rope_forward(q, None, qw, None)[0])
    assert (x[:, 1::2] == 7).all()


def test_offsets_beyond_32_bits():
    """Strides that put a head more than 2^31 elements from the first."""
    far = (1 << 31) + 8
    try:
        x = torch.empty(far + 128, dtype=BF, device=DEV)
    except torch.OutOfMemoryError:
        pytest.skip("no room")
    q = x.as_strided((1, 2, 2, 64), (0, 64, far, 1))
    q.copy_(_bf(1, 2, 2, 64, seed=1))
    w, (ph, _) = _weights(64, False, 2), up.rope_phases(64)
    want = up.norm_rope_forward(q.contiguous(), None, w, None, ph)[0]
    dy = _bf(1, 2, 2, 64, seed=3)
    d_want = up.norm_rope_backward(dy, None, q.contiguous(), None, w, None, ph)
    d = up.norm_rope_backward(dy, None, q, None, w, None, ph)
    assert torch.equal(d[0], d_want[0]) and torch.equal(d[2], d_want[2])
    up.norm_rope_forward(q, None, w, None, ph, inplace=True)
    assert torch.equal(q, want)
