"""Head norms of heads whose squares leave the range of 32 bits, at both ends and with an eps of any size
(needs an sm_103a GPU).

Tolerances as in test_gpu_norm_rope.py: the heads are scaled by powers of two before they are summed, which
rounds nothing. Results beyond bf16's largest number are not looked at, and what lies below its smallest
normal one may be lost.
"""
import numpy as np
import pytest
import torch

import context_parallelism_gb300 as up
from oracle import norm_rope_bwd_ref, norm_rope_ref
from tests.test_gpu_norm_rope import _bf, _check, _np, _pairs, _weights, _words

pytestmark = pytest.mark.gpu
DEV = "cuda"
TINY = 2.0 ** -126


def _back(dx, dw, dy, x, w, pos, ph, inter, eps):
    rx, rw, size, w_size = norm_rope_bwd_ref(dy, x, w, pos, _words(ph), 1.0, inter, eps)
    inside = np.abs(rx) < 3e38
    err = np.abs(_np(dx) - rx) - 2.0 ** -8 * np.abs(rx) - 2.0 ** -18 * size - TINY
    assert (err <= 0)[inside].all(), float(err[inside].max())
    assert (np.abs(_np(dw) - rw) <= 2.0 ** -15 * w_size).all()


# exponents of the heads; of one head's elements (far apart: the small squares do not count); eps
SMALL = [([-20, -62, -64, -75, -90, -110, -126, -133], 0.0), ([-40, -46, -47, -48, -49, -50, -80, -120], 1e-40),
         ([-30, -60, -80, -83, -84, -90, -100, -133], 1e-50), ([-70] * 8, 1e-38), ([-100] * 8, 1e-100),
         ([-133] * 8, 0.0)]
LARGE = [([40, 57, 58, 59, 60, 62, 64, 100], 0.0), ([55, 59, 61, 62, 63, 64, 65, 100], 1e38),
         ([0, 30, 50, 60, 62, 63, 64, 126], 3e38), ([-100, -50, 0, 1, 40, 50, 60, 62], 1e37)]


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("D,rot", [(128, 64), (512, 0), (24, 16)])
@pytest.mark.parametrize("powers,eps", SMALL + LARGE)
def test_heads_of_any_size(powers, eps, D, rot, inter):
    # magnitudes from 1/2 to 1, so that no square is far from its head's
    x = (_bf(1, 2, 8, D, seed=1).float().clamp(-1, 1) * 0.5)
    x = x + 0.5 * torch.where(x < 0, -1.0, 1.0)
    x = (x.double() * 2.0 ** torch.tensor(powers, device=DEV, dtype=torch.float64)[:, None]).to(torch.bfloat16)
    x = torch.where(x == 0, torch.tensor(2.0 ** -133, device=DEV, dtype=torch.bfloat16), x)
    dy, w = _bf(1, 2, 8, D, seed=2), _weights(D, True, 3)
    if eps == 0:
        dy = dy * 2.0 ** -20  # gradients within bf16's range
    ph = up.rope_phases(rot)[0] if rot else None
    pos = np.array([[9, 10]])
    y, _ = up.norm_rope_forward(x, None, w, None, ph, eps=eps, interleaved=inter, start=9)
    ref = norm_rope_ref(x, w, pos, _words(ph), 1.0, inter, eps)
    flat = norm_rope_ref(x, w, None, None, eps=eps)
    size = np.abs(flat) if ph is None else _pairs(flat, rot, inter)
    err = np.abs(_np(y) - ref) - 2.0 ** -8 * np.abs(ref) - 2.0 ** -18 * size - TINY
    assert (err <= 0).all(), float(err.max())
    dx, _, dw, _ = up.norm_rope_backward(dy, None, x, None, w, None, ph, eps=eps, interleaved=inter, start=9)
    _back(dx, dw, dy, x, w, pos, ph, inter, eps)


def test_zeros_and_small_eps():
    """A head of zeros is zeros while eps is there, however small, and has no direction without it; its
    neighbours do not see it."""
    x, w = _bf(1, 1, 5, 64, seed=1), _weights(64, True, 2)
    x[0, 0, 2] = 0
    dy = _bf(1, 1, 5, 64, seed=3) * 2.0 ** -30
    for eps in (1e-6, 1e-38, 1e-44, 1e-50):
        y, _ = up.norm_rope_forward(x, None, w, None, eps=eps)
        assert (y[0, 0, 2] == 0).all()
        _check(y, x, w, None, None, eps=eps)
        dx, _, dw, _ = up.norm_rope_backward(dy, None, x, None, w, None, eps=eps)
        _back(dx, dw, dy, x, w, None, None, False, eps)
    good = [0, 1, 3, 4]
    y, _ = up.norm_rope_forward(x, None, w, None, eps=0.0)
    assert y[0, 0, 2].isnan().all()
    _check(y[:, :, good], x[:, :, good], w, None, None, eps=0.0)
    dx, _, _, _ = up.norm_rope_backward(dy, None, x, None, w, None, eps=0.0)
    assert dx[0, 0, 2].isnan().all() and dx[0, 0, good].isfinite().all()


def test_append_of_small_heads():
    """The cache gets what the forward gives; v is not normed."""
    k = (_bf(2, 1, 2, 64, seed=1) * 2.0 ** -90).to(torch.bfloat16)
    v = torch.zeros_like(k)
    w = _weights(64, False, 2)
    kp, vp = torch.zeros(2, 16, 2, 64, dtype=k.dtype, device=DEV), torch.ones(2, 16, 2, 64, dtype=k.dtype,
                                                                             device=DEV)
    table = torch.tensor([[0], [1]], dtype=torch.int32, device=DEV)
    lens = torch.tensor([1, 5], dtype=torch.int32, device=DEV)
    up.kv_append(k, v, kp, vp, table, lens, k_weight=w, eps=0.0)
    want, _ = up.norm_rope_forward(k, None, w, None, eps=0.0)
    _check(want, k, w, None, None, eps=0.0)
    assert torch.equal(kp[0, 0], want[0, 0]) and torch.equal(kp[1, 4], want[1, 0])
    assert not vp[0, 0].any() and not vp[1, 4].any() and (vp[0, 1:] == 1).all()
