"""Pins of the oracles of the head norms, the token embedding and the token log probabilities (no
GPU)."""
import math

import numpy as np
import pytest
import torch

import context_parallelism_gb300 as up
from oracle import (ce_loss_bwd_ref, ce_loss_ref, embed_bwd_ref, embed_ref, logp_ref,
                    norm_rope_bwd_ref, norm_rope_ref, rope_ref)


def _phases(rot):
    return up.upipe_rope_phases(up.upipe_rope_frequencies(rot)[0])


def _rand(*shape, seed=0):
    return np.random.default_rng(seed).standard_normal(shape)


def test_norm_of_known_heads():
    x = np.array([3.0, 4.0, 0.0, 0.0])[None, None]
    y = norm_rope_ref(x, None, None, None, eps=0.0)
    assert np.allclose(y[0, 0], [1.2, 1.6, 0, 0])          # rms 2.5
    assert np.allclose(norm_rope_ref(1e30 * x, None, None, None), y, rtol=1e-12)
    y = norm_rope_ref(x, np.array([1.0, 0.0, 2.0, 2.0]), None, None, eps=0.0, offset=1.0)
    assert np.allclose(y[0, 0], [2.4, 1.6, 0, 0])
    assert (norm_rope_ref(0 * x, None, None, None) == 0).all()


@pytest.mark.parametrize("inter", [False, True])
def test_norm_then_rotation(inter):
    """The rotation keeps a head's length, and is rope_ref's of the normed head."""
    x, w = _rand(2, 5, 3, 32), 1 + 0.1 * _rand(32, seed=1)
    pos = np.arange(10).reshape(2, 5) + 70
    ph = _phases(16)
    y = norm_rope_ref(x, w, pos, ph, 1.5, inter)
    flat = norm_rope_ref(x, w, None, None)
    assert np.allclose(y, rope_ref(flat, pos, ph, 1.5, inter), rtol=1e-13)
    assert np.allclose((norm_rope_ref(x, None, pos, ph, 1.0, inter, eps=0.0) ** 2).mean(-1), 1.0)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("offset", [0.0, 1.0])
def test_norm_gradient_against_differences(inter, offset):
    x, dy, w = _rand(1, 2, 2, 24), _rand(1, 2, 2, 24, seed=1), _rand(24, seed=2)
    pos, ph = np.array([[5, 900]]), _phases(16)

    def f(x, w):
        return (dy * norm_rope_ref(x, w, pos, ph, 1.3, inter, 1e-3, offset)).sum()

    dx, dw, size, dw_size = norm_rope_bwd_ref(dy, x, w, pos, ph, 1.3, inter, 1e-3, offset)
    h = 1e-6
    for at in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[at] = h
        assert (f(x + e, w) - f(x - e, w)) / (2 * h) == pytest.approx(dx[at], abs=1e-7)
    for i in range(24):
        e = np.zeros(24)
        e[i] = h
        assert (f(x, w + e) - f(x, w - e)) / (2 * h) == pytest.approx(dw[i], abs=1e-7)
    assert (size >= np.abs(dx) - 1e-12).all() and (dw_size >= np.abs(dw) - 1e-12).all()


def test_norm_gradient_closed_forms():
    """Without eps the norm does not see the head's length: dx is orthogonal to x."""
    x, dy = _rand(1, 4, 2, 16), _rand(1, 4, 2, 16, seed=1)
    dx, dw, _, _ = norm_rope_bwd_ref(dy, x, None, None, None, eps=0.0)
    assert np.allclose((dx * x).sum(-1), 0, atol=1e-12) and dw is None


def test_embedding():
    w = _rand(5, 3)
    t = np.array([[4, 0], [-1, 5]])
    h = embed_ref(t, w, 2.0)
    assert np.allclose(h[0], 2 * w[[4, 0]]) and (h[1, 0] == 0).all() and np.isnan(h[1, 1]).all()
    dh = _rand(6, 3, seed=1)
    t = np.array([2, 2, 7, -3, 0, 2])
    dw, size = embed_bwd_ref(t, dh, 5, 0.5)
    onehot = (t[:, None] == np.arange(5)).astype(float)
    assert np.allclose(dw, 0.5 * onehot.T @ dh) and np.allclose(size, 0.5 * onehot.T @ np.abs(dh))


def test_embedding_gradient_is_the_transpose():
    """<dh, embed(w)> = <embed_bwd(dh), w> for every w and dh."""
    w, dh = _rand(7, 4), _rand(9, 4, seed=1)
    t = np.random.default_rng(2).integers(-1, 7, 9)
    assert (dh * embed_ref(t, w, 3.0)).sum() == pytest.approx(
        (embed_bwd_ref(t, dh, 7, 3.0)[0] * w).sum(), rel=1e-12)


def test_logp_closed_forms():
    # equal logits: ln V, in order of the index
    logp, ent, lse, tl, ti = logp_ref(np.zeros((2, 3)), _rand(8, 3), [3, -1], 4)
    assert np.allclose(logp, [-math.log(8), 0]) and np.allclose(ent, math.log(8))
    assert np.allclose(lse, math.log(8)) and np.allclose(tl, -math.log(8))
    assert (ti == [0, 1, 2, 3]).all()
    # logits 0 and ln 3: probabilities 1/4 and 3/4
    logp, ent, lse, tl, ti = logp_ref([[math.log(3.0)]], [[0.0], [1.0]], [2], 2)
    assert np.isnan(logp).all() and lse[0] == pytest.approx(math.log(4))
    assert ent[0] == pytest.approx(math.log(4) - 0.75 * math.log(3))
    assert (ti == [[1, 0]]).all() and np.allclose(tl, np.log([[0.75, 0.25]]))


def test_logp_is_minus_the_loss():
    h, w, t = _rand(6, 5), _rand(11, 5, seed=1), np.array([0, 10, -1, 4, 4, 7])
    logp, ent, lse, _, _ = logp_ref(h, w, t)
    loss, l2 = ce_loss_ref(h, w, t)
    assert np.allclose(logp, -loss, rtol=1e-13) and np.allclose(lse, l2, rtol=1e-13)
    p = torch.distributions.Categorical(logits=torch.from_numpy(h @ w.T))
    assert np.allclose(ent, p.entropy().numpy(), rtol=1e-12)
    # the gradient of given log probabilities is the loss's for -g
    g = _rand(6, seed=2)
    hh = torch.from_numpy(h).requires_grad_()
    lp = torch.log_softmax(hh @ torch.from_numpy(w).T, -1)
    tot = sum(g[i] * lp[i, t[i]] for i in range(6) if t[i] >= 0)
    dh = ce_loss_bwd_ref(h, w, t, -g)[2]
    assert np.allclose(torch.autograd.grad(tot, hh)[0].numpy(), dh, rtol=1e-11)
