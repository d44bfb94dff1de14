"""fp64 CPU oracles of the head norms with the rotation, the token embedding and the token log
probabilities.

TEST INFRASTRUCTURE ONLY. Plain definitions, sharing no code with the CUDA path.

Norm: y = R (offset + w) x / sqrt(mean x^2 + eps), R the rotation of paged_ref.rope_ref. Its gradient
is written from the quotient rule on the whole head (the Jacobian of x -> x / |x|_rms), not from the
kernel's sums; the tests pin it against differences.
"""
from __future__ import annotations

import numpy as np

from .attn_ref import _f64
from .paged_ref import rope_ref

__all__ = ["norm_rope_ref", "norm_rope_bwd_ref", "embed_ref", "embed_bwd_ref", "logp_ref"]


def _turn(x, pos, phases, mscale, interleaved, back=False):
    if phases is None:
        return x
    return rope_ref(x, pos, phases, mscale, interleaved, back)


def norm_rope_ref(x, w, pos, phases, mscale=1.0, interleaved=False, eps=1e-6, offset=0.0):
    """x [..., S, H, D]; w [D] or None (ones); phases None: not rotated."""
    x = _f64(x)
    n = x / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps)
    if w is not None:
        n = n * (offset + _f64(w))
    return _turn(n, pos, phases, mscale, interleaved)


def norm_rope_bwd_ref(dy, x, w, pos, phases, mscale=1.0, interleaved=False, eps=1e-6, offset=0.0):
    """dx, dw (None without w) of <dy, norm_rope_ref(x)>, and what the tests' tolerances take: the
    size of the terms of each dx and of the sum in each dw."""
    x, dy = _f64(x), _f64(dy)
    D = x.shape[-1]
    g = _turn(dy, pos, phases, mscale, interleaved, True)
    ga = np.abs(g)
    if phases is not None:  # both products of each pair
        rot = 2 * len(phases)
        d = np.abs(dy) * mscale
        s = (d[..., 0:rot:2] + d[..., 1:rot:2] if interleaved
             else d[..., :rot // 2] + d[..., rot // 2:rot])
        if interleaved:
            ga[..., 0:rot:2], ga[..., 1:rot:2] = s, s
        else:
            ga[..., :rot // 2], ga[..., rot // 2:rot] = s, s
    scale = np.ones(D) if w is None else offset + _f64(w)
    rms = np.sqrt((x ** 2).mean(-1, keepdims=True) + eps)
    t = g * scale
    # d(x_j / rms) / d x_i = [i == j] / rms - x_j x_i / (D rms^3)
    dx = t / rms - x * (t * x).sum(-1, keepdims=True) / (D * rms ** 3)
    ta = ga * np.abs(scale)
    size = ta / rms + np.abs(x) * (ta * np.abs(x)).sum(-1, keepdims=True) / (D * rms ** 3)
    if w is None:
        return dx, None, size, None
    axes = tuple(range(x.ndim - 1))
    return dx, (g * x / rms).sum(axes), size, (ga * np.abs(x) / rms).sum(axes)


def embed_ref(tokens, w, scale=1.0):
    """scale * w[token]; zeros for a negative token, NaN for one outside the table."""
    t, w = np.asarray(tokens), _f64(w)
    h = np.zeros(t.shape + w.shape[1:])
    for at in np.ndindex(t.shape):
        if t[at] >= w.shape[0]:
            h[at] = np.nan
        elif t[at] >= 0:
            h[at] = scale * w[t[at]]
    return h


def embed_bwd_ref(tokens, dh, V, scale=1.0):
    """The gradient of the table, and the sum of the magnitudes in each of its elements."""
    t, dh = np.asarray(tokens).reshape(-1), _f64(dh)
    dh = dh.reshape(-1, dh.shape[-1])
    dw, size = np.zeros((V, dh.shape[1])), np.zeros((V, dh.shape[1]))
    for i, v in enumerate(t):
        if 0 <= v < V:
            dw[v] += scale * dh[i]
            size[v] += abs(scale) * np.abs(dh[i])
    return dw, size


def logp_ref(h, w, target=None, top=0):
    """logp [S] (None without target; 0 for a negative target, NaN for one outside), entropy [S],
    lse [S], top_logp [S, top], top_index [S, top] (the largest logits, equal ones by index)."""
    x = _f64(h) @ _f64(w).T
    S, V = x.shape
    m = x.max(-1, keepdims=True)
    e = np.exp(x - m)
    z = e.sum(-1, keepdims=True)
    lse = m + np.log(z)
    p = x - lse
    entropy = -np.where(e > 0, e / z * np.where(e > 0, p, 0.0), 0.0).sum(-1)
    logp = None
    if target is not None:
        logp = np.array([0.0 if t < 0 else np.nan if t >= V else p[i, t]
                         for i, t in enumerate(np.asarray(target))])
    order = np.argsort(-x, axis=-1, kind="stable")[:, :top]
    return logp, entropy, lse[:, 0], np.take_along_axis(p, order, -1), order
