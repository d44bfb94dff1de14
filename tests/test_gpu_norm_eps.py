"""Gradients of the head norms with eps = 0 (needs an sm_103a GPU): sets of lanes that have no head left at
the end of a call add nothing to the weights' gradients, whatever eps is.

Tolerances as in test_gpu_norm_rope.py: a sum of dw has at most eight heads a thread and step, one or two
steps, up to 64 sets and 608 / 32 blocks a run and 5 joins here, under 2^7 roundings of 2^-24.
"""
import numpy as np
import pytest
import torch

import context_parallelism_gb300 as up
from tests.test_gpu_norm_rope import _bf, _check_back, _weights

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("eps", [0.0, 1e-60])
@pytest.mark.parametrize("B,S,Hq,Hkv,D,rot", [
    (1, 3, 2, 0, 64, 0),        # walkers without a token
    (2, 5, 3, 1, 128, 128),     # groups of two heads that are not full
    (1, 1, 1, 1, 8, 0), (1, 7, 5, 2, 192, 96), (3, 33, 7, 3, 80, 16),
    (1, 2600, 11, 3, 80, 0),    # groups of eight heads, none full
])
def test_sets_without_a_head(B, S, Hq, Hkv, D, rot, eps):
    ph = up.rope_phases(rot)[0] if rot else None
    pos = np.tile(np.arange(S), (B, 1))
    q, dq, qw = _bf(B, S, Hq, D, seed=1), _bf(B, S, Hq, D, seed=2), _weights(D, True, 3)
    k = dk = kw = None
    if Hkv:
        k, dk, kw = _bf(B, S, Hkv, D, seed=4), _bf(B, S, Hkv, D, seed=5), _weights(D, True, 6)
    for inter in (False, True):
        got = up.norm_rope_backward(dq, dk, q, k, qw, kw, ph, eps=eps, interleaved=inter)
        _check_back(got[0], got[2], dq, q, qw, pos, ph, inter=inter, eps=eps)
        if Hkv:
            _check_back(got[1], got[3], dk, k, kw, pos, ph, inter=inter, eps=eps)
