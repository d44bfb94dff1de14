"""Head norms in calls long enough for eight heads a thread (needs an sm_103a GPU): forward and append from
152 * 1536 chunks of 16 features (tokens * heads * ceil(D / 16)), the backward from 152 * 1024.

Tolerances as in test_gpu_norm_rope.py. An element of dw is the sum of a thread's eight heads a token, at
most four tokens of a walker here, up to 128 sets of a block, 19 blocks a run and 5 joins: under 2^8
roundings of 2^-24, with the terms' own errors under 2^-15 of the sum of the magnitudes.
"""
import numpy as np
import pytest
import torch

import context_parallelism_gb300 as up
from tests.test_gpu_norm_rope import _bf, _check, _check_back, _weights
from tests.test_gpu_paged import Batch

pytestmark = pytest.mark.gpu
DEV = "cuda"

SHAPES = [  # B, S, Hq, Hkv, D, rot
    (1, 1500, 17, 3, 128, 128), (2, 1000, 9, 2, 192, 96), (1, 3000, 13, 3, 80, 80), (3, 833, 16, 8, 64, 32),
    (1, 700, 20, 1, 256, 16), (1, 2000, 12, 3, 128, 0), (1, 1300, 33, 3, 72, 48), (1, 260, 25, 4, 512, 64),
]


def _long(shape, border, extra=0):
    B, S, Hq, Hkv, D, _ = shape
    assert B * S * (Hq + Hkv + extra) * ((D + 15) // 16) >= 152 * border


@pytest.mark.parametrize("wide,offset,given", [(False, 0.0, False), (True, 1.0, True)])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("shape", SHAPES)
def test_forward_and_backward(shape, inter, wide, offset, given):
    _long(shape, 1536)
    B, S, Hq, Hkv, D, rot = shape
    q, k = _bf(B, S, Hq, D, seed=1), _bf(B, S, Hkv, D, seed=2, scale=8.0)
    qw, kw = _weights(D, wide, 3, offset), _weights(D, wide, 4, offset)
    ph = up.rope_phases(rot, theta=500000.0)[0] if rot else None
    how = dict(phases=ph, mscale=1.25, interleaved=inter, offset=offset)
    pos = np.tile(1000 + np.arange(S), (B, 1))
    if given:
        pos = np.random.default_rng(5).integers(-(1 << 20), 1 << 40, (B, S))
        how["positions"] = torch.from_numpy(pos).to(DEV)
    else:
        how["start"] = 1000
    y, z = up.norm_rope_forward(q, k, qw, kw, **how)
    ref = (pos, ph, 1.25, inter, 1e-6, offset)
    _check(y, q, qw, *ref)
    _check(z, k, kw, *ref)
    dy, dz = _bf(B, S, Hq, D, seed=5), _bf(B, S, Hkv, D, seed=6)
    dq, dk, dqw, dkw = up.norm_rope_backward(dy, dz, q, k, qw, kw, **how)
    _check_back(dq, dqw, dy, q, qw, *ref)
    _check_back(dk, dkw, dz, k, kw, *ref)
    again = up.norm_rope_backward(dy, dz, q, k, qw, kw, **how, inplace=True)
    assert again[0] is dy and torch.equal(dy, dq) and torch.equal(dz, dk)
    assert torch.equal(again[2], dqw) and torch.equal(again[3], dkw)
    up.norm_rope_forward(q, k, qw, kw, **how, inplace=True)
    assert torch.equal(q, y) and torch.equal(k, z)


@pytest.mark.parametrize("inter", [False, True])
def test_inside_a_projection(inter):
    """Heads of one fused tensor, one tensor without weights; a head-major gradient."""
    B, S, Hq, Hkv, D = 2, 1024, 14, 2, 128
    _long((B, S, Hq, Hkv, D, D), 1536)
    x = _bf(B, S, (Hq + 2 * Hkv) * D, seed=1)
    q = x[..., :Hq * D].unflatten(-1, (Hq, D))
    k = x[..., Hq * D:(Hq + Hkv) * D].unflatten(-1, (Hkv, D))
    kw = _weights(D, False, 3)
    ph, _ = up.rope_phases(D)
    pos = np.tile(np.arange(S), (B, 1))
    y, z = up.norm_rope_forward(q, k, None, kw, ph, interleaved=inter)
    _check(y, q, None, pos, ph, inter=inter)
    _check(z, k, kw, pos, ph, inter=inter)
    dy = _bf(B, Hq, S, D, seed=4).transpose(1, 2)
    dz = _bf(B, S, 1, D, seed=5).expand(B, S, Hkv, D)
    dq, dk, dqw, dkw = up.norm_rope_backward(dy, dz, q, k, None, kw, ph, interleaved=inter)
    _check_back(dq, dqw, dy, q, None, pos, ph, inter=inter)
    _check_back(dk, dkw, dz, k, kw, pos, ph, inter=inter)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("packed", [False, True])
def test_append_of_a_prompt(packed, inter):
    """Prompts of several sequences, rows behind the last one where they are packed: the cache and q hold
    what the forward gives, v is copied, other slots stay."""
    Hq, Hkv, D = 16, 3, 128
    counts = [750, 1, 0, 611] if packed else [670, 670]
    lens = [755, 40, 9, 611] if packed else [670, 797]
    b = Batch(counts, lens, Hq, Hkv, D, 48, 0, seed=3, packed=packed, behind=5)
    lead = b.q.shape[:-2]
    k, v = _bf(*lead, Hkv, D, seed=4), _bf(*lead, Hkv, D, seed=5)
    _long((1, k.numel() // (Hkv * D), Hq, Hkv, D, 0), 1536, Hkv)
    qw, kw = _weights(D, True, 6), _weights(D, True, 7)
    ph, _ = up.rope_phases(64)
    flat = lambda t: t.reshape(1, -1, *t.shape[-2:])  # noqa: E731
    pos, row = torch.zeros(flat(k).shape[:2], dtype=torch.int64), 0
    for n, ln in zip(counts, lens):
        pos[0, row:row + n] = 50 + ln - n + torch.arange(n)
        row += n
    how = dict(phases=ph, mscale=1.5, interleaved=inter, offset=0.5, eps=1e-5)
    qn, kn = up.norm_rope_forward(flat(b.q), flat(k), qw, kw, positions=pos.to(DEV), **how)
    _check(qn, flat(b.q), qw, pos.numpy(), ph, 1.5, inter, 1e-5, 0.5)
    kp, vp, kp2, vp2 = b.kp.clone(), b.vp.clone(), b.kp.clone(), b.vp.clone()
    qo = torch.full_like(b.q, 7.0)
    up.kv_append(k, v, kp, vp, b.table, b.seq_len, q=b.q, q_out=qo, cu_seqlens=b.cu, q_weight=qw,
                 k_weight=kw, start=50, **how)
    up.upipe_sync_status()
    up.kv_append(kn.view(k.shape), v, kp2, vp2, b.table, b.seq_len, cu_seqlens=b.cu)
    bits = lambda t: t.contiguous().view(torch.int16)  # noqa: E731
    assert torch.equal(bits(kp), bits(kp2)) and torch.equal(bits(vp), bits(vp2))
    assert torch.equal(flat(qo)[0, :row], qn[0, :row]) and (flat(qo)[0, row:] == 7.0).all()
