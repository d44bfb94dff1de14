"""Pins of the rotary and paged-attention oracles, and of the host arithmetic of the rotary
frequencies (no GPU)."""
import math

import numpy as np
import pytest

import context_parallelism_gb300 as up
from oracle import attn_fwd_ref, paged_attn_ref, rope_ref


def _phases(rot, **kw):
    f, m = up.upipe_rope_frequencies(rot, **kw)
    return f, up.upipe_rope_phases(f), m


@pytest.mark.parametrize("rot", [16, 64, 128])
def test_plain_frequencies(rot):
    f, _, m = _phases(rot, theta=500000.0)
    want = [500000.0 ** (-2 * i / rot) for i in range(rot // 2)]
    assert m == 1.0 and np.allclose(f, want, rtol=1e-15)


def test_scaled_frequencies():
    plain, _, _ = _phases(64)
    lin, _, m = _phases(64, scaling=up.UPIPE_ROPE_LINEAR, factor=4.0)
    assert m == 1.0 and np.allclose(lin, np.array(plain) / 4, rtol=1e-15)
    ntk, _, m = _phases(64, scaling=up.UPIPE_ROPE_NTK, factor=4.0)
    # the fastest pair keeps its frequency, the slowest is slowed by the whole factor
    assert m == 1.0 and ntk[0] == 1.0 and ntk[-1] == pytest.approx(plain[-1] / 4, rel=1e-12)
    parts, _, m = _phases(64, scaling=up.UPIPE_ROPE_BY_PARTS, factor=4.0, trained_len=4096)
    turns = 4096 * np.array(plain) / (2 * math.pi)
    assert m == pytest.approx(0.1 * math.log(4.0) + 1, rel=1e-15)
    assert np.allclose(np.array(parts)[turns > 32], np.array(plain)[turns > 32], rtol=1e-15)
    assert np.allclose(np.array(parts)[turns < 1], np.array(plain)[turns < 1] / 4, rtol=1e-15)
    mid = (turns > 1) & (turns < 32)
    assert mid.any() and (np.array(parts)[mid] < np.array(plain)[mid]).all()
    assert (np.array(parts)[mid] > np.array(plain)[mid] / 4).all()


def test_phases_are_fractions_of_a_turn():
    w = up.upipe_rope_phases([0.0, math.pi, math.pi / 2, 2 * math.pi, -math.pi / 2, 7 * math.pi])
    # pi rounds to a double just below or above: compare to 2^-50 of a turn
    for got, turns in zip(w, (0.0, 0.5, 0.25, 0.0, 0.75, 0.5)):
        d = (got / 2.0 ** 64 - turns) % 1.0
        assert min(d, 1 - d) < 2.0 ** -50


@pytest.mark.parametrize("args", [
    dict(rot_dim=0), dict(rot_dim=7), dict(rot_dim=16, theta=1.0), dict(rot_dim=16, theta=math.nan),
    dict(rot_dim=16, scaling=4), dict(rot_dim=16, scaling=1, factor=0.5),
    dict(rot_dim=2, scaling=2, factor=2.0),
    dict(rot_dim=16, scaling=3, factor=2.0, trained_len=0.0),
    dict(rot_dim=16, scaling=3, factor=2.0, trained_len=64.0, turns_fast=1.0, turns_slow=1.0),
])
def test_frequency_refusals(args):
    with pytest.raises(up.UpipeError) as e:
        up.upipe_rope_frequencies(**args)
    assert e.value.status == up.UPIPE_ERR_INVALID_ARG


def test_phase_refusals():
    for f in ([], [math.inf], [0.1, math.nan]):
        with pytest.raises(up.UpipeError):
            up.upipe_rope_phases(f)


@pytest.mark.parametrize("inter", [False, True])
def test_rope_oracle_angles_and_norm(inter):
    f, ph, _ = _phases(32)
    rng = np.random.default_rng(1)
    x = rng.standard_normal((3, 2, 48))
    pos = [0, 7, 123456]
    y = rope_ref(x, pos, ph, 1.0, inter)
    assert np.array_equal(y[0], x[0]) and np.array_equal(y[..., 32:], x[..., 32:])
    assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1), rtol=1e-12)
    for s in range(3):
        for i in range(16):
            a, b = (2 * i, 2 * i + 1) if inter else (i, 16 + i)
            c, d = math.cos(pos[s] * f[i]), math.sin(pos[s] * f[i])
            # the phase is the frequency truncated to 2^-64 of a turn and rounded to 53 bits
            assert np.allclose(y[s, :, a], x[s, :, a] * c - x[s, :, b] * d, atol=1e-9)
            assert np.allclose(y[s, :, b], x[s, :, b] * c + x[s, :, a] * d, atol=1e-9)


@pytest.mark.parametrize("inter", [False, True])
def test_rope_oracle_gradient_against_differences(inter):
    _, ph, _ = _phases(16)
    rng = np.random.default_rng(2)
    x, dy = rng.standard_normal((2, 1, 24)), rng.standard_normal((2, 1, 24))
    pos = [5, 1 << 40]
    dx = rope_ref(dy, pos, ph, 1.25, inter, back=True)
    # with mscale the tail's gradient is copied, as the tail is
    for at in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[at] = 1e-4
        num = ((rope_ref(x + e, pos, ph, 1.25, inter) -
                rope_ref(x - e, pos, ph, 1.25, inter)) * dy).sum() / 2e-4
        assert dx[at] == pytest.approx(num, abs=1e-9)


def _cache(rng, pages, ps, H, D):
    return rng.standard_normal((pages, ps, H, D)), rng.standard_normal((pages, ps, H, D))


def test_paged_oracle_is_causal_attention_on_one_sequence():
    rng = np.random.default_rng(3)
    S, Hq, Hkv, D, ps = 37, 4, 2, 8, 16
    kp, vp = _cache(rng, 5, ps, Hkv, D)
    table = np.array([[3, 1, 4]])
    k = kp[[3, 1, 4]].reshape(-1, Hkv, D)[:S]
    v = vp[[3, 1, 4]].reshape(-1, Hkv, D)[:S]
    q = rng.standard_normal((S, Hq, D))
    ro, rl = attn_fwd_ref(q[None], k[None], v[None], causal=True)
    o, lse, _, _ = paged_attn_ref(q, kp, vp, table, [S], [S])
    assert np.allclose(o, ro[0], atol=1e-13) and np.allclose(lse, rl[0].T, atol=1e-13)
    # its last rows alone, as a step after the others
    o2, lse2, _, _ = paged_attn_ref(q[-5:], kp, vp, table, [S], [5])
    assert np.allclose(o2, o[-5:], atol=1e-13) and np.allclose(lse2, lse[-5:], atol=1e-13)
    # the same keys with the first 20 as a shared prefix in pages of their own
    kp2, vp2 = _cache(rng, 9, ps, Hkv, D)
    kp2[[7, 2]].reshape(-1, Hkv, D)
    for c2, c in ((kp2, k), (vp2, v)):
        c2[7], c2[2, :4] = c[:16], c[16:20]
        c2[0], c2[5, :1] = c[20:36], c[36:37]
    o3, lse3, _, _ = paged_attn_ref(q[-5:], kp2, vp2, np.array([[0, 5]]), [S - 20], [5],
                                    [7, 2], 20)
    assert np.allclose(o3, o2, atol=1e-13) and np.allclose(lse3, lse2, atol=1e-13)


def test_paged_oracle_rows_without_keys_and_spread():
    rng = np.random.default_rng(4)
    kp, vp = _cache(rng, 2, 16, 1, 8)
    q = rng.standard_normal((3, 2, 8))
    o, lse, spread, _ = paged_attn_ref(q, kp, vp, np.array([[0], [1]]), [1, 0], [2, 1])
    assert (o[0] == 0).all() and np.isneginf(lse[0]).all()     # before its sequence's first key
    assert np.allclose(o[1], vp[0, 0]) and np.allclose(spread[1], 0)  # one key: its value
    assert (o[2] == 0).all() and np.isneginf(lse[2]).all()
