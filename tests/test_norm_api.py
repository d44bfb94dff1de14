"""Refusals of the calls with head norms, all before any device access (no GPU)."""
import ctypes

import pytest
import torch

import context_parallelism_gb300 as up
from tests.test_paged_api import C, FAKE, H

INV, UNS = up.UPIPE_ERR_INVALID_ARG, up.UPIPE_ERR_UNSUPPORTED
SMALL = up.UPIPE_ERR_WORKSPACE_TOO_SMALL


def N(qw=FAKE, kw=FAKE, offset=0.0, eps=1e-6, wide=0):
    return up.Norm(qw, kw, offset, eps, wide)


def _fwd(q=H(), k=None, q_out=H(), k_out=None, norm=N(), pos=None, phase=FAKE, mscale=1.0, B=1,
         S=8, D=64, rot=64, inter=0):
    return up._lib.upipe_norm_rope_fwd(q, k, q_out, k_out, norm, pos, 0, phase, mscale, B, S, D, rot,
                                       inter, None)


def _bwd(dqo=H(), dko=None, q=H(), k=None, dq=H(), dk=None, dqw=FAKE, dkw=None, norm=N(), pos=None,
         phase=FAKE, mscale=1.0, B=1, S=8, D=64, rot=64, inter=0, ws=FAKE, wb=1 << 40):
    return up._lib.upipe_norm_rope_bwd(dqo, dko, q, k, dq, dk, dqw, dkw, norm, pos, 0, phase, mscale,
                                       B, S, D, rot, inter, ws, wb, None)


def _append(norm=N(), q=H(4), q_out=H(4), k=H(2), v=H(2), cache=None, B=2, S=1, rot=64, phase=FAKE):
    return up._lib.upipe_kv_append_norm(q, q_out, k, v, norm, cache if cache is not None else C(),
                                        FAKE, 4, 4, FAKE, None, None, 0, phase, 1.0, B, S, rot, 0,
                                        None)


BOTH = [
    (dict(norm=None), INV), (dict(norm=N(eps=-1e-6)), INV), (dict(norm=N(eps=float("nan"))), INV),
    (dict(norm=N(eps=float("inf"))), INV), (dict(norm=N(offset=float("inf"))), INV),
    (dict(norm=N(wide=2)), INV), (dict(norm=N(qw=FAKE + 8)), INV),
    (dict(D=520, rot=64), UNS), (dict(D=60), UNS), (dict(rot=24), UNS), (dict(rot=80), UNS),
    (dict(inter=2), INV), (dict(mscale=float("inf")), INV), (dict(B=-1), INV),
    (dict(S=1 << 41), UNS), (dict(pos=FAKE + 4), INV), (dict(phase=FAKE + 8), INV),
    (dict(phase=None, D=4), UNS), (dict(), INV), (dict(phase=None, rot=0), INV),  # no device memory
]


@pytest.mark.parametrize("kw,status", BOTH + [
    (dict(q=None), INV), (dict(q_out=None), INV), (dict(q_out=H(5)), INV), (dict(q=H(ss=260)), INV),
    (dict(q_out=H(ss=0)), INV), (dict(q=H(data=FAKE + 2)), INV), (dict(k=H(), k_out=H()), INV),
    (dict(q=H(70000), q_out=H(70000)), UNS),
])
def test_forward_refusals(kw, status):
    assert _fwd(**kw) == status, up.upipe_last_error_message()
    assert up.upipe_last_error_message()


@pytest.mark.parametrize("kw,status", BOTH + [
    (dict(dqo=None), INV), (dict(dq=None), INV), (dict(dq=H(3)), INV), (dict(q=None), INV),
    (dict(q=H(5)), INV), (dict(q=H(data=FAKE + 2)), INV), (dict(q=H(ss=4)), INV),
    (dict(dq=H(sh=8)), INV), (dict(norm=N(qw=None)), INV),     # a gradient without the weights
    (dict(dkw=FAKE), INV), (dict(dqw=FAKE + 2), INV), (dict(ws=None), INV),
    (dict(ws=FAKE + 16), INV), (dict(wb=255), SMALL), (dict(dqo=H(70000), q=H(70000), dq=H(70000)), UNS),
])
def test_backward_refusals(kw, status):
    assert _bwd(**kw) == status, up.upipe_last_error_message()
    assert up.upipe_last_error_message()


@pytest.mark.parametrize("kw,status", [
    (dict(norm=None), INV), (dict(norm=N(eps=-1.0)), INV), (dict(norm=N(kw=FAKE + 4)), INV),
    (dict(cache=C(D=520, stride_head=520, stride_slot=1040, stride_page=16640), rot=64), UNS),
    (dict(k=None), INV), (dict(q_out=None), INV), (dict(rot=24), UNS), (dict(), INV),
])
def test_append_refusals(kw, status):
    assert _append(**kw) == status, up.upipe_last_error_message()
    assert up.upipe_last_error_message()


def test_calls_without_rows_do_nothing():
    assert _fwd(S=0) == up.UPIPE_OK and _append(B=0) == up.UPIPE_OK
    assert _bwd(S=0, dqw=None, ws=None, wb=0) == up.UPIPE_OK


def test_workspace():
    """2 D partial sums for each of at most 608 blocks (more where the heads alone ask for more)."""
    ws = up.upipe_norm_rope_workspace_bytes
    assert ws(1, 1 << 30, 32, 8, 128) == 608 * 2 * 128 * 4
    assert 0 < ws(1, 1, 1, 0, 64) <= 608 * 2 * 64 * 4
    # a block for each four groups of eight heads at least
    assert ws(1, 1, 65536, 0, 512) == 65536 // 8 // 4 * 2 * 512 * 4
    for bad in ((0, 1, 4, 1, 64), (1, 0, 4, 1, 64), (1, 1, 0, 0, 64), (1, 1, 65536, 1, 64),
                (1, 1, 4, 1, 60), (1, 1, 4, 1, 520), (2, 1 << 40, 4, 1, 64), (1, 1, -1, 3, 64)):
        assert ws(*bad) == 0
    assert ctypes.sizeof(up.Norm) == 40


def test_binding_refusals():
    q, k, w = (torch.zeros(s, dtype=torch.bfloat16) for s in ((1, 3, 4, 64), (1, 3, 2, 64), (64,)))
    ph = torch.zeros(32, dtype=torch.int64)
    kp = torch.zeros((4, 16, 2, 64), dtype=torch.bfloat16)
    table, lens = torch.zeros((1, 2), dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    for bad in (lambda: up.norm_rope_forward(None, None, w, w),
                lambda: up.norm_rope_forward(q, k[:, :2], w, w),
                lambda: up.norm_rope_forward(q, k, w[:32], w),
                lambda: up.norm_rope_forward(q, k, w, w.expand(2, 64)),
                lambda: up.norm_rope_forward(q, k, w, w, ph.int()),
                lambda: up.norm_rope_forward(q, k, w, w, positions=torch.zeros(3)),
                lambda: up.norm_rope_backward(q, k, q[:, :2], k, w, w),
                lambda: up.norm_rope_backward(q, k, q, k.expand(2, 3, 2, 64), w, w),
                lambda: up.kv_append(k, k, kp, kp.clone(), table, lens, k_weight=w)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: up.norm_rope_forward(q.float(), k, w, w),
                lambda: up.norm_rope_forward(q, k, w.half(), w),
                lambda: up.norm_rope_forward(q, k, w.float(), w)):
        with pytest.raises(TypeError):
            bad()
    for call in (lambda: up.norm_rope_forward(q, k, w, w, ph),  # host memory
                 lambda: up.norm_rope_backward(q, k, q, k, w, w, ph, inplace=True)):
        with pytest.raises(up.UpipeError):
            call()
