"""Refusals of the token-embedding calls, all before any device access (no GPU)."""
import pytest
import torch

import context_parallelism_gb300 as up

FAKE = 1 << 20  # an aligned non-null address; validation must fail before it is dereferenced
INV, UNS, OK = up.UPIPE_ERR_INVALID_ARG, up.UPIPE_ERR_UNSUPPORTED, up.UPIPE_OK
SMALL = up.UPIPE_ERR_WORKSPACE_TOO_SMALL


def _fwd(token=FAKE, w=FAKE, h=FAKE, S=5, Dm=64, V=100, scale=1.0):
    return up._lib.upipe_embed_fwd(token, w, h, S, Dm, V, scale, None)


def _bwd(token=FAKE, dh=FAKE, dw=FAKE, S=5, Dm=64, V=100, scale=1.0, add=0, ws=FAKE, wb=1 << 40):
    return up._lib.upipe_embed_bwd(token, dh, dw, S, Dm, V, scale, add, ws, wb, None)


SIZES = [(dict(S=-1), INV), (dict(Dm=0), INV), (dict(V=0), INV), (dict(Dm=60), UNS), (dict(Dm=(1 << 24) + 8), UNS),
         (dict(S=(1 << 30) + 1), UNS), (dict(V=1 << 31), UNS), (dict(scale=float("nan")), INV),
         (dict(scale=float("inf")), INV), (dict(S=1 << 30, Dm=1 << 20), UNS),
         (dict(token=None), INV), (dict(token=FAKE + 4), INV), (dict(), INV)]  # no device memory


@pytest.mark.parametrize("kw,status", SIZES + [(dict(w=None), INV), (dict(h=FAKE + 8), INV)])
def test_forward_refusals(kw, status):
    assert _fwd(**kw) == status, up.upipe_last_error_message()
    assert up.upipe_last_error_message()


@pytest.mark.parametrize("kw,status", SIZES + [
    (dict(dh=None), INV), (dict(dw=None), INV), (dict(dw=FAKE + 8), INV), (dict(add=2), INV),
    (dict(ws=None), INV), (dict(ws=FAKE + 16), INV), (dict(wb=255), SMALL),
    (dict(S=0, dw=None), INV),
])
def test_backward_refusals(kw, status):
    assert _bwd(**kw) == status, up.upipe_last_error_message()
    assert up.upipe_last_error_message()


def test_calls_without_tokens():
    assert _fwd(S=0, token=None) == OK and _bwd(S=0, add=1, dw=None, ws=None, wb=0) == OK


def test_workspace():
    """Two orders of the tokens and their places, counts, a bit for each row of the table, and at most
    two partial rows for each chunk of 8 places or more."""
    ws = up.upipe_embed_workspace_bytes
    for S, Dm, V in [(1, 8, 1), (4097, 1000, 32003), (131072, 4096, 128256), (1 << 20, 512, 1 << 20)]:
        tiles = -(-S // 2048) + 1
        most = 16 * S + tiles * 512 * 4 + V // 8 + 4 + -(-S // 8) * 2 * Dm * 4 + 7 * 256
        assert 16 * S < ws(S, Dm, V) <= most
    assert ws(131072, 4096, 128256) < 80 << 20
    for bad in ((0, 64, 100), (5, 0, 100), (5, 64, 0), (5, 60, 100), (5, 64, 1 << 31)):
        assert ws(*bad) == 0


def test_binding_refusals():
    t, w = torch.zeros((2, 3), dtype=torch.int64), torch.zeros((9, 16), dtype=torch.bfloat16)
    dh = torch.zeros((2, 3, 16), dtype=torch.bfloat16)
    for bad in (lambda: up.embed_forward(t.int(), w), lambda: up.embed_forward(t, w.float()),
                lambda: up.embed_backward(t, dh.float(), 9),
                lambda: up.embed_backward(t, dh, 9, dw=w)):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: up.embed_forward(t.t(), w), lambda: up.embed_forward(t, w.t()),
                lambda: up.embed_forward(t, dh), lambda: up.embed_backward(t, dh[0], 9),
                lambda: up.embed_backward(t[:, :2], dh, 9),
                lambda: up.embed_backward(t, dh, 9, dw=w.float()[:8])):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(up.UpipeError):  # host memory
        up.embed_forward(t, w)
