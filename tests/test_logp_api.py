"""Refusals of the token-log-probability call, all before any device access (no GPU)."""
import pytest
import torch

import context_parallelism_gb300 as up

FAKE = 1 << 20  # an aligned non-null address; validation must fail before it is dereferenced
INV, UNS, OK = up.UPIPE_ERR_INVALID_ARG, up.UPIPE_ERR_UNSUPPORTED, up.UPIPE_OK


def _call(h=FAKE, w=FAKE, target=FAKE, logp=FAKE, entropy=FAKE, lse=FAKE, tl=FAKE, ti=FAKE, S=5,
          Dm=64, V=100, top=3, tile=128, ws=FAKE, wb=1 << 50):
    return up._lib.upipe_logp_fwd(h, w, target, logp, entropy, lse, tl, ti, S, Dm, V, top, tile, ws,
                                  wb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(S=-1), INV), (dict(Dm=0), INV), (dict(V=0), INV), (dict(top=-1), INV), (dict(tile=0), INV),
    (dict(Dm=60), UNS), (dict(V=(1 << 30) + 1), UNS), (dict(top=25), UNS), (dict(tile=100), UNS),
    (dict(tile=1 << 25), UNS), (dict(Dm=(1 << 24) + 8), UNS),
    (dict(target=None), INV), (dict(logp=None), INV), (dict(tl=None), INV), (dict(ti=None), INV),
    (dict(top=0), INV), (dict(h=None), INV), (dict(w=None), INV), (dict(h=FAKE + 8), INV),
    (dict(ws=None), INV), (dict(ws=FAKE + 128), INV), (dict(target=FAKE + 4), INV),
    (dict(lse=FAKE + 2), INV), (dict(ti=FAKE + 4), INV), (dict(), INV),   # no device memory
    (dict(target=None, logp=None, entropy=None, lse=None), INV),          # the same
])
def test_refusals(kw, status):
    assert _call(**kw) == status, up.upipe_last_error_message()
    assert up.upipe_last_error_message()


def test_calls_without_tokens_do_nothing():
    assert _call(S=0, h=None, target=None, ws=None) == OK


def _groups(M, V):
    """Columns go in tiles of up to 128 (16 rows), else 256, as many rounds of 152 as those make, evenly."""
    most, m = (128, 1) if M <= 16 else (256, -(-M // 128))
    n = -(-m * -(-V // most) // 152) * 152 // m
    tile = max(16 if M <= 16 else 64, -(-V // n))
    tile = most if tile > most * 31 // 32 else tile
    return -(-V // tile) * (2 if tile > 128 else 1)


def test_workspace():
    """As documented: partial sums of the groups of columns, target logits, logits, slots."""
    al = lambda x: -(-x // 256) * 256  # noqa: E731
    for S, Dm, V, top, tile, host in [(1, 4096, 128256, 5, 4096, 0), (300, 64, 1000, 0, 128, 2),
                                      (70, 8, 1, 24, 128, 0), (131072, 4096, 128256, 20, 8192, 2),
                                      (64, 72, 2433, 1, 256, 0)]:
        T = min(S, tile)
        groups = max(m * _groups(m, V) for m in (T, S % T) if m)
        want = al(16 * groups) + al(4 * T)
        want += al(512 * groups) + al(4 * T * (top + 4)) if top else 0
        want += 2 * al(2 * T * Dm) if host else 0
        assert up.upipe_logp_workspace_bytes(S, Dm, V, top, tile, host) == want
    for bad in ((0, 64, 100, 1, 128), (5, 60, 100, 1, 128), (5, 64, 0, 1, 128), (5, 64, 100, 25, 128),
                (5, 64, 100, 1, 100)):
        assert up.upipe_logp_workspace_bytes(*bad) == 0
    assert up.upipe_logp_workspace_bytes(5, 64, 100, 1, 128, up.UPIPE_HOST_KV) == 0


def test_binding_refusals():
    h, w = torch.zeros((3, 16), dtype=torch.bfloat16), torch.zeros((9, 16), dtype=torch.bfloat16)
    t = torch.zeros(3, dtype=torch.int64)
    for bad in (lambda: up.token_logprobs(h[:, :8], w), lambda: up.token_logprobs(h, w[:, :8]),
                lambda: up.token_logprobs(h[None], w), lambda: up.token_logprobs(h, w, t[:2]),
                lambda: up.token_logprobs(h, w, t.int())):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: up.token_logprobs(h.float(), w), lambda: up.token_logprobs(h, w.float())):
        with pytest.raises(TypeError):
            bad()
