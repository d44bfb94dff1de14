"""How the token log probabilities add up a logit's products, and sizes that only long calls have (needs an
sm_103a GPU).

An fp32 sum that a tensor core carries on is cut at 2^-23 of itself at every step of 16 products, so that
what is below that beside a large sum is lost, however much of it there is. The products here are powers of
two: the first sixteen add up to 16, each later step to 2^-20, half of the last bit of 16. In pieces of 64
(up to 16 tokens) or 512 products every piece's sum is exact, and so is each addition of a piece to the
others, a multiple of 2^-19 each; carried on in one sum, or in pieces twice as long, 28 steps of 2^-20 and
more are lost, 2.6e-5. What is left to round: the exponentials (2^-22 of each) and the sum z of equal ones
(2^-15 of ln z, as in test_gpu_logp.py, where ln z - ln count is 5e-5 and below), the sum of the two (half a
step of 16, 2^-20) and, for a target whose logit is 0, as much again.
"""
import math

import pytest
import torch

import context_parallelism_gb300 as up
from tests.test_gpu_logp import _check, _inputs

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


@pytest.mark.parametrize("Dm", [512, 1024, 4096, 4104])
@pytest.mark.parametrize("S,piece", [(1, 64), (16, 64), (17, 512), (130, 512)])
def test_small_products_beside_large_ones(S, piece, Dm):
    V, at = 700, 432
    w = torch.zeros((V, Dm), device=DEV)
    w[at, 0] = 16.0
    w[at, piece:] = 2.0 ** -24
    h = torch.ones((S, Dm), device=DEV).to(BF)
    target = torch.full((S,), 5, device=DEV)
    target[0] = at
    logp, entropy, lse, tl, ti = up.token_logprobs(h, w.to(BF), target, top=2)
    x = 16.0 + max(Dm - piece, 0) * 2.0 ** -24
    q = (V - 1) * math.exp(-x)
    ln = math.log1p(q)
    assert ((lse.double() - (x + ln)).abs() <= 2.0 ** -20 + 2.0 ** -15 * ln).all()
    assert abs(logp[0].item() + ln) <= 2.0 ** -15 * ln and tl[0, 0] == logp[0]
    assert ((logp[1:].double() + x + ln).abs() <= 2.0 ** -19 + 2.0 ** -15 * ln).all()
    assert ((tl[:, 1].double() + x + ln).abs() <= 2.0 ** -19 + 2.0 ** -15 * ln).all()
    # H = ln(1 + q) + q x / (1 + q): a change of x by d moves it by about q x d
    assert ((entropy.double() - (ln + q * x / (1 + q))).abs() <= 2.0 ** -15 * (1 + x) * ln).all()
    assert (ti == torch.tensor([at, 0], device=DEV)).all()


@pytest.mark.parametrize("S,V,top", [(4500, 700, 5), (4097, 300, 0), (8400, 129, 24)])
def test_more_than_32_tiles_of_tokens(S, V, top):
    """128 tokens a tile; the kernel walks 32 of them together, here two and three such groups, the last
    of them short."""
    h, w, t = _inputs(S, 72, V, seed=S)
    got = up.token_logprobs(h, w, t, top=top, seq_tile=8448)
    up.upipe_sync_status()
    _check(got, h, w, t, top)
    parts = up.token_logprobs(h, w, t, top=top, seq_tile=4096)
    assert top == 0 or torch.equal(got[4], parts[4])


@pytest.mark.parametrize("S", [1, 16, 130])
@pytest.mark.parametrize("V", [45613, 128256])
def test_many_equal_logits(S, V):
    """More groups, and more logits, at the maximum than are ranked one against the other: a row of zeros,
    and one whose larger half is all the same."""
    h, w, t = _inputs(S, 64, V)
    h[0] = 0
    w[:, 0] = 0
    w[1001::2, 0] = 3.0
    if S > 1:
        h[1] = 0
        h[1, 0] = 1.0
    got = up.token_logprobs(h, w, t, top=24)
    up.upipe_sync_status()
    assert got[4][0].tolist() == list(range(24))
    assert got[1][0].item() == pytest.approx(math.log(V), rel=2.0 ** -20)
    assert (got[3][0] == -got[2][0]).all()
    if S > 1:
        assert got[4][1].tolist() == list(range(1001, 1049, 2))
        n = len(range(1001, V, 2))
        lse = 3 + math.log(n + (V - n) * math.exp(-3))
        assert got[2][1].item() == pytest.approx(lse, rel=2.0 ** -20)


@pytest.mark.parametrize("S", [3, 70])
def test_alternatives_are_valued_as_targets_are(S):
    """The value of an alternative is the log probability that the call gives the same token as a target,
    bit for bit; in the order of the exact sums, so that neighbours may be out of order by what the values
    lost: half a step of the logit and of the sum after it, twice."""
    h, w, _ = _inputs(S, 4096, 3000, seed=3)
    # pairs of rows that differ in the last bits of one small product
    w[1::2] = w[::2]
    w[1::2, 7] += (2.0 ** -12 * torch.randn(1500, device=DEV)).to(BF)
    _, _, lse, tl, ti = up.token_logprobs(h, w, None, top=20)
    for k in range(20):
        logp, _, lse2, tl2, ti2 = up.token_logprobs(h, w, ti[:, k].contiguous(), top=20)
        assert torch.equal(logp, tl[:, k]) and torch.equal(ti, ti2) and torch.equal(lse, lse2)
    x = h.double() @ w.double().t()
    exact = x.gather(1, ti)
    assert (exact[:, 1:] <= exact[:, :-1] + 2.0 ** -40 * x.abs().amax()).all()
    assert (tl <= 0).all()
