"""Token log probabilities on the GPU against the 64-bit oracle (needs an sm_103a GPU).

Tolerances. A logit is a sum of Dm products, which the tensor cores add to an fp32 accumulator 16 at
a time, up to 512 to an accumulator: each of the 32 steps and of the Dm / 256 additions of accumulators
may lose a few units of 2^-24 of the magnitudes' sum A_i = max_j sum_k |h_ik w_jk|; 2^-21 is allowed
for each. The exponentials are good to 2^-22 and a group's sum of up to 256 of them to 2^-16,
the joins to less: 2^-15 of ln z. logp, lse and the alternatives carry the error of two logits and of
ln z; the entropy, whose gradient is p_j (ln p_j + H), that of the logits times 2 (1 + H).
"""
import math

import numpy as np
import pytest
import torch

import context_parallelism_gb300 as up
from oracle import logp_ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


def _np(t):
    return t.detach().double().cpu().numpy()


def _inputs(S, Dm, V, seed=0, sure=3.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    w = (torch.randn((V, Dm), generator=g, device=DEV) * (2 / math.sqrt(Dm))).to(BF)
    t = torch.randint(0, V, (S,), generator=g, device=DEV)
    h = (torch.randn((S, Dm), generator=g, device=DEV) +
         sure * torch.rand((S, 1), generator=g, device=DEV) * w[t].float()).to(BF)
    t[::7] = -1
    return h, w, t


def _logit_error(h, w):
    Dm = h.shape[1]
    size = (h.double().abs() @ w.double().abs().t()).amax(-1).cpu().numpy()
    return (min(Dm, 512) / 16 + 2 + Dm / 256) * 2.0 ** -21 * size


def _check(got, h, w, t, top):
    logp, entropy, lse, tl, ti = got
    V = w.shape[0]
    rp, rh, rl, rt, ri = logp_ref(h.double().cpu(), w.double().cpu(),
                                  None if t is None else t.cpu().numpy(), top)
    ex = _logit_error(h, w)
    tol = 2 * ex + 2.0 ** -15
    assert (np.abs(_np(lse) - rl) <= tol + 2.0 ** -23 * np.abs(rl)).all()
    assert (np.abs(_np(entropy) - rh) <= (2 * ex + 2.0 ** -15) * (1 + rh)).all()
    if t is None:
        assert logp is None
    else:
        out = t.cpu().numpy() >= V
        assert np.isnan(_np(logp)[out]).all()
        assert (np.abs(_np(logp) - rp) <= tol + 2.0 ** -22 * np.abs(rp))[~out].all()
        assert (logp[t < 0] == 0).all()
    if not top:
        assert tl is None and ti is None
        return
    k = min(top, V)
    assert (ti.cpu().numpy()[:, :k] == ri).all()
    assert (np.abs(_np(tl)[:, :k] - rt) <= tol[:, None] + 2.0 ** -22 * np.abs(rt)).all()
    assert (ti[:, k:] == -1).all() and (tl[:, k:] == -math.inf).all()


SHAPES = [  # S, Dm, V, top
    (1, 8, 1, 3), (1, 64, 2, 1), (2, 72, 7, 24), (3, 256, 31, 0), (16, 264, 33, 5), (17, 64, 255, 24),
    (32, 512, 257, 8), (33, 1000, 1000, 20), (64, 1024, 2433, 5), (1, 4096, 40000, 5),
    (48, 328, 20011, 20), (5, 2048, 5003, 24), (16, 4096, 3000, 5), (17, 4096, 3000, 5),
    (65, 8, 1, 2), (66, 64, 31, 24), (128, 72, 256, 5), (129, 256, 257, 0), (200, 264, 1000, 1),
    (300, 1000, 2433, 20), (257, 1024, 5003, 24), (70, 2048, 20011, 5), (511, 16, 300, 8),
    # tiles of other numbers of columns, whole and broken last ones, one and several rounds of them
    (3, 72, 38912, 24), (16, 136, 45613, 9), (2, 200, 97281, 0), (9, 72, 128256, 5), (1, 264, 38913, 3),
    (100, 136, 45613, 9), (17, 72, 128256, 24), (128, 200, 97281, 0), (19, 2048, 38913, 24),
    (255, 64, 60001, 5), (40, 64, 9729, 3), (40, 64, 19457, 3), (385, 72, 9999, 2),
]


@pytest.mark.parametrize("S,Dm,V,top", SHAPES)
def test_against_the_oracle(S, Dm, V, top):
    h, w, t = _inputs(S, Dm, V, seed=S + Dm)
    got = up.token_logprobs(h, w, t, top=top)
    up.upipe_sync_status()
    _check(got, h, w, t, top)
    again = up.token_logprobs(h, w, t, top=top)
    for a, b in zip(got, again):
        assert (a is None and b is None) or torch.equal(a, b)


def test_without_targets_and_beyond_the_vocabulary():
    h, w, t = _inputs(40, 64, 500)
    _check(up.token_logprobs(h, w, None, top=3), h, w, None, 3)
    t[5], t[6], t[7] = 500, 1 << 40, 499
    _check(up.token_logprobs(h, w, t), h, w, t, 0)
    h, w, t = _inputs(140, 64, 500)
    t[5], t[6], t[7] = 500, 1 << 40, 499
    _check(up.token_logprobs(h, w, t, top=2), h, w, t, 2)


@pytest.mark.parametrize("S", [266, 300, 400])
def test_tiles(S):
    """seq_tile cuts the tokens; a last tile of few tokens takes the kernel for short calls."""
    h, w, t = _inputs(S, 128, 777)
    got = up.token_logprobs(h, w, t, top=6, seq_tile=128)
    _check(got, h, w, t, 6)


@pytest.mark.parametrize("S", [3, 400])
def test_host_activations(S):
    h, w, t = _inputs(S, 128, 777)
    want = up.token_logprobs(h, w, t, top=4, seq_tile=128)
    hh = h.cpu().pin_memory()
    got = up.token_logprobs(hh, w, t, top=4, seq_tile=128)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("S", [2, 100])
def test_equal_logits_go_by_index(S):
    """Rows of the table that are the same, in the same and in other groups; a row of h that is zero."""
    h, w, t = _inputs(S, 64, 3000)
    w[2900], w[17], w[18], w[1500] = w[3], w[3], w[3], w[3]
    h[0] = 4 * w[3].float().div(w[3].float().norm()).to(BF)
    h[1] = 0
    got = up.token_logprobs(h, w, t, top=24)
    _check(got, h, w, t, 24)
    assert got[4][0, :5].tolist() == [3, 17, 18, 1500, 2900]
    assert got[4][1].tolist() == list(range(24))
    assert got[1][1].item() == pytest.approx(math.log(3000), rel=2.0 ** -20)


@pytest.mark.parametrize("S", [1, 80])
def test_order_below_the_resolution_of_32_bits(S):
    """Logits of 1 + 2^-30 and 1 + 2^-31 are one in fp32; the larger comes first all the same, and so do
    sums whose large terms cancel."""
    Dm, V = 64, 2000
    w = torch.zeros((V, Dm), device=DEV)
    w[:, 0] = -1.0
    w[100, 0] = w[1500, 0] = 1.0
    w[100, 1], w[1500, 1] = 2.0 ** -31, 2.0 ** -30
    w[7, 0], w[7, 2], w[7, 3], w[7, 4] = 0.5, 2.0 ** 20, 2.0 ** -8, -2.0 ** 20
    w[900, 0], w[900, 2], w[900, 3], w[900, 4] = 0.5, 2.0 ** 20, 2.0 ** -7, -2.0 ** 20
    h = torch.ones((S, Dm), device=DEV).to(BF)
    _, _, _, _, ti = up.token_logprobs(h, w.to(BF), top=4)
    assert (ti == torch.tensor([1500, 100, 900, 7], device=DEV)).all()


@pytest.mark.parametrize("S", [1, 70])
def test_probabilities_near_one(S):
    """logp of a nearly certain token keeps its digits: the logits are exact here (powers of two), so
    the error is that of the sums, relative to logp itself; likewise the entropy."""
    Dm, V = 64, 5000
    w = torch.zeros((V, Dm), device=DEV)
    w[4321, 0] = 1.0
    h = torch.zeros((S, Dm), device=DEV)
    for gap in (8.0, 16.0, 24.0, 32.0):
        h[:, 0] = gap
        t = torch.full((S,), 4321, device=DEV)
        logp, entropy, lse, tl, ti = up.token_logprobs(h.to(BF), w.to(BF), t, top=2)
        q = (V - 1) * math.exp(-gap)
        assert logp[0].item() == pytest.approx(-math.log1p(q), rel=2.0 ** -15)
        assert tl[0, 0] == logp[0] and ti[0].tolist() == [4321, 0]
        want = math.log1p(q) + q / (1 + q) * gap
        assert entropy[0].item() == pytest.approx(want, rel=2.0 ** -15)
        assert lse[0].item() == pytest.approx(gap + math.log1p(q), rel=2.0 ** -20)


@pytest.mark.parametrize("Dm", [64, 1200])
@pytest.mark.parametrize("S", [9, 90])
def test_values_that_are_not_finite(S, Dm):
    h, w, t = _inputs(S, Dm, 700)
    t = t.clamp(min=0)
    good = up.token_logprobs(h, w, t, top=3)
    h2 = h.clone()
    h2[4, 10] = float("nan")
    h2[5, 3] = float("inf")
    bad = up.token_logprobs(h2, w, t, top=3)
    rows = torch.ones(S, dtype=torch.bool, device=DEV)
    rows[4] = rows[5] = False
    for a, b in zip(good, bad):
        assert torch.equal(a[rows], b[rows])
    for x in bad[:4]:
        assert x[4:6].isnan().all()
    assert (bad[4][4:6] == -1).all()
    # a column of -inf has no probability and changes nothing else; one of NaN or +inf takes all rows
    h3 = h.clone()
    h3[:, 0] = 1.0
    w3 = w.clone()
    w3[333, 0] = -math.inf
    got = up.token_logprobs(h3, w3, t, top=3)
    keep = torch.arange(700, device=DEV) != 333
    ref = torch.log_softmax(h3.double() @ w3[keep].double().t(), -1)
    lse_ref = torch.logsumexp(h3.double() @ w3[keep].double().t(), -1)
    assert ((got[2].double() - lse_ref).abs() <= 1e-3).all()
    assert ((got[1].double() + (ref.exp() * ref).sum(-1)).abs() <= 1e-2).all()
    assert (got[0][t == 333] == -math.inf).all() and got[3].isfinite().all()
    for x in (math.inf, math.nan):
        w3[333, 0] = x
        got = up.token_logprobs(h3, w3, t, top=3)
        assert got[2].isnan().all() and got[1].isnan().all() and (got[4] == -1).all()
    w3[:, 0] = -math.inf
    got = up.token_logprobs(h3, w3, t, top=3)
    assert got[2].isnan().all() and (got[4] == -1).all()


def test_a_row_does_not_see_the_others():
    """The result of a token depends on its own h alone, in calls of one kind."""
    h, w, t = _inputs(16, 264, 1500)
    all_ = up.token_logprobs(h, w, t, top=5)
    for i in (0, 7, 15):
        one = up.token_logprobs(h[i:i + 1].clone(), w, t[i:i + 1].clone(), top=5)
        assert all(torch.equal(a[i:i + 1], b) for a, b in zip(all_, one))
    h, w, t = _inputs(300, 264, 1500)
    all_ = up.token_logprobs(h, w, t, top=5)
    half = up.token_logprobs(h[150:].clone(), w, t[150:].clone(), top=5)
    assert all(torch.equal(a[150:], b) for a, b in zip(all_, half))


@pytest.mark.parametrize("S", [5, 130])
def test_streams_and_graphs(S):
    h, w, t = _inputs(S, 256, 3000)
    want = up.token_logprobs(h, w, t, top=7)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = up.token_logprobs(h, w, t, top=7, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graphs, outs, spaces = [], [], []
    size = up.upipe_logp_workspace_bytes(S, 256, 3000, 7, 4096)
    for _ in range(2):
        ws = torch.full((size,), 255, dtype=torch.uint8, device=DEV)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(up.token_logprobs(h, w, t, top=7, workspace=ws))
        graphs.append(g)
        spaces.append(ws)
    for new in (7, 8):
        h.copy_(_inputs(S, 256, 3000, seed=new)[0])
        want = up.token_logprobs(h, w, t, top=7)
        torch.cuda.synchronize()
        graphs[0].replay()
        with torch.cuda.stream(s):
            graphs[1].replay()
        torch.cuda.synchronize()
        for o in outs:
            assert all(torch.equal(a, b) for a, b in zip(want, o))


@pytest.mark.parametrize("S,V,top,host", [(1, 7, 24, False), (64, 2433, 5, False), (130, 1000, 0, False),
                                          (300, 257, 24, True), (200, 5003, 1, False)])
def test_workspace_bounds(S, V, top, host):
    """Exactly the declared bytes, between bands that stay as they are; what they held before does not
    matter; outputs stay within theirs."""
    h, w, t = _inputs(S, 72, V)
    want = up.token_logprobs(h, w, t, top=top, seq_tile=128)
    hh = h.cpu().pin_memory() if host else h
    size, band = up.upipe_logp_workspace_bytes(S, 72, V, top, 128, up.UPIPE_HOST_ACT if host else 0), 1 << 20
    for fill in (0, 255):
        big = torch.full((size + 2 * band,), fill, dtype=torch.uint8, device=DEV)
        f = [torch.full((S + 2,), 7.0, device=DEV) for _ in range(3)]
        tl = torch.full((S + 2, max(top, 1)), 7.0, device=DEV)
        ti = torch.full((S + 2, max(top, 1)), 7, device=DEV)
        up.upipe_logp_fwd(hh, w, t, f[0][1:], f[1][1:], f[2][1:], tl[1:] if top else None,
                          ti[1:] if top else None, S, 72, V, top, 128, big[band:band + size])
        torch.cuda.synchronize()
        for a, b in zip(f, want):
            assert torch.equal(a[1:-1], b) and a[0] == 7 and a[-1] == 7
        if top:
            assert torch.equal(tl[1:-1], want[3]) and torch.equal(ti[1:-1], want[4])
        assert (tl[0] == 7).all() and (tl[-1] == 7).all() and (ti[-1] == 7).all()
        assert (big[:band] == fill).all() and (big[band + size:] == fill).all()
    with pytest.raises(up.UpipeError) as e:
        up.upipe_logp_fwd(hh, w, t, f[0], f[1], f[2], tl if top else None, ti if top else None, S, 72, V,
                          top, 128, big, workspace_bytes=size - 1)
    assert e.value.status == up.UPIPE_ERR_WORKSPACE_TOO_SMALL


def test_only_what_is_asked_for():
    h, w, t = _inputs(20, 64, 300)
    want = up.token_logprobs(h, w, t)
    ws = torch.empty(up.upipe_logp_workspace_bytes(20, 64, 300, 0, 128), dtype=torch.uint8, device=DEV)
    out = torch.zeros(20, device=DEV)
    up.upipe_logp_fwd(h, w, None, None, None, out, None, None, 20, 64, 300, 0, 128, ws)
    assert torch.equal(out, want[2])
    up.upipe_logp_fwd(h, w, t, out, None, None, None, None, 20, 64, 300, 0, 128, ws)
    assert torch.equal(out, want[0])


def test_no_tokens():
    w = _inputs(4, 64, 300)[1]
    got = up.token_logprobs(torch.zeros((0, 64), dtype=BF, device=DEV), w,
                            torch.zeros(0, dtype=torch.int64, device=DEV), top=3)
    assert got[0].shape == (0,) and got[4].shape == (0, 3)


def test_gradient_is_the_losss():
    """The gradient of sum g logp through ce_loss_backward with this lse, against autograd in 64 bits
    (dh and dw carry the bf16 rounding of the logits' gradients: 1e-2 of their norm, as the loss's)."""
    S, Dm, V = 192, 128, 640
    h, w, t = _inputs(S, Dm, V)
    g = torch.randn(S, device=DEV)
    logp, _, lse, _, _ = up.token_logprobs(h, w, t)
    dh, dw = up.ce_loss_backward(h, w, t, lse, -g, seq_tile=128)
    h64, w64 = h.double().requires_grad_(), w.double().requires_grad_()
    p = torch.log_softmax(h64 @ w64.t(), -1).gather(1, t.clamp(min=0)[:, None])[:, 0]
    rh, rw = torch.autograd.grad((p * g * (t >= 0)).sum(), (h64, w64))
    assert (dh.double() - rh).norm() <= 1e-2 * rh.norm()
    assert (dw.double() - rw).norm() <= 1e-2 * rw.norm()


def test_short_and_long_calls_agree():
    """The last tokens of a long call alone: the same logits to the rounding of the pieces' sums, the same
    alternatives."""
    h, w, t = _inputs(300, 1024, 3000)
    a = up.token_logprobs(h, w, t, top=10)
    b = up.token_logprobs(h[290:].clone(), w, t[290:].clone(), top=10)
    assert torch.equal(a[4][290:], b[4])
    ex = torch.from_numpy(_logit_error(h, w)).to(DEV)[290:] * 2 + 2.0 ** -15
    for i in (0, 2):
        assert ((a[i][290:] - b[i]).abs().double() <= 2 * ex).all()
