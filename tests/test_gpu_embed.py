"""Token embedding and its gradient on the GPU against the 64-bit oracle (needs an sm_103a GPU).

Tolerances: h is one bf16 rounding (2^-8 |h|) of a product in fp32 (2^-23 |h|). An element of dw is a
sum of n rows in fp32 in some order: n roundings of 2^-24 and two for the factor, of the sum of the
magnitudes.
"""
import numpy as np
import pytest
import torch

import context_parallelism_gb300 as up
from oracle import embed_bwd_ref, embed_ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


def _bf(*shape, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(shape, generator=g, device=DEV).to(BF)


def _tokens(n, V, seed, kind):
    rng = np.random.default_rng(seed)
    if kind == "even":
        t = rng.integers(0, V, n)
    elif kind == "one":
        t = np.full(n, V - 1)
    elif kind == "sorted":
        t = np.sort(rng.integers(0, V, n))[::-1].copy()
    else:  # a few tokens make up most of a text, some places hold none
        p = 1 / (np.arange(V) + 1.0) ** 1.2
        t = rng.permutation(V)[rng.choice(V, n, p=p / p.sum())]
        t[rng.random(n) < 0.1] = -1
        t[rng.random(n) < 0.02] = V + 5
    return torch.from_numpy(t.astype(np.int64))


def _check_dw(dw, t, dh, V, scale, before=None):
    ref, size = embed_bwd_ref(t, dh, V, scale)
    n = np.bincount(t[(t >= 0) & (t < V)].numpy(), minlength=V)[:, None]
    if before is not None:
        ref, size = ref + before, size + np.abs(before)
    err = np.abs(dw.double().cpu().numpy() - ref) - (n + 3) * 2.0 ** -24 * size
    assert (err <= 0).all(), float(err.max())


CASES = [  # places, Dm, V
    (1, 8, 1), (3, 8, 1), (7, 64, 5), (33, 1000, 300), (65, 2056, 17), (129, 8, 70000),
    (2048, 64, 511), (4097, 32, 512), (8192, 24, 513), (300, 4096, 128256), (9000, 16, 300000),
    (20000, 8, 1 << 20),
]


KINDS = ["even", "one", "sorted", "text"]  # the largest table: one of them


@pytest.mark.parametrize("n,Dm,V,kind", [(*c, k) for c in CASES for k in KINDS
                                         if c[1] * c[2] <= 1 << 24 or k == "text"])
def test_gradient(n, Dm, V, kind):
    t, dh = _tokens(n, V, n, kind), _bf(n, Dm, seed=1)
    dw = up.embed_backward(t.to(DEV), dh, V, scale=0.75)
    _check_dw(dw, t, dh, V, 0.75)
    # added to what is there: rows without a token keep their bits
    base = torch.randn((V, Dm), device=DEV)
    want = base.clone()
    got = up.embed_backward(t.to(DEV), dh, V, scale=0.75, dw=base)
    assert got is base
    _check_dw(base, t, dh, V, 0.75, want.double().cpu().numpy())
    absent = torch.ones(V, dtype=torch.bool)
    absent[t[(t >= 0) & (t < V)]] = False
    assert torch.equal(base[absent.to(DEV)], want[absent.to(DEV)])
    assert (dw[absent.to(DEV)] == 0).all()
    again = up.embed_backward(t.to(DEV), dh, V, scale=0.75)
    assert torch.equal(dw, again)


@pytest.mark.parametrize("scale", [1.0, 64.0, -0.3])
@pytest.mark.parametrize("n,Dm,V", CASES)
def test_forward(n, Dm, V, scale):
    t, w = _tokens(n, V, n, "text"), _bf(V, Dm, seed=2)
    h = up.embed_forward(t.to(DEV), w, scale=scale)
    rows = {int(v): i for i, v in enumerate(np.unique(t[(t >= 0) & (t < V)].numpy()))}
    small = torch.stack([w[v] for v in rows]) if rows else w[:1]
    s = torch.tensor([rows[v] if v in rows else -1 if v < 0 else len(small) for v in t.tolist()])
    ref = embed_ref(s, small, scale)
    got = h.double().cpu().numpy()
    assert (np.isnan(got) == np.isnan(ref)).all()
    err = np.abs(got - ref) - (2.0 ** -8 + 2.0 ** -23) * np.abs(ref)
    assert not (err > 0).any()
    if scale == 1.0:
        assert torch.equal(h[t < V], torch.where((t >= 0)[:, None].to(DEV), w[t.clamp(0, V - 1).to(DEV)],
                                                  torch.zeros((), dtype=BF, device=DEV))[t < V])


def test_shapes_and_offsets():
    """Any leading shape, a view of tokens that starts at an odd place, one token."""
    w, ids = _bf(50, 40, seed=1), torch.randint(0, 50, (31,), device=DEV)
    t = ids[1:].view(2, 3, 5)
    h = up.embed_forward(t, w)
    assert h.shape == (2, 3, 5, 40) and torch.equal(h, w[t])
    dw = up.embed_backward(t, h, 50)
    _check_dw(dw, t.reshape(-1).cpu(), h.reshape(-1, 40), 50, 1.0)
    assert torch.equal(up.embed_forward(ids[3], w), w[ids[3]])


def test_values_that_are_not_finite():
    """They reach their own row alone; those of places without a row reach none."""
    t = torch.tensor([2, 0, -1, 2, 9, 1])
    dh = _bf(6, 16, seed=1)
    dh[1, 3], dh[2], dh[4, 5] = float("inf"), float("nan"), float("nan")
    dw = up.embed_backward(t.to(DEV), dh, 4)
    assert dw[0, 3] == float("inf")
    dw[0, 3] = 0
    assert dw.isfinite().all() and (dw[3] == 0).all()


def test_no_tokens():
    t = torch.zeros((0,), dtype=torch.int64, device=DEV)
    w, dh = _bf(5, 8), torch.zeros((0, 8), dtype=BF, device=DEV)
    assert up.embed_forward(t, w).shape == (0, 8)
    assert (up.embed_backward(t, dh, 5) == 0).all()
    base = torch.ones((5, 8), device=DEV)
    assert (up.embed_backward(t, dh, 5, dw=base) == 1).all()
    none = torch.full((9,), -1, device=DEV)
    assert (up.embed_backward(none, _bf(9, 8), 5) == 0).all()


@pytest.mark.parametrize("n,V", [(8192, 3000), (8193, 3000), (300001, 40000), (1100000, 70000)])
def test_long_sequence(n, V):
    """Both sides of the border between the sorts, more tiles than a scatter adds up itself, runs over many
    chunks; against index_add in 64 bits."""
    Dm = 16
    t, dh = _tokens(n, V, 5, "text").to(DEV), _bf(n, Dm, seed=6)
    dw = up.embed_backward(t, dh, V)
    live = (t >= 0) & (t < V)
    ref = torch.zeros((V, Dm), dtype=torch.float64, device=DEV).index_add_(0, t[live], dh[live].double())
    size = torch.zeros((V, Dm), dtype=torch.float64, device=DEV).index_add_(
        0, t[live], dh[live].double().abs())
    count = torch.bincount(t[live], minlength=V)[:, None]
    assert ((dw.double() - ref).abs() <= (count + 3) * 2.0 ** -24 * size).all()


@pytest.mark.parametrize("n,Dm,V", [(300, 8, 152 * 2048 * 32 + 33), (20001, 1032, 5000), (8191, 2056, 400),
                                    (8192, 64, 31), (40000, 4104, 100)])
def test_large_tables_and_odd_chunks(n, Dm, V):
    """A bitmap that a block makes in pieces; chunks of lengths that divide nothing; against index_add."""
    t, dh = torch.randint(-1, V, (n,), device=DEV), _bf(n, Dm, seed=4)
    t[n // 3], t[n // 2:n // 2 + n // 5] = V - 1, V // 2
    dw = up.embed_backward(t, dh, V)
    live = t >= 0
    rows, at, count = t[live].unique(return_inverse=True, return_counts=True)
    ref = torch.zeros((len(rows), Dm), dtype=torch.float64, device=DEV)
    size = torch.zeros_like(ref)
    for lo in range(0, int(live.sum()), 4096):
        x = dh[live][lo:lo + 4096].double()
        ref.index_add_(0, at[lo:lo + 4096], x)
        size.index_add_(0, at[lo:lo + 4096], x.abs())
    assert ((dw[rows].double() - ref).abs() <= (count[:, None] + 3) * 2.0 ** -24 * size).all()
    absent = torch.ones(V, dtype=torch.bool, device=DEV)
    absent[rows] = False
    assert not dw[absent].any()


def test_streams_graphs_and_two_workspaces():
    n, Dm, V = 5000, 128, 3000
    t, dh, w = _tokens(n, V, 1, "text").to(DEV), _bf(n, Dm, seed=1), _bf(V, Dm, seed=2)
    s = torch.cuda.Stream()
    want = up.embed_backward(t, dh, V), up.embed_forward(t, w, 2.0)
    s.wait_stream(torch.cuda.current_stream())
    got = up.embed_backward(t, dh, V, stream=s), up.embed_forward(t, w, 2.0, stream=s)
    s.synchronize()
    bits = lambda x: x.contiguous().view(torch.int16)  # noqa: E731 (NaN rows too)
    assert torch.equal(got[0], want[0]) and torch.equal(bits(got[1]), bits(want[1]))
    size = up.upipe_embed_workspace_bytes(n, Dm, V)
    graphs, outs, spaces = [], [], []
    for _ in range(2):
        ws = torch.full((size,), 255, dtype=torch.uint8, device=DEV)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(up.embed_backward(t, dh, V, workspace=ws))
        graphs.append(g)
        spaces.append(ws)
    for new in (7, 8):
        t.copy_(_tokens(n, V, new, "text"))
        want = up.embed_backward(t, dh, V)
        torch.cuda.synchronize()
        graphs[0].replay()
        with torch.cuda.stream(s):
            graphs[1].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want) and torch.equal(outs[1], want)


@pytest.mark.parametrize("n,Dm,V", [(1, 8, 1), (4097, 1000, 333), (9000, 64, 70000)])
def test_workspace_bounds(n, Dm, V):
    """Exactly the declared bytes, between bands that stay as they are; what they held before does not
    matter."""
    t, dh = _tokens(n, V, 3, "text").to(DEV), _bf(n, Dm, seed=4)
    size, band = up.upipe_embed_workspace_bytes(n, Dm, V), 1 << 20
    want = up.embed_backward(t, dh, V)
    for fill in (0, 255):
        big = torch.full((size + 2 * band,), fill, dtype=torch.uint8, device=DEV)
        out = torch.full((V + 2, Dm), 7.0, device=DEV)
        up.upipe_embed_bwd(t, dh, out[1:-1] if Dm % 4 == 0 else out, n, Dm, V, 1.0, 0,
                           big[band:band + size])
        assert torch.equal(out[1:-1], want) and (out[0] == 7).all() and (out[-1] == 7).all()
        assert (big[:band] == fill).all() and (big[band + size:] == fill).all()
    with pytest.raises(up.UpipeError) as e:
        up.upipe_embed_bwd(t, dh, out[:V], n, Dm, V, 1.0, 0, big, workspace_bytes=size - 1)
    assert e.value.status == up.UPIPE_ERR_WORKSPACE_TOO_SMALL


def test_tied_table():
    """One gradient for the readout's and the embedding's table, as one call after the other gives it."""
    S, Dm, V = 256, 128, 320
    t = torch.randint(0, V, (S,), device=DEV)
    w = (_bf(V, Dm, seed=1).float() * 0.1).to(BF)
    h = up.embed_forward(t, w, scale=4.0)
    target = t.roll(-1)
    g = torch.full((S,), 1.0 / S, device=DEV)
    loss, lse, dh, dw = up.ce_loss_fused(h, w, target, g, seq_tile=128)
    alone = dw.clone()
    up.embed_backward(t, dh, V, scale=4.0, dw=dw)
    _check_dw(dw, t.cpu(), dh, V, 4.0, alone.double().cpu().numpy())
