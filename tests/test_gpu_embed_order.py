"""What follows the embedding's gradient in a stream or a captured graph sees the whole of it (needs an
sm_103a GPU): also where no token's places go over the border of two chunks, so that the last launch has
nothing to join.
"""
import numpy as np
import pytest
import torch

import context_parallelism_gb300 as up

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


def _tokens(n, V, kind, seed):
    rng = np.random.default_rng(seed)
    t = rng.permutation(V)[:n]
    if kind == "padding":
        t[rng.random(n) < 0.99] = -1
    elif kind == "none":
        t[:] = -1
    return torch.from_numpy(t.astype(np.int64)).to(DEV)


def _want(t, dh, V):
    """Each token once: its row as it is."""
    dw = torch.zeros((V, dh.shape[1]), device=DEV)
    dw[t[t >= 0]] = dh[t >= 0].float()
    return dw


@pytest.mark.parametrize("add", [False, True])
@pytest.mark.parametrize("kind", ["distinct", "padding", "none"])
@pytest.mark.parametrize("n,Dm,V", [(8000, 1024, 60000), (20000, 512, 70001), (3000, 4096, 9000)])
def test_the_next_operation_reads_all_of_it(n, Dm, V, kind, add):
    t = _tokens(n, V, kind, 0)
    dh = torch.randn((n, Dm), device=DEV).to(BF)
    dw = torch.empty((V, Dm), device=DEV)
    ws = torch.empty(up.upipe_embed_workspace_bytes(n, Dm, V), dtype=torch.uint8, device=DEV)
    out = torch.empty_like(dw)

    def step():
        up.upipe_embed_bwd(t, dh, dw, n, Dm, V, 1.0, add, ws)
        out.copy_(dw)

    step()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for seed in range(6):
        t.copy_(_tokens(n, V, kind, seed))
        dh.copy_(torch.randn((n, Dm), device=DEV))
        want = _want(t, dh, V)
        for run in (step, g.replay):
            dw.fill_(0.0 if add else float("nan"))
            out.fill_(float("nan"))
            run()
            assert torch.equal(out, want)
