"""Workspace bounds: every call is given a workspace of exactly the declared size, cut out of a
larger buffer whose guard bands before and after it hold a canary byte pattern. After the call
the guards must be unchanged: no kernel or staging copy writes outside the bytes the library
declared (the caller-owned arena is the library's only scratch). Needs an sm_103a GPU."""
import pytest
import torch

import context_parallelism_gb300 as up
from workloads import LOSS_WORKLOADS, MLP_WORKLOADS, WORKLOADS, make_inputs, \
    make_loss_inputs, make_mlp_inputs

pytestmark = pytest.mark.gpu

GUARD = 1 << 20  # bytes on each side, a multiple of 256 so the workspace stays aligned
CANARY = 0xA5


class Guarded:
    def __init__(self, nbytes):
        self.n = nbytes
        self.buf = torch.full((nbytes + 2 * GUARD,), CANARY, dtype=torch.uint8, device="cuda")
        self.ws = self.buf[GUARD:GUARD + nbytes]

    def check(self):
        torch.cuda.synchronize()
        lo, hi = self.buf[:GUARD], self.buf[GUARD + self.n:]
        assert int((lo != CANARY).sum()) == 0, "write before the workspace"
        assert int((hi != CANARY).sum()) == 0, "write past the end of the workspace"


def _pinned(t):
    out = torch.empty(t.shape, dtype=t.dtype, pin_memory=True)
    out.copy_(t)
    return out


@pytest.mark.parametrize("S,hc,T,kv_host,act_host", [
    (1000, 4, 256, False, False),   # several trunks, ragged
    (1000, 8, 1000, False, False),  # one trunk
    (777, 4, 256, True, False),     # host K/V slots
    (640, 4, 256, True, True),      # everything on the host
])
def test_attention_stays_inside_its_workspace(S, hc, T, kv_host, act_host):
    w = WORKLOADS["llama8b_s8k"].with_(S=S, Hq=8, Hkv=2, seed=71 + S)
    q, k, v, do = make_inputs(w, "cpu")
    B, Hq, Hkv, D = w.B, w.Hq, w.Hkv, w.D
    dev = (lambda t: _pinned(t)) if act_host else (lambda t: t.cuda())
    kvd = (lambda t: _pinned(t)) if kv_host else (lambda t: t.cuda())
    qi, doi, ki, vi = dev(q), dev(do), kvd(k), kvd(v)
    mask = (up.UPIPE_HOST_KV if kv_host else 0) | (up.UPIPE_HOST_ACT if act_host else 0)
    for pass_ in (up.UPIPE_PASS_FWD, up.UPIPE_PASS_BWD):
        g = Guarded(up.upipe_workspace_bytes(B, S, Hq, Hkv, D, 1, hc, T, pass_, mask))
        if pass_ == up.UPIPE_PASS_FWD:
            o, lse = up.attention_forward(qi, ki, vi, head_chunk=hc, seq_trunk=T,
                                          workspace=g.ws, o_on_host=act_host)
        else:
            up.attention_backward(qi, ki, vi, o, lse, doi, head_chunk=hc, seq_trunk=T,
                                  workspace=g.ws, dkdv_on_host=kv_host, dq_on_host=act_host)
        up.upipe_sync_status()
        g.check()


@pytest.mark.parametrize("S,T,host", [(1000, 256, False), (1000, 256, True), (100, 128, True)])
def test_tiled_paths_stay_inside_their_workspace(S, T, host):
    lw = LOSS_WORKLOADS["readout_small"].with_(S=S, seed=73 + S)
    h, w, t, gl = make_loss_inputs(lw, "cpu")
    hi = _pinned(h) if host else h.cuda()
    wg, tg, gg = w.cuda(), t.cuda(), gl.cuda()
    mask = up.UPIPE_HOST_ACT if host else 0
    g = Guarded(up.upipe_ce_workspace_bytes(S, lw.Dm, lw.V, T, up.UPIPE_PASS_FWD, mask))
    loss, lse = up.ce_loss_forward(hi, wg, tg, seq_tile=T, workspace=g.ws)
    up.upipe_sync_status()
    g.check()
    g = Guarded(up.upipe_ce_workspace_bytes(S, lw.Dm, lw.V, T, up.UPIPE_PASS_BWD, mask))
    up.ce_loss_backward(hi, wg, tg, lse, gg, seq_tile=T, workspace=g.ws, dh_on_host=host)
    up.upipe_sync_status()
    g.check()

    mw = MLP_WORKLOADS["mlp_small"].with_(S=S, seed=75 + S)
    x, w_gu, w_d, dy = make_mlp_inputs(mw, "cpu")
    xi = _pinned(x) if host else x.cuda()
    dyi = _pinned(dy) if host else dy.cuda()
    wgu, wdd = w_gu.cuda(), w_d.cuda()
    g = Guarded(up.upipe_mlp_workspace_bytes(S, mw.Dm, mw.F, T, up.UPIPE_PASS_FWD, mask))
    up.mlp_forward(xi, wgu, wdd, seq_tile=T, workspace=g.ws, y_on_host=host)
    up.upipe_sync_status()
    g.check()
    g = Guarded(up.upipe_mlp_workspace_bytes(S, mw.Dm, mw.F, T, up.UPIPE_PASS_BWD, mask))
    up.mlp_backward(xi, wgu, wdd, dyi, seq_tile=T, workspace=g.ws, dx_on_host=host)
    up.upipe_sync_status()
    g.check()


def _paged(counts, lens, Hq, Hkv, D, page, prefix, packed, max_q, max_len):
    """Paged attention on a workspace of exactly the declared size; its bytes before the call differ
    from run to run, so that a part read before it is written shows."""
    g = torch.Generator(device="cuda").manual_seed(sum(lens) + prefix)
    need = [-(-m // page) for m in lens]
    shared = -(-prefix // page)
    n = shared + sum(need)
    kp, vp = (torch.randn((n, page, Hkv, D), generator=g, device="cuda").bfloat16() for _ in range(2))
    table = torch.full((len(lens), max(1, max(need))), -1, dtype=torch.int32)
    at = shared
    for b, x in enumerate(need):
        table[b, :x] = torch.arange(at, at + x)
        at += x
    rows = sum(counts)
    shape = (rows + 2, Hq, D) if packed else (len(lens), counts[0], Hq, D)
    q = torch.randn(shape, generator=g, device="cuda").bfloat16()
    kw = dict(prefix_table=torch.arange(shared, dtype=torch.int32, device="cuda"), prefix_len=prefix)
    if packed:
        cu = torch.zeros(len(counts) + 1, dtype=torch.int32)
        cu[1:] = torch.tensor(counts).cumsum(0)
        kw["cu_seqlens"] = cu.cuda()
    size = up.upipe_attn_paged_workspace_bytes(
        len(lens), rows + 2 if packed else rows, Hq, Hkv, D, prefix,
        max_q if packed else counts[0], max_len)
    got = []
    for fill in (CANARY, 0xFF, 0x00):
        gd = Guarded(size)
        gd.ws.fill_(fill)
        out, lse = torch.zeros_like(q), torch.zeros(
            (Hq, rows + 2) if packed else (len(lens), Hq, counts[0]), device="cuda")
        up.paged_attention(q, kp, vp, table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                           max_q=max_q, max_len=max_len, out=out, lse=lse, workspace=gd.ws, **kw)
        up.upipe_sync_status()
        gd.check()
        got.append((out, lse))
    for out, lse in got:
        assert torch.isfinite(out).all() and not torch.isnan(lse).any()
        assert torch.equal(out, got[0][0]) and torch.equal(lse, got[0][1])


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("hint", [(1, 1), (4, 700), (64, 100000)])
@pytest.mark.parametrize("case", [
    ([1] * 5, [1, 700, 33, 0, 64], 8, 2, 128, 16, 0),          # own pages in tiles of 8 rows
    ([3] * 4, [3, 500, 20, 5], 16, 4, 64, 32, 130),            # tiles of 16, a short prefix beside
    ([1] * 3, [10, 20, 30], 32, 1, 128, 16, 40),               # 64 rows
    ([50] * 2, [50, 400], 4, 2, 64, 64, 100),
    ([1] * 24, [9] * 24, 8, 1, 128, 16, 1700),                 # tensor-core prefix, two row tiles
    ([2] * 6, [2, 9, 600, 33, 4, 5], 8, 2, 128, 64, 5600),     # one row tile, two key streams
    ([1] * 40, [b + 1 for b in range(40)], 16, 2, 64, 32, 900),
    ([20] * 2, [30, 90], 32, 2, 128, 128, 3500),               # 64-row tiles beside it
])
def test_paged_attention_stays_inside_its_workspace(case, hint, packed):
    counts, lens, Hq, Hkv, D, page, prefix = case
    if packed:
        counts = [n - b % 2 if n > 1 else n for b, n in enumerate(counts)]
    _paged(counts, lens, Hq, Hkv, D, page, prefix, packed, *hint)
