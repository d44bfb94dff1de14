"""The binding's one-to-one functions of the rotary, append and paged-attention entries give what the
functions that allocate for the caller give (needs an sm_103a GPU)."""
import pytest
import torch

import context_parallelism_gb300 as up
from tests.test_gpu_paged import Batch

pytestmark = pytest.mark.gpu
DEV = "cuda"


def heads(t):
    s = t.stride()
    return up.Heads(t.data_ptr(), s[0] if t.dim() == 4 else 0, s[-3], s[-2], t.shape[-2])


def pages(kp, vp):
    return up.Pages(kp.data_ptr(), vp.data_ptr(), kp.shape[0], *kp.stride()[:3], kp.shape[1],
                    kp.shape[2], kp.shape[3])


@pytest.mark.parametrize("inter", [False, True])
def test_rotary(inter):
    q, k = torch.randn((2, 9, 4, 64), device=DEV).bfloat16(), torch.randn((2, 9, 2, 64), device=DEV).bfloat16()
    ph, m = up.rope_phases(32, scaling=up.UPIPE_ROPE_BY_PARTS, factor=4.0, trained_len=512)
    pos = torch.randint(0, 5000, (2, 9), device=DEV)
    for raw, call in ((up.upipe_rope_fwd, up.rope_forward), (up.upipe_rope_bwd, up.rope_backward)):
        for p, start in ((None, 700), (pos, 0)):
            qo, ko = torch.zeros_like(q), torch.zeros_like(k)
            raw(heads(q), heads(k), heads(qo), heads(ko), p, start, ph, m, 2, 9, 64, 32, inter)
            want = call(q, k, ph, m, inter, positions=p, start=start)
            assert torch.equal(qo, want[0]) and torch.equal(ko, want[1])
        with pytest.raises(up.UpipeError):
            raw(None, None, None, None, None, 0, ph, m, 2, 9, 64, 32, inter)


@pytest.mark.parametrize("packed", [False, True])
def test_append_and_attention(packed):
    counts = [2, 0, 1] if packed else [2, 2, 2]
    b = Batch(counts, [40, 7, 130], 8, 2, 128, 16, 50, seed=3, packed=packed)
    n = b.rows if packed else 2
    k, v = (torch.randn((*b.q.shape[:-2], 2, 128), device=DEV).bfloat16() for _ in range(2))
    ph, m = up.rope_phases(128)
    kp, vp, q2 = b.kp.clone(), b.vp.clone(), torch.zeros_like(b.q)
    want_q = up.kv_append(k, v, b.kp, b.vp, b.table, b.seq_len, q=b.q, phases=ph, start=50,
                          cu_seqlens=b.cu)
    ts, mp = b.table.stride(0), b.table.shape[1]
    up.upipe_kv_append(heads(b.q), heads(q2), heads(k), heads(v), pages(kp, vp), b.table, ts, mp,
                       b.seq_len, b.cu, None, 50, ph, m, 3, n, 128, False)
    bits = lambda t: t.contiguous().view(torch.int16)  # noqa: E731
    assert torch.equal(q2, want_q)
    assert torch.equal(bits(kp), bits(b.kp)) and torch.equal(bits(vp), bits(b.vp))
    b.q = q2
    o, lse = b.attend()
    o2, lse2 = torch.zeros_like(o), torch.zeros_like(lse)
    size = up.upipe_attn_paged_workspace_bytes(3, b.rows, 8, 2, 128, 50, n, mp * 16)
    ws = torch.empty(size, dtype=torch.uint8, device=DEV)
    args = (heads(q2), heads(o2), lse2, pages(kp, vp), b.table, ts, mp, b.seq_len, b.cu, b.ptable, 50,
            3, n, n, mp * 16, ws)
    up.upipe_attn_paged_fwd(*args)
    assert torch.equal(o2, o) and torch.equal(lse2, lse)
    with pytest.raises(up.UpipeError) as e:
        up.upipe_attn_paged_fwd(*args, workspace_bytes=size - 1)
    assert e.value.status == up.UPIPE_ERR_WORKSPACE_TOO_SMALL
    b.check(o, lse)
