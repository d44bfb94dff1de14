"""Streams that a caller names in the rotary and paged-cache calls: what the binding allocates (and
zeroes) is allocated for the stream that the kernels run on, whether that is a torch stream, a
handle or the default stream's handle 0."""
import contextlib

import pytest
import torch

import context_parallelism_gb300 as up

DEV = "cuda"


class _Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


def test_allocations_follow_the_handle(monkeypatch):
    """Without a GPU, torch's stream functions replaced: handle 0 is the default stream. (As an
    ExternalStream, 0 is some stream of torch's pool, whose zero-fill nothing orders before the
    kernel.)"""
    seen = []

    @contextlib.contextmanager
    def stream(s):
        seen.append(s.cuda_stream)
        yield

    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: _Stream(0))
    monkeypatch.setattr(torch.cuda, "ExternalStream",
                        lambda h, device=None: _Stream(h if h else 0x1234))
    like = torch.ones(3, 4)
    for given, handle in ((0, 0), (77, 77), (_Stream(5), 5)):
        out = up._empty(given, like, (2, 5), torch.float32, zero=True)
        assert out.shape == (2, 5) and (out == 0).all()
        assert seen.pop() == handle and not seen


@pytest.mark.gpu
def test_the_default_streams_handle():
    """stream=0, again and again on a packed batch with rows behind it: the rows are the same and
    those behind are zero."""
    rows, behind = 40, 20000
    kp = torch.zeros((8, 16, 2, 64), dtype=torch.bfloat16, device=DEV)
    vp = torch.zeros_like(kp)
    table = torch.arange(8, dtype=torch.int32, device=DEV)[None, :3].contiguous()
    lens = torch.tensor([rows], dtype=torch.int32, device=DEV)
    cu = torch.tensor([0, rows], dtype=torch.int32, device=DEV)
    x = torch.randn((rows + behind, 8, 64), device=DEV).bfloat16()
    q, k, v = x[:, :4], x[:, 4:6], x[:, 6:]
    ph, _ = up.rope_phases(64)
    kw = dict(q=q, phases=ph, cu_seqlens=cu)
    qr = up.kv_append(k, v, kp, vp, table, lens, **kw)
    o, lse = up.paged_attention(qr, kp, vp, table, lens, cu_seqlens=cu, with_lse=True)
    torch.cuda.synchronize()
    for _ in range(20):
        q2 = up.kv_append(k, v, kp, vp, table, lens, stream=0, **kw)
        o2, lse2 = up.paged_attention(q2, kp, vp, table, lens, cu_seqlens=cu, with_lse=True, stream=0)
        torch.cuda.synchronize()
        assert torch.equal(q2, qr) and torch.equal(o2, o) and torch.equal(lse2, lse)
        assert (q2[rows:] == 0).all() and (o2[rows:] == 0).all() and (lse2[:, rows:] == 0).all()
    a, b = up.rope_forward(q[None], None, ph, stream=0)[0], up.rope_forward(q[None], None, ph)[0]
    torch.cuda.synchronize()
    assert torch.equal(a, b)
    up.upipe_sync_status()


@pytest.mark.gpu
@pytest.mark.parametrize("call", [up.rope_forward, up.rope_backward])
def test_rotary_outputs_keep_the_inputs_layout_on_any_stream(call):
    ph, _ = up.rope_phases(64)
    q = torch.randn((2, 4, 30, 64), device=DEV).bfloat16().transpose(1, 2)  # head-major
    k = torch.randn((2, 30, 12, 64), device=DEV).bfloat16()[:, :, 3:5]
    want = call(q, k, ph)
    assert want[0].stride() == q.stride()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (side, side.cuda_stream, 0):
        got = call(q, k, ph, stream=stream)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b) and a.stride() == b.stride()
