"""The shared prefix on the tensor cores in the forms in which steps use it: packed batches, captured
graphs, calls beside each other (needs an sm_103a GPU).

Every case asks how many kernels ran: two without the tensor-core prefix kernel (own keys, join),
three with it, so that a moved border cannot take these tests off it unseen. Tolerances: those of
tests/test_gpu_paged_masked.py, whose fp32 term counts the steps of the case's sums.
"""
import threading

import numpy as np
import pytest
import torch

import context_parallelism_gb300 as up
from tests.test_gpu_paged import Batch, _bf
from tests.test_gpu_paged_masked import check

pytestmark = pytest.mark.gpu
DEV = "cuda"
NAN = float("nan")


def counted(call):
    n = up.upipe_launch_count()
    out = call()
    return out, up.upipe_launch_count() - n


# (counts, lens, Hq, Hkv, D, page, prefix, max_q): with max_q the own keys go to 8- or 16-row tiles,
# without it to 64-row ones
PACKED = {
    "one_tile": ([0, 1, 3, 0, 2, 2], [0, 1, 60, 40, 2, 333], 8, 2, 128, 16, 8321, 3),
    "one_tile_64": ([0, 1, 3, 0, 2, 2], [0, 1, 60, 40, 2, 333], 8, 2, 128, 48, 22000, None),
    "one_tile_d64": ([2, 0, 1, 4], [5, 0, 1, 130], 16, 4, 64, 32, 7000, 4),
    "one_tile_d64_64": ([2, 0, 1, 4], [5, 0, 1, 130], 16, 4, 64, 128, 25000, None),
    "two_tiles": ([3, 0, 1, 2] * 8, [3, 0, 70, 9] * 8, 8, 2, 128, 64, 1800, 3),
    "two_tiles_64": ([20, 0, 15, 7], [20, 33, 90, 300], 8, 2, 128, 16, 6001, 20),
    "two_tiles_d64": ([4, 1, 0, 2] * 6, [64, 1, 0, 65] * 6, 4, 1, 64, 16, 1700, 4),
    # 20 and 17 rows a sequence and kv-head: the border to the prefix kernel lies four times as high
    "below_the_border": ([5, 1, 0, 2] * 5, [64, 1, 0, 65] * 5, 4, 1, 64, 16, 1700, 5),
    "two_tiles_d64_64": ([30, 0, 21], [30, 7, 200], 8, 2, 64, 64, 5500, 30),
    "third_in_part": ([1, 2, 0] * 45, [1, 5, 2] * 45, 4, 2, 128, 256, 1100, 2),
    "third_of_no_sequence": ([1] * 62, [2] * 62, 4, 1, 64, 16, 1300, 1),
    "one_row": ([0, 0, 1], [4, 0, 17], 16, 1, 128, 16, 9000, 1),
    "below_the_border_17": ([0, 0, 1], [4, 0, 17], 17, 1, 128, 16, 9000, 1),
}


@pytest.mark.parametrize("with_lse", [True, False])
@pytest.mark.parametrize("case", list(PACKED))
def test_packed_rows(case, with_lse):
    """Sequences without a row, NaN in the q rows behind the last sequence; those rows of o and lse
    stay as they are."""
    counts, lens, Hq, Hkv, D, page, prefix, max_q = PACKED[case]
    b = Batch(counts, lens, Hq, Hkv, D, page, prefix, seed=len(case), packed=True, behind=4)
    b.q[b.rows:] = NAN
    b.q[b.rows + 1:, :, 5] = float("inf")
    out, lse = torch.full_like(b.q, 7.0), torch.full((Hq, b.rows + 4), 7.0, device=DEV)
    kernels = 2 if case.startswith("below") else 3
    (o, l), n = counted(lambda: b.attend(out=out, lse=lse, max_q=max_q))
    assert n == kernels and o is out and l is lse
    if not with_lse:
        lone = torch.full_like(b.q, 7.0)
        (_, none), n = counted(lambda: up.paged_attention(
            b.q, b.kp, b.vp, b.table, b.seq_len, prefix_table=b.ptable, prefix_len=prefix,
            cu_seqlens=b.cu, max_q=max_q, out=lone))
        assert n == kernels and none is None
        o = lone
    check(b, o, lse)
    assert (o[b.rows:] == 7).all() and (lse[:, b.rows:] == 7).all()


def test_packed_rows_that_start_late():
    """cu_seqlens may start above zero: the rows before the first sequence are no sequence's."""
    b = Batch([2, 1, 3], [2, 40, 9], 8, 2, 128, 16, 9000, seed=4, packed=True, behind=3)
    o, lse = b.attend(max_q=3)
    late = Batch([2, 1, 3], [2, 40, 9], 8, 2, 128, 16, 9000, seed=4, packed=True, behind=3)
    late.cu = late.cu + 3
    late.q = b.q.roll(3, 0)
    late.q[:3] = NAN
    out, lse2 = torch.full_like(b.q, 7.0), torch.full_like(lse, 7.0)
    (_, _), n = counted(lambda: late.attend(max_q=3, out=out, lse=lse2))
    assert n == 3
    up.upipe_sync_status()
    assert (out[:3] == 7).all() and (lse2[:, :3] == 7).all()
    check(b, out[3:], lse2[:, 3:])


@pytest.mark.parametrize("shape", [(8, 2, 128, 16, 8400), (16, 1, 64, 32, 7000)])
def test_captured_steps(shape):
    """A captured append and attention with the prefix kernel: lengths, the division of the rows among
    the sequences and the inputs change between replays."""
    Hq, Hkv, D, page, prefix = shape
    b = Batch([3, 1, 0, 4], [30, 200, 20, 70], Hq, Hkv, D, page, prefix, seed=6, packed=True, behind=2)
    shp = (b.rows + 2, Hkv, D)
    k, v = _bf(shp, 61), _bf(shp, 62)
    ph, _ = up.rope_phases(D)
    ws = torch.empty(up.upipe_attn_paged_workspace_bytes(4, b.rows + 2, Hq, Hkv, D, prefix, 4, 256),
                     dtype=torch.uint8, device=DEV)
    qn, o = torch.zeros_like(b.q), torch.zeros_like(b.q)
    lse = torch.zeros((Hq, b.rows + 2), device=DEV)

    def step():
        up.kv_append(k, v, b.kp, b.vp, b.table, b.seq_len, q=b.q, q_out=qn, phases=ph, start=prefix,
                     cu_seqlens=b.cu)
        up.paged_attention(qn, b.kp, b.vp, b.table, b.seq_len, prefix_table=b.ptable,
                           prefix_len=prefix, cu_seqlens=b.cu, max_q=4, max_len=256, out=o, lse=lse,
                           workspace=ws)

    up.upipe_sync_status()
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        _, n = counted(step)
    assert n == 4  # append, prefix, own keys, join
    for r, (counts, lens) in enumerate([([3, 1, 0, 4], [30, 200, 20, 70]),
                                        ([0, 2, 4, 1], [10, 180, 17, 70]),
                                        ([1, 1, 1, 1], [1, 1, 1, 1])]):
        b.counts, b.lens, b.rows = counts, lens, sum(counts)
        b.cu.copy_(torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32))
        b.seq_len.copy_(torch.tensor(lens, dtype=torch.int32))
        b.q.copy_(_bf(b.q.shape, 63 + r))
        k.copy_(_bf(shp, 70 + r))
        torch.cuda.synchronize()
        g.replay()
        g.replay()  # once more behind itself: the same workspace, the same slots
        torch.cuda.synchronize()
        q = b.q
        b.q = qn
        check(b, o, lse)
        b.q = q


def test_two_streams_and_two_threads():
    """Calls beside each other, each with a workspace of its own, give what they give alone."""
    bs = [Batch([1] * 32, [7 * i + 1 for i in range(32)], 8, 2, 128, 16, 9000, seed=81),
          Batch([2] * 40, [900 - 20 * i for i in range(40)], 8, 2, 64, 32, 7000, seed=82)]
    want = []
    for b in bs:
        out, n = counted(b.attend)
        assert n == 3
        want.append(out)
    torch.cuda.synchronize()
    for b, (o, lse) in zip(bs, want):
        check(b, o, lse)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(10):  # one thread, two streams
        for i in range(2):
            got[i].append(bs[i].attend(stream=streams[i]))
    torch.cuda.synchronize()

    def work(i):
        for _ in range(10):
            got[i].append(bs[i].attend(stream=streams[i]))
        streams[i].synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    up.upipe_sync_status()
    for i in range(2):
        assert len(got[i]) == 20
        for o, lse in got[i]:
            assert torch.equal(o, want[i][0]) and torch.equal(lse, want[i][1])


def test_counters_name_the_kernels():
    b = Batch([1] * 32, [5] * 32, 8, 2, 128, 16, 9000, seed=83)
    torch.cuda.synchronize()
    up.upipe_profile_enable(True)
    try:
        up.upipe_profile_read()
        b.attend()
        torch.cuda.synchronize()
        stats = up.upipe_profile_read()
    finally:
        up.upipe_profile_enable(False)
    ran = {k: n for k, (_, n) in stats.items() if n}
    assert ran == {"attn_prefix": 1, "attn_paged": 1, "paged_merge": 1}
