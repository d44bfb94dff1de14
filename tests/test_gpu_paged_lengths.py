"""Lengths at and beyond what the page table holds (needs an sm_103a GPU)."""
import numpy as np
import pytest
import torch

import context_parallelism_gb300 as up
from tests.test_gpu_paged import Batch

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _page_error():
    with pytest.raises(up.UpipeError) as e:
        up.upipe_sync_status()
    assert e.value.status == up.UPIPE_ERR_PAGE


# (counts, own tokens that the table holds, Hq, Hkv, D, page, prefix)
@pytest.mark.parametrize("case", [
    ([1], 96, 8, 2, 128, 16, 0), ([3], 64, 4, 4, 64, 32, 0), ([4], 160, 8, 2, 128, 16, 90),
    ([40], 192, 8, 2, 64, 64, 0), ([40], 192, 8, 1, 128, 64, 30), ([2], 48, 8, 1, 128, 16, 40000)])
@pytest.mark.parametrize("beyond", [1, 2, 3, 50, 10 ** 6])
def test_attention_with_a_length_beyond_the_table(case, beyond):
    """Row i of n new tokens sees own keys 0 .. len - n + i, of which the table holds the first
    `cap`: what a table wide enough would give, less the keys behind this one."""
    up.upipe_sync_status()
    counts, cap, Hq, Hkv, D, page, prefix = case
    n = counts[0]
    b = Batch(counts, [cap], Hq, Hkv, D, page, prefix, seed=60)
    b.seq_len[0] = cap + beyond
    o, lse = b.attend()
    _page_error()
    assert b.table.shape[1] * page == cap
    for i in range(n):
        see = min(cap, cap + beyond - n + i + 1)
        one = Batch([1], [see], Hq, Hkv, D, page, prefix, seed=60)
        # a decode step of this row alone, on the same pages
        one.q, one.kp, one.vp = b.q[:, i:i + 1].contiguous(), b.kp, b.vp
        one.table, one.table_np = b.table, b.table_np
        one.ptable, one.ptable_np = b.ptable, b.ptable_np
        one.check(o[:, i:i + 1], lse[:, :, i:i + 1])


def test_the_longest_sequence():
    """2^31 - 1024 own keys, the most that is supported: 64 pages named in turn by a table that is
    exactly as wide, so each of their 1024 keys counts 2^21 - 1 times. One more is reported.

    Tolerance: 1216 warps sum 1.77 million keys each. A lane's sum of weights takes 4 of a tile's 32
    keys one after the other, 2^-24 a step; a numerator 2 steps a tile, 2^-23 each: 220753 2^-24 and
    110377 2^-23 of the sums, 0.0264, beside the weights' own 2^-8."""
    up.upipe_sync_status()
    n = (1 << 31) - 1024
    g = torch.Generator(device=DEV).manual_seed(5)
    kp, vp, q = (torch.randn(s, generator=g, device=DEV).bfloat16()
                 for s in ((64, 16, 1, 64), (64, 16, 1, 64), (1, 1, 2, 64)))
    table = (torch.arange(n // 16, dtype=torch.int32, device=DEV) % 64)[None]
    lens = torch.tensor([n], dtype=torch.int32, device=DEV)
    o, lse = up.paged_attention(q, kp, vp, table, lens, with_lse=True)
    up.upipe_sync_status()
    k, v = kp.view(-1, 64).double().cpu(), vp.view(-1, 64).double().cpu()
    s = q[0, 0].double().cpu() @ k.t() / 8
    want = torch.softmax(s, -1) @ v
    off = 220753 * 2.0 ** -24 + 110377 * 2.0 ** -23 + 2.0 ** -8
    assert (o[0, 0].double().cpu() - want).abs().max() <= 2 * off * v.abs().max()
    assert (lse[0, :, 0].double().cpu() - torch.logsumexp(s, -1) - np.log(n // 1024)).abs().max() <= 2 * off
    lens += 1
    up.paged_attention(q, kp, vp, table, lens)
    _page_error()
