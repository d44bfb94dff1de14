"""Lengths at and beyond what the page table holds (needs an sm_103a GPU)."""
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
