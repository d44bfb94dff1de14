"""Infinities and NaN at keys that a row must not see, in calls with several new tokens a sequence
(needs an sm_103a GPU).

A later token's key and value belong to rows from that token on: earlier rows, and rows without a
place in the cache, give what the definition gives over the keys that they see, whatever the later
ones hold. Tolerances: those of tests/test_gpu_paged.py for the finite elements, with the term of
the fp32 sums taken from the case: a key's 2^-23 of the largest value for each step of a sum, 16 keys
a step where the matrix instruction takes them and one where a row's keys are added one by one (at
most two tiles of 64 of them), and one step for each of up to 2432 parts joined in eights.
"""
import numpy as np
import pytest
import torch

from oracle import paged_attn_ref
from tests.test_gpu_paged import Batch
import context_parallelism_gb300 as up

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


def check(b, o, lse):
    """Finite elements within the tolerance, infinities and NaN where the definition has them."""
    up.upipe_sync_status()
    with np.errstate(invalid="ignore"):
        ro, rl, spread, size = paged_attn_ref(b.flat(b.q), b.kp.cpu(), b.vp.cpu(), b.table_np,
                                              b.lens, b.counts, b.ptable_np, b.prefix)
    o = b.flat(o).double().cpu().numpy()
    lse = lse.t() if b.packed else lse.transpose(1, 2).reshape(-1, b.Hq)
    lse = lse[:b.rows].double().cpu().numpy()
    assert np.array_equal(np.isnan(o), np.isnan(ro))
    assert np.array_equal(np.isposinf(o), np.isposinf(ro))
    assert np.array_equal(np.isneginf(o), np.isneginf(ro))
    fin = np.isfinite(ro)
    ds = b.D * 2.0 ** -23 * size
    dw = np.broadcast_to((2.0 ** -8 + 2 * ds + 2.0 ** -18)[..., None], ro.shape)[fin]
    vmax = float(torch.nan_to_num(b.vp.float(), 0, 0, 0).abs().max())
    steps = (b.prefix + max(b.lens)) / 16 + 128 + 2432 / 8
    tol = (1 + dw) * dw * spread[fin] + 2.0 ** -8 * np.abs(ro[fin]) + steps * 2.0 ** -23 * vmax
    assert (np.abs(o[fin] - ro[fin]) <= tol).all()
    assert np.array_equal(np.isnan(lse), np.isnan(rl))
    assert np.array_equal(np.isneginf(lse), np.isneginf(rl))
    ok = np.isfinite(rl)
    assert (np.abs(lse[ok] - rl[ok]) <= (2 * ds + 2.0 ** -18)[ok] + 2.0 ** -22 * np.abs(rl[ok])).all()
    return fin


# (counts, lens, Hq, Hkv, D, page, prefix): 8-row, 16-row and 64-row tiles, with and without a
# prefix, one piece and several, a prefix on the tensor cores
CASES = {
    "tile8": ([2] * 4, [2, 16, 17, 130], 8, 2, 128, 16, 0),
    "tile8_d64": ([5] * 3, [5, 64, 65], 4, 4, 64, 16, 90),
    "tile16": ([3] * 4, [3, 10, 67, 130], 8, 2, 128, 16, 140),
    "tile16_d64": ([4] * 3, [4, 500, 33], 12, 3, 64, 32, 0),
    "tile16_long": ([4], [3000], 4, 1, 128, 16, 0),
    "tile64": ([70] * 2, [70, 200], 8, 2, 128, 64, 33),
    "tile64_d64": ([40], [300], 8, 1, 64, 48, 0),
    "without_place": ([4] * 3, [2, 0, 9], 4, 2, 64, 16, 50),
    "without_place_64": ([30] * 2, [3, 29], 4, 2, 128, 16, 0),
    "tensor_prefix": ([3] * 40, [3 + 2 * b for b in range(40)], 8, 1, 128, 16, 2100),
}


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("case", list(CASES))
def test_values_behind_a_rows_own_key(case, packed):
    counts, lens, Hq, Hkv, D, page, prefix = CASES[case]
    if packed:  # sequences of different numbers of new tokens, one of them none
        counts = [n - (b % 2) for b, n in enumerate(counts)] + [0]
        lens = lens + [20]
    b = Batch(counts, lens, Hq, Hkv, D, page, prefix, seed=90 + len(case), packed=packed)
    for s, (n, m) in enumerate(zip(counts, lens)):
        for back, (f, x) in enumerate([(0, INF), (3, -INF), (D - 1, NAN), (D // 2 + 5, INF)]):
            j = m - 1 - back
            if j > max(m - n, 0):  # not the first new token's: some row must not see it
                b.vp[int(b.table_np[s, j // page]), j % page, :, f] = x
    fin = check(b, *b.attend())
    assert not fin.all() and fin.any()


def test_keys_behind_a_rows_own_key():
    for counts, lens, D in (([3] * 2, [10, 40], 128), ([40], [100], 64)):
        b = Batch(counts, lens, 8, 2, D, 16, 70, seed=97)
        j = lens[0] - 1
        b.kp[int(b.table_np[0, j // 16]), j % 16, 0, 7] = NAN
        check(b, *b.attend())
