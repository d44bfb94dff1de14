"""The paged cache and the attention over it on the GPU against the 64-bit oracle (needs an
sm_103a GPU).

Tolerances, from the arithmetic. A score is an fp32 sum of D exact bf16 products: off by at most
ds = D 2^-23 sum_d |q_d k_d| / sqrt(D) (2^-23 a step covers adders that truncate). A weight is
exp2 of it (2 steps of fp32) rounded to bf16 (2^-8 of itself), so each is off by a factor within
1 +- dw, dw = 2^-8 + 2 ds + 2^-18, and numerator and denominator use the same weights:
|o - ref| <= (1 + dw) dw spread + 2^-8 |o| (one output rounding) + 2^-18 max |v| (fp32 sums over
at most 2^11 keys), where spread = sum_j P_j |v_j - o|. lse uses the unrounded weights:
|lse - ref| <= 2 ds + 2^-18 + 2^-22 |lse|.
"""
import numpy as np
import pytest
import torch

import context_parallelism_gb300 as up
from oracle import append_index_ref, paged_attn_ref, rope_ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
NAN = float("nan")


def _bf(shape, seed, scale=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(torch.bfloat16)


class Batch:
    """A random batch: sequences with counts[b] new tokens among lens[b] own ones in shuffled
    pages; unused slots hold NaN and infinities, unused table entries -1."""

    def __init__(self, counts, lens, Hq, Hkv, D, page, prefix, seed=0, packed=False,
                 head_major=False, behind=0, scale=1.0):
        self.counts, self.lens, self.prefix, self.page = counts, lens, prefix, page
        self.Hq, self.Hkv, self.D, self.packed = Hq, Hkv, D, packed
        rng = np.random.default_rng(seed)
        B = len(lens)
        need = [-(-m // page) for m in lens]
        shared = -(-prefix // page)
        n_pages = shared + sum(need) + 3
        perm = rng.permutation(n_pages)
        self.ptable_np = perm[:shared]
        self.table_np = np.full((B, max(1, max(need))), -1)
        at = shared
        for b in range(B):
            self.table_np[b, :need[b]] = perm[at:at + need[b]]
            at += need[b]
        shape = (n_pages, Hkv, page, D) if head_major else (n_pages, page, Hkv, D)
        kp, vp = _bf(shape, seed + 1, scale), _bf(shape, seed + 2)
        if head_major:
            kp, vp = kp.transpose(1, 2), vp.transpose(1, 2)
        used = torch.zeros((n_pages, page), dtype=torch.bool)
        for pages, n in [(self.ptable_np, prefix)] + list(zip(self.table_np, lens)):
            for j in range(0, n, page):
                used[int(pages[j // page]), :min(page, n - j)] = True
        kp[~used.to(DEV)] = NAN
        vp[~used.to(DEV)] = torch.tensor([float("inf"), NAN] * (D // 2), dtype=vp.dtype,
                                         device=DEV)
        self.kp, self.vp = kp, vp
        self.table = torch.tensor(self.table_np, dtype=torch.int32, device=DEV)
        self.ptable = torch.tensor(self.ptable_np, dtype=torch.int32, device=DEV)
        self.seq_len = torch.tensor(lens, dtype=torch.int32, device=DEV)
        self.rows = sum(counts)
        self.cu = None
        if packed:
            self.cu = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32,
                                   device=DEV)
            self.q = _bf((self.rows + behind, Hq, D), seed + 3, scale)
        else:
            self.q = _bf((B, counts[0], Hq, D), seed + 3, scale)

    def flat(self, t):
        return t.reshape(-1, *t.shape[-2:])[:self.rows]

    def attend(self, **kw):
        return up.paged_attention(self.q, self.kp, self.vp, self.table, self.seq_len,
                                  prefix_table=self.ptable if self.prefix else None,
                                  prefix_len=self.prefix, cu_seqlens=self.cu, with_lse=True, **kw)

    def check(self, o, lse):
        up.upipe_sync_status()
        ro, rl, spread, size = paged_attn_ref(self.flat(self.q), self.kp.cpu(), self.vp.cpu(),
                                              self.table_np, self.lens, self.counts,
                                              self.ptable_np, self.prefix)
        o = self.flat(o).double().cpu().numpy()
        lse = (lse.t() if self.packed else lse.transpose(1, 2).reshape(-1, self.Hq))
        lse = lse[:self.rows].double().cpu().numpy()
        ds = self.D * 2.0 ** -23 * size
        dw = (2.0 ** -8 + 2 * ds + 2.0 ** -18)[..., None]
        vmax = float(torch.nan_to_num(self.vp.float(), 0, 0, 0).abs().max())
        tol = (1 + dw) * dw * spread + 2.0 ** -8 * np.abs(ro) + 2.0 ** -18 * vmax
        assert np.isfinite(o).all()
        assert (np.abs(o - ro) <= tol).all(), float((np.abs(o - ro) - tol).max())
        empty = np.isneginf(rl)
        assert np.array_equal(np.isneginf(lse), empty) and (o[empty] == 0).all()
        d = np.abs(lse[~empty] - rl[~empty])
        lim = (2 * ds + 2.0 ** -18)[~empty] + 2.0 ** -22 * np.abs(rl[~empty])
        assert (d <= lim).all(), float((d - lim).max())


# (counts, lens, Hq, Hkv, D, page, prefix)
DECODE = {
    "one_key": ([1], [1], 4, 4, 64, 16, 0),
    "one_key_of_prefix": ([1], [1], 8, 1, 128, 16, 1),
    "tile_edges": ([1] * 9, [1, 15, 16, 17, 63, 64, 65, 128, 129], 4, 2, 128, 16, 0),
    "splits": ([1, 1], [1000, 257], 4, 1, 128, 64, 0),
    "empty_sequences": ([1] * 4, [0, 5, 0, 64], 4, 2, 64, 32, 0),
    "empty_own_with_prefix": ([1] * 3, [0, 1, 0], 8, 2, 128, 48, 77),
    "prefix_edges_127": ([1] * 3, [3, 70, 1], 8, 2, 128, 16, 127),
    "prefix_edges_128": ([1] * 3, [3, 70, 1], 8, 2, 64, 128, 128),
    "prefix_edges_129": ([1] * 3, [3, 70, 1], 8, 2, 128, 256, 129),
    "group_of_seven": ([1] * 5, [9, 33, 64, 100, 2], 28, 4, 128, 16, 300),
    "group_of_five_d64": ([1] * 4, [9, 33, 64, 100], 10, 2, 64, 80, 513),
    "mha_many_rows": ([1] * 130, [b % 7 + 1 for b in range(130)], 2, 2, 64, 16, 200),
    "long_prefix": ([1] * 20, [b + 1 for b in range(20)], 16, 2, 128, 64, 1500),
    "wide_group": ([1] * 2, [30, 90], 40, 1, 128, 32, 260),
}


@pytest.mark.parametrize("head_major", [False, True])
@pytest.mark.parametrize("case", list(DECODE))
def test_decode(case, head_major):
    counts, lens, Hq, Hkv, D, page, prefix = DECODE[case]
    b = Batch(counts, lens, Hq, Hkv, D, page, prefix, seed=len(case), head_major=head_major)
    b.check(*b.attend())


PREFIX = {  # shapes that the tensor-core kernel takes: one row tile, two, two and part of a third
    "one_tile_d64": ([1] * 25, [b % 9 for b in range(25)], 8, 2, 64, 32, 10777),
    "one_tile": ([1] * 32, [b % 5 + 1 for b in range(32)], 8, 2, 128, 16, 8321),
    "one_tile_small": ([3], [5], 8, 1, 128, 64, 44000),
    "two_tiles_d64": ([2] * 30, [b % 7 + 2 for b in range(30)], 8, 2, 64, 64, 4500),
    "two_tiles": ([1] * 18, [b % 3 for b in range(18)], 40, 4, 128, 256, 6001),
    "third_alone": ([1] * 75, [1] * 75, 4, 1, 128, 16, 900),
    "third_alone_d64": ([1] * 75, [2] * 75, 4, 1, 64, 128, 900),
    "many_d64": ([3] * 40, [b + 3 for b in range(40)], 16, 2, 64, 16, 1391),
}


@pytest.mark.parametrize("with_lse", [True, False])
@pytest.mark.parametrize("case", list(PREFIX))
def test_prefix_row_tiles(case, with_lse):
    counts, lens, Hq, Hkv, D, page, prefix = PREFIX[case]
    b = Batch(counts, lens, Hq, Hkv, D, page, prefix, seed=30 + len(case))
    o, lse = b.attend()
    if with_lse:
        b.check(o, lse)
        return
    # without lse (other weight sums are kept) the same o
    o2, none = up.paged_attention(b.q, b.kp, b.vp, b.table, b.seq_len, prefix_table=b.ptable,
                                  prefix_len=prefix)
    up.upipe_sync_status()
    assert none is None
    b.check(o2, lse)


@pytest.mark.parametrize("prefix", [100, 4000])
def test_one_row_on_long_own_pages_and_on_a_long_prefix(prefix):
    b = Batch([1], [3000], 8, 2, 128, 16, prefix, seed=33)
    b.check(*b.attend())
    b = Batch([1] * 2, [3000, 1], 4, 4, 64, 48, prefix, seed=34)
    b.check(*b.attend())


MULTI = {
    "draft": ([3] * 4, [3, 10, 67, 130], 8, 2, 128, 16, 140),
    "draft_d64": ([5] * 3, [5, 64, 65], 4, 4, 64, 16, 0),
    "chunk": ([70] * 2, [70, 200], 8, 2, 128, 64, 33),
    "chunk_mqa": ([40], [300], 8, 1, 64, 48, 129),
    "new_tokens_without_place": ([4] * 3, [2, 0, 9], 4, 2, 128, 16, 0),
    "many": ([9] * 16, [9 + 5 * b for b in range(16)], 16, 2, 128, 32, 700),
}


@pytest.mark.parametrize("case", list(MULTI))
def test_several_new_tokens(case):
    counts, lens, Hq, Hkv, D, page, prefix = MULTI[case]
    b = Batch(counts, lens, Hq, Hkv, D, page, prefix, seed=3 + len(case))
    b.check(*b.attend())


PACKED = {
    "zero_to_three": ([0, 1, 3, 0, 2], [0, 1, 60, 40, 2], 8, 2, 128, 16, 100),
    "one_long": ([1, 50, 1], [64, 50, 1000], 4, 1, 64, 32, 0),
    "nothing_but_one": ([0, 0, 1], [0, 7, 20], 8, 8, 128, 16, 65),
}


@pytest.mark.parametrize("hints", [None, (1, 1), (64, 2000)])
@pytest.mark.parametrize("case", list(PACKED))
def test_packed_rows_and_hints(case, hints):
    """Rows behind the last sequence stay as they are; hints far too small or too large change no
    result beyond the tolerance."""
    counts, lens, Hq, Hkv, D, page, prefix = PACKED[case]
    b = Batch(counts, lens, Hq, Hkv, D, page, prefix, seed=7, packed=True, behind=4)
    out = torch.full_like(b.q, 7.0)
    lse = torch.full((Hq, b.rows + 4), 7.0, device=DEV)
    b.q[b.rows:] = NAN
    kw = {} if hints is None else dict(max_q=hints[0], max_len=hints[1])
    b.check(*b.attend(out=out, lse=lse, **kw))
    assert (out[b.rows:] == 7).all() and (lse[:, b.rows:] == 7).all()


@pytest.mark.parametrize("counts,max_q", [([40, 3], 1), ([200], 16)])
def test_row_tiles_beyond_the_hint(counts, max_q):
    b = Batch(counts, [300, 50][:len(counts)], 4, 1, 128, 16, 0, seed=8, packed=True)
    b.check(*b.attend(max_q=max_q, max_len=64))


def test_large_scores_and_dominant_keys():
    """One key that takes a row over gives that key's value, scores of some hundreds give no
    infinities."""
    b = Batch([1] * 4, [40, 64, 100, 1], 8, 2, 128, 16, 300, seed=9, scale=4.0)
    b.kp[int(b.ptable_np[3]), 5] *= 8
    b.kp[int(b.table_np[2, 1]), 3] *= 16
    b.check(*b.attend())


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,G,prefix", [(40, 16, 1500), (24, 4, 4000)])
def test_scores_that_rise_along_the_prefix(n, G, prefix, D):
    """Two row tiles, and two key streams, of the tensor-core kernel: later keys whose scores lie tens,
    hundreds and thousands above all before them, for single heads' rows or for all."""
    b = Batch([1] * n, [9] * n, G, 1, D, 16, prefix, seed=12)
    up.upipe_sync_status()
    for at, by in ((200, 6.0), (300, 30.0), (301, 30.0), (700, 60.0), (1100, 400.0), (1400, 900.0)):
        b.kp[int(b.ptable_np[at // 16]), at % 16] *= by
    b.q[::3] *= 0.01
    b.check(*b.attend())


def test_strided_q_and_output():
    b = Batch([2] * 3, [5, 70, 33], 8, 2, 64, 16, 90, seed=10)
    o, lse = b.attend()
    wide = torch.full((3, 2, 12, 64), 3.0, dtype=torch.bfloat16, device=DEV)
    wide[:, :, :8] = b.q
    q = b.q
    b.q = wide[:, :, :8]
    out = torch.zeros((8, 2, 3, 64), dtype=torch.bfloat16, device=DEV).permute(2, 1, 0, 3)
    o2, lse2 = b.attend(out=out)
    b.q = q
    assert torch.equal(o2, o) and torch.equal(lse2, lse)
    b.check(o2, lse2)


def test_results_repeat_bitwise_and_on_another_stream():
    b = Batch([1] * 6, [500, 30, 64, 1, 0, 333], 16, 4, 128, 16, 1000, seed=11)
    o, lse = b.attend()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o2, lse2 = b.attend(stream=side)
    side.synchronize()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_cache_beyond_32_bit_offsets():
    """Pages whose element offsets pass 2^32 (a cache of 8.6 GB a side)."""
    ps, H, D = 16, 2, 128
    n = (1 << 32) // (ps * H * D) + 40
    kp = torch.empty((n, ps, H, D), dtype=torch.bfloat16, device=DEV)
    vp = torch.empty((n, ps, H, D), dtype=torch.bfloat16, device=DEV)
    pages = [n - 1, 3, n - 7, n // 2 + 1]
    small = Batch([1], [50], 4, H, D, ps, 0, seed=12)
    small.kp, small.vp = kp, vp
    small.table = torch.tensor([pages], dtype=torch.int32, device=DEV)
    k, v = _bf((50, H, D), 13), _bf((50, H, D), 14)
    up.kv_append(k, v, kp, vp, small.table, small.seq_len,
                 cu_seqlens=torch.tensor([0, 50], dtype=torch.int32, device=DEV))
    o, lse = small.attend()
    got = kp[pages].reshape(-1, H, D)[:50]
    assert torch.equal(got, k) and torch.equal(vp[pages].reshape(-1, H, D)[:50], v)
    # the oracle on a cache of these pages alone
    small.kp, small.vp = kp[pages].clone(), vp[pages].clone()
    del kp, vp
    small.kp.view(-1, H, D)[50:] = NAN
    small.table_np = np.array([[0, 1, 2, 3]])
    small.vp.view(-1, H, D)[50:] = NAN
    small.check(o, lse)


# ---- append ---------------------------------------------------------------------------------

def _check_append(b, k, v, kp0, vp0, ph, m, inter, start, q, q_out):
    """Every slot of the caches and every row of q_out."""
    up.upipe_sync_status()
    words = [int(w) % (1 << 64) for w in ph.tolist()] if ph is not None else None
    kf, vf = k.reshape(-1, *k.shape[-2:]), v.reshape(-1, *v.shape[-2:])
    qf, qo = q.reshape(-1, *q.shape[-2:]), q_out.reshape(-1, *q.shape[-2:])
    kp, vp = kp0.clone(), vp0.clone()
    bits = lambda t: t.contiguous().view(torch.int16)  # noqa: E731
    for row, s, j in append_index_ref(b.counts, b.lens):
        def near(y, x):
            if words is None:
                assert torch.equal(y, x)
                return
            ref = rope_ref(x[None], [start + j], words, m, inter)[0]
            size = x.double().abs().max().item()
            err = np.abs(y.double().cpu().numpy() - ref)
            # as for the rotary calls; 2 max |x| bounds a pair's |x1| + |x2|
            assert (err <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -20 * 2 * size * m).all()
        near(qo[row], qf[row])
        if j < 0:
            continue
        page, slot = int(b.table_np[s, j // b.page]), j % b.page
        near(b.kp[page, slot], kf[row])
        assert torch.equal(b.vp[page, slot], vf[row])
        kp[page, slot], vp[page, slot] = b.kp[page, slot], b.vp[page, slot]
    # nothing else moved
    assert torch.equal(bits(kp), bits(b.kp)) and torch.equal(bits(vp), bits(b.vp))


APPEND = {
    "one": ([1], [1], 4, 4, 64, 16, 64),
    "decode": ([1] * 6, [1, 16, 17, 0, 64, 333], 32, 8, 128, 16, 128),
    "part": ([1] * 3, [5, 6, 7], 7, 1, 128, 1, 32),
    "chunk": ([37] * 2, [37, 100], 8, 2, 128, 48, 128),
    "without_place": ([4] * 2, [2, 0], 4, 2, 64, 16, 64),
    "odd_head": ([3] * 2, [3, 9], 5, 5, 80, 7, 48),
}


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("case", list(APPEND))
def test_append(case, inter):
    counts, lens, Hq, Hkv, D, page, rot = APPEND[case]
    b = Batch(counts, lens, Hq, Hkv, D, page, 0, seed=20)
    k, v = _bf((len(lens), counts[0], Hkv, D), 21), _bf((len(lens), counts[0], Hkv, D), 22)
    kp0, vp0 = b.kp.clone(), b.vp.clone()
    ph, m = up.rope_phases(rot, scaling=up.UPIPE_ROPE_BY_PARTS, factor=4.0, trained_len=2048)
    q_out = up.kv_append(k, v, b.kp, b.vp, b.table, b.seq_len, q=b.q, phases=ph, mscale=m,
                         interleaved=inter, start=5000)
    _check_append(b, k, v, kp0, vp0, ph, m, inter, 5000, b.q, q_out)


@pytest.mark.parametrize("rotate", [True, False])
def test_append_packed_head_major_strided(rotate):
    counts, lens = [0, 2, 1, 0, 5], [0, 2, 40, 9, 33]
    b = Batch(counts, lens, 8, 2, 64, 16, 0, seed=23, packed=True, behind=3, head_major=True)
    x = _bf((b.rows + 3, (8 + 4) * 64), 24)
    q = x[:, :512].unflatten(-1, (8, 64))
    k, v = x[:, 512:640].unflatten(-1, (2, 64)), x[:, 640:].unflatten(-1, (2, 64))
    kp0, vp0 = b.kp.clone(), b.vp.clone()
    q0 = q.clone()
    ph, m = up.rope_phases(64) if rotate else (None, 1.0)
    q_out = torch.full_like(q0, 7.0)
    up.kv_append(k, v, b.kp, b.vp, b.table, b.seq_len, q=q, q_out=q_out, phases=ph,
                 cu_seqlens=b.cu, start=11)
    _check_append(b, k, v, kp0, vp0, ph, m, False, 11, q0, q_out)
    assert (q_out[b.rows:] == 7).all()
    # in place, and given positions (the same ones): the same
    pos = torch.zeros(b.rows + 3, dtype=torch.int64)
    for row, s, j in append_index_ref(counts, lens):
        pos[row] = 11 + j
    up.kv_append(k, v, b.kp, b.vp, b.table, b.seq_len, q=q, q_out=q, phases=ph,
                 cu_seqlens=b.cu, positions=pos.to(DEV))
    assert torch.equal(q[:b.rows], q_out[:b.rows]) and torch.equal(q[b.rows:], q0[b.rows:])
    _check_append(b, k, v, kp0, vp0, ph, m, False, 11, q0, q)


def test_append_without_q_and_into_a_prefix():
    """A prefix is filled as one sequence whose table lists its pages."""
    b = Batch([1], [1], 4, 2, 128, 32, 100, seed=25)
    k, v = _bf((1, 100, 2, 128), 26), _bf((1, 100, 2, 128), 27)
    ph, m = up.rope_phases(128)
    n = torch.tensor([100], dtype=torch.int32, device=DEV)
    assert up.kv_append(k, v, b.kp, b.vp, b.ptable[None], n, phases=ph) is None
    kr = up.rope_forward(None, k, ph, m)[1]
    pages = b.ptable.long()
    assert torch.equal(b.kp[pages].reshape(-1, 2, 128)[:100], kr[0])
    assert torch.equal(b.vp[pages].reshape(-1, 2, 128)[:100], v[0])
    b.check(*b.attend())


# ---- together ---------------------------------------------------------------------------------

def test_prefill_append_and_attend_agree_with_causal_attention():
    """The serving path: a prompt through rope_forward and attention_forward, its keys appended as
    the shared prefix; then steps of a few tokens a sequence, appended and attended. One sequence's
    steps give what causal attention over the whole gives in its last rows: both are within the
    attention's own 1e-2 of the exact result for values of this size, and the cached keys are the
    same roundings."""
    Hq, Hkv, D, P, steps, page = 8, 2, 128, 300, 5, 16
    S = P + steps
    ph, m = up.rope_phases(D, theta=500000.0)
    q, k, v = _bf((1, S, Hq, D), 30), _bf((1, S, Hkv, D), 31), _bf((1, S, Hkv, D), 32)
    qr, kr = up.rope_forward(q, k, ph, m)
    want, _ = up.attention_forward(qr, kr, v, with_lse=False)
    n_pages = -(-P // page) + 2
    kp = torch.full((n_pages, page, Hkv, D), NAN, dtype=torch.bfloat16, device=DEV)
    vp = torch.full_like(kp, NAN)
    ptable = torch.arange(2, n_pages, dtype=torch.int32, device=DEV).flip(0).contiguous()
    table = torch.tensor([[1], [0]], dtype=torch.int32, device=DEV)
    one = torch.tensor([P], dtype=torch.int32, device=DEV)
    up.kv_append(k[:, :P], v[:, :P], kp, vp, ptable[None], one, phases=ph)
    # two sequences: the first goes on with the prompt's own next tokens, the second with others
    q2, k2, v2 = _bf((1, steps, Hq, D), 33), _bf((1, steps, Hkv, D), 34), _bf((1, steps, Hkv, D), 35)
    for lo, hi in ((0, 1), (1, 2), (2, 5)):
        n = torch.tensor([hi, hi], dtype=torch.int32, device=DEV)
        cat = lambda a, b: torch.cat((a[:, P + lo:P + hi], b[:, lo:hi]))  # noqa: E731
        qn = up.kv_append(cat(k, k2), cat(v, v2), kp, vp, table, n, q=cat(q, q2), phases=ph,
                          start=P)
        assert torch.equal(qn[0], qr[0, P + lo:P + hi])
        o, _ = up.paged_attention(qn, kp, vp, table, n, prefix_table=ptable, prefix_len=P)
        up.upipe_sync_status()
        assert (o[0].float() - want[0, P + lo:P + hi].float()).abs().max() <= 2e-2
    assert torch.equal(kp[1, :steps], kr[0, P:])


def test_steps_captured_into_a_graph_and_two_graphs_with_their_own_workspaces():
    """A captured step follows lengths, tables and inputs that change between replays; two graphs
    with workspaces of their own replay side by side."""
    up.upipe_sync_status()
    runs, kept = [], []
    for seed in (40, 50):
        b = Batch([1] * 5, [3, 64, 200, 0, 17], 8, 2, 128, 16, 150, seed=seed)
        k, v = _bf((5, 1, 2, 128), seed + 5), _bf((5, 1, 2, 128), seed + 6)
        ph, _ = up.rope_phases(128)
        ws = torch.empty(up.upipe_attn_paged_workspace_bytes(5, 5, 8, 2, 128, 150, 1, 208),
                         dtype=torch.uint8, device=DEV)
        qn, o, lse = torch.empty_like(b.q), torch.empty_like(b.q), torch.empty((5, 8, 1), device=DEV)

        def step(b=b, k=k, v=v, ph=ph, ws=ws, qn=qn, o=o, lse=lse):
            up.kv_append(k, v, b.kp, b.vp, b.table, b.seq_len, q=b.q, q_out=qn, phases=ph,
                         start=150)
            up.paged_attention(qn, b.kp, b.vp, b.table, b.seq_len, prefix_table=b.ptable,
                               prefix_len=150, max_len=208, out=o, lse=lse, workspace=ws)
        step()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        runs.append((b, k, v, qn, o, lse, g))
        kept.append((ph, ws))  # a graph does not own what it was given
    for lens in ([3, 64, 200, 0, 17], [4, 61, 201, 0, 1]):
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        for (b, k, v, qn, o, lse, g), s in zip(runs, streams):
            b.lens = lens
            b.seq_len.copy_(torch.tensor(lens, dtype=torch.int32))
            b.q.copy_(_bf(b.q.shape, 60 + lens[0]))
            torch.cuda.synchronize()
        for (b, k, v, qn, o, lse, g), s in zip(runs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for b, k, v, qn, o, lse, g in runs:
            q = b.q
            b.q = qn
            b.check(o, lse)
            b.q = q


@pytest.mark.parametrize("counts,prefix", [([1] * 4, 0), ([1] * 4, 300), ([40] * 4, 0),
                                           ([3] * 48, 2100)])
def test_output_in_the_place_of_q(counts, prefix):
    """o may be q: rows finished by the first kernel, joined ones, and the tensor-core prefix."""
    b = Batch(counts, ([41, 500, 64, 45] * 12)[:len(counts)], 8, 1, 128, 16, prefix, seed=30)
    o, lse = b.attend()
    b.check(o, lse)
    q = b.q.clone()
    o2, lse2 = b.attend(out=b.q)
    assert o2 is b.q and torch.equal(o2, o) and torch.equal(lse2, lse)
    b.q = q


def test_sequences_that_name_the_same_pages():
    """Two continuations of one history read the same full pages and write their own last one."""
    b = Batch([1] * 2, [100, 105], 8, 2, 64, 16, 40, seed=31)
    b.table_np[1, :6] = b.table_np[0, :6]
    b.table = torch.tensor(b.table_np, dtype=torch.int32, device=DEV)
    b.check(*b.attend())


def test_calls_from_two_threads_on_two_streams():
    """Each call takes a workspace of its own: results do not depend on what runs beside them."""
    import threading
    bs = [Batch([1] * 6, [500, 30, 64, 1, 0, 2000], 16, 4, 128, 16, 1000, seed=32 + i)
          for i in range(2)]
    want = [b.attend() for b in bs]
    torch.cuda.synchronize()
    got = [[], []]

    def work(i):
        s = torch.cuda.Stream()
        for _ in range(20):
            got[i].append(bs[i].attend(stream=s))
        s.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for i in range(2):
        assert len(got[i]) == 20
        for o, lse in got[i]:
            assert torch.equal(o, want[i][0]) and torch.equal(lse, want[i][1])


def test_workspace_of_a_captured_call():
    """A workspace made inside a capture belongs to the graph: eager calls between the replays
    do not get its memory."""
    b = Batch([1] * 5, [3, 1300, 200, 0, 17], 8, 2, 128, 16, 150, seed=34)
    want = b.attend()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o, lse = b.attend()
    side = torch.cuda.Stream()
    for _ in range(10):
        g.replay()
        other = b.attend(stream=side)
    torch.cuda.synchronize()
    for x, y in (want, other):
        assert torch.equal(o, x) and torch.equal(lse, y)


def test_missing_pages_are_reported_and_stay_inside_the_cache():
    """A table entry that names no page (the kernels check it before they follow it): the append
    drops the token, attention reads zeros there, and the status word says so once."""
    up.upipe_sync_status()
    b = Batch([1] * 2, [20, 40], 4, 2, 64, 16, 0, seed=70)
    k, v = _bf((2, 1, 2, 64), 71), _bf((2, 1, 2, 64), 72)
    good = b.table.clone()
    kp0, vp0 = b.kp.clone(), b.vp.clone()
    for bad in (-1, b.kp.shape[0], 1 << 30):
        b.table.copy_(good)
        b.table[1, 2] = bad
        up.kv_append(k, v, b.kp, b.vp, b.table, b.seq_len)
        with pytest.raises(up.UpipeError) as e:
            up.upipe_sync_status()
        assert e.value.status == up.UPIPE_ERR_PAGE
        changed = (b.kp.view(torch.int16) != kp0.view(torch.int16)).flatten(1).any(1)
        assert changed.nonzero().flatten().tolist() in ([], [int(good[0, 1])])
        o, _ = b.attend()
        with pytest.raises(up.UpipeError) as e:
            up.upipe_sync_status()
        assert e.value.status == up.UPIPE_ERR_PAGE
        assert torch.isfinite(o).all()
        up.upipe_sync_status()  # cleared
    b.table.copy_(good)
    # a length beyond the table
    b.seq_len[0] = 16 * b.table.shape[1] + 1
    up.kv_append(k, v, b.kp, b.vp, b.table, b.seq_len)
    with pytest.raises(up.UpipeError) as e:
        up.upipe_sync_status()
    assert e.value.status == up.UPIPE_ERR_PAGE


def test_batches_without_rows():
    b = Batch([1], [1], 4, 2, 64, 16, 0, seed=80)
    e = torch.empty((0, 4, 64), dtype=torch.bfloat16, device=DEV)
    cu = torch.zeros(2, dtype=torch.int32, device=DEV)
    o, lse = up.paged_attention(e, b.kp, b.vp, b.table, b.seq_len, cu_seqlens=cu, with_lse=True)
    assert o.shape == (0, 4, 64) and lse.shape == (4, 0)
    kv = torch.empty((0, 2, 64), dtype=torch.bfloat16, device=DEV)
    up.kv_append(kv, kv, b.kp, b.vp, b.table, b.seq_len, cu_seqlens=cu)
    # rows, but none that a sequence owns
    q = _bf((3, 4, 64), 81)
    out = torch.full_like(q, 7.0)
    up.paged_attention(q, b.kp, b.vp, b.table, b.seq_len, cu_seqlens=cu, out=out)
    up.upipe_sync_status()
    assert (out == 7).all()
