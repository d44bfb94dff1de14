"""fp64 CPU oracles of the rotary positions, the paged cache and the attention over it.

TEST INFRASTRUCTURE ONLY. Plain definitions, row by row, sharing no code with the CUDA path.

Rotary: each pair of features times the complex number mscale e^{i a}. The angle a of position p
is 2 pi frac(p * phase / 2^64) in exact integer arithmetic, for phases as the library keeps them
(tests pin them against p * f in 64-bit floating point).
Attention: full score rows, the whole row's softmax at once. Besides o and lse it returns, per
element of o, the spread sum_j P_j |v_j - o|: what one relative error in every weight can move o
by, from which the tests derive their tolerance.
"""
from __future__ import annotations

import math

import numpy as np

from .attn_ref import _f64

__all__ = ["rope_ref", "append_index_ref", "paged_attn_ref"]


def rope_ref(x, pos, phases, mscale=1.0, interleaved=False, back=False):
    """x [..., S, H, D] rotated by pos [..., S] (ints of any size); phases: unsigned 64-bit words."""
    x = _f64(x).copy()
    rot = 2 * len(phases)
    pos = np.asarray(pos, dtype=object)
    turns = np.empty(pos.shape + (len(phases),))
    for at in np.ndindex(pos.shape):
        for i, w in enumerate(phases):
            turns[at + (i,)] = (int(pos[at]) * int(w) % 2 ** 64) / 2.0 ** 64
    z = mscale * np.exp((-2j if back else 2j) * math.pi * turns)[..., None, :]
    if interleaved:
        a, b = x[..., 0:rot:2].copy(), x[..., 1:rot:2].copy()
    else:
        a, b = x[..., :rot // 2].copy(), x[..., rot // 2:rot].copy()
    y = (a + 1j * b) * z
    if interleaved:
        x[..., 0:rot:2], x[..., 1:rot:2] = y.real, y.imag
    else:
        x[..., :rot // 2], x[..., rot // 2:rot] = y.real, y.imag
    return x


def append_index_ref(counts, lens):
    """(row, sequence, index in the sequence's pages) of every row of a packed batch."""
    out, row = [], 0
    for b, (n, m) in enumerate(zip(counts, lens)):
        for i in range(n):
            out.append((row, b, m - n + i))
            row += 1
    return out


def _gather(cache, pages, n, h):
    """First n tokens of kv-head h in the pages listed."""
    ps = cache.shape[1]
    ids = [int(pages[j // ps]) for j in range(0, n, ps)]
    if not ids:
        return np.zeros((0, cache.shape[-1]))
    return _f64(cache[ids][:, :, h]).reshape(-1, cache.shape[-1])[:n]


def paged_attn_ref(q, k_pages, v_pages, table, lens, counts, prefix_table=None, prefix_len=0):
    """q [rows, Hq, D] packed by counts. Returns o, lse [rows, Hq], spread [rows, Hq, D] and
    the largest sum_d |q_d k_d| / sqrt(D) of each row over the keys it sees."""
    q = _f64(q)
    rows, Hq, D = q.shape
    Hkv = k_pages.shape[2]
    G = Hq // Hkv
    o, spread = np.zeros((rows, Hq, D)), np.zeros((rows, Hq, D))
    lse, size = np.full((rows, Hq), -np.inf), np.zeros((rows, Hq))
    for h in range(Hkv):
        pk = _gather(k_pages, prefix_table, prefix_len, h)
        pv = _gather(v_pages, prefix_table, prefix_len, h)
        row = 0
        for b, (n, m) in enumerate(zip(counts, lens)):
            k = np.concatenate([pk, _gather(k_pages, table[b], m, h)])
            v = np.concatenate([pv, _gather(v_pages, table[b], m, h)])
            for i in range(n):
                see = prefix_len + max(0, m - n + i + 1)
                for e in range(h * G, (h + 1) * G):
                    if not see:
                        continue
                    s = k[:see] @ q[row, e] / math.sqrt(D)
                    top = s.max()
                    p = np.exp(s - top)
                    lse[row, e] = top + math.log(p.sum())
                    p /= p.sum()
                    o[row, e] = p @ v[:see]
                    spread[row, e] = p @ np.abs(v[:see] - o[row, e])
                    size[row, e] = (np.abs(k[:see]) @ np.abs(q[row, e])).max() / math.sqrt(D)
                row += 1
    return o, lse, spread, size
