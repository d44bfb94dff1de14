"""Refusals of the rotary and paged-cache calls, all before any device access (no GPU): bad
shapes, strides, alignments and missing tensors give a status and a message, through the C ABI
and through the binding."""
import ctypes

import pytest
import torch

import context_parallelism_gb300 as up

FAKE = 1 << 20  # an aligned non-null address; validation must fail before it is dereferenced
INV, UNS = up.UPIPE_ERR_INVALID_ARG, up.UPIPE_ERR_UNSUPPORTED


def H(heads=4, sb=4096, ss=512, sh=64, data=FAKE):
    return up.Heads(data, sb, ss, sh, heads)


def C(**kw):
    d = dict(k=FAKE, v=FAKE, n_pages=8, stride_page=16 * 128, stride_slot=128, stride_head=64,
             page_size=16, heads=2, D=64)
    d.update(kw)
    return up.Pages(*[d[n] for n, _ in up.Pages._fields_])


def _rope(q=None, k=None, q_out=None, k_out=None, pos=None, phase=FAKE, mscale=1.0, B=1, S=8,
          D=64, rot=64, inter=0, back=False):
    fn = up._lib.upipe_rope_bwd if back else up._lib.upipe_rope_fwd
    return fn(q, k, q_out, k_out, pos, 0, phase, mscale, B, S, D, rot, inter, None)


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("kw,status", [
    (dict(q=None), INV),                                       # neither q nor k
    (dict(q_out=None), INV),                                   # input without output
    (dict(q_out=H(5)), INV),                                   # heads differ
    (dict(q=H(ss=260), ), INV),                                # stride not a multiple of 8
    (dict(q=H(ss=-512)), INV),                                 # negative stride
    (dict(q_out=H(ss=0)), INV),                                # a written tensor that overlaps
    (dict(q=H(data=FAKE + 2)), INV),                           # alignment
    (dict(q=H(data=None)), INV),
    (dict(q=H(-1), q_out=H(-1)), INV),
    (dict(phase=None), INV),
    (dict(pos=FAKE + 4), INV),                                 # positions not 8-byte aligned
    (dict(inter=2), INV),
    (dict(mscale=float("nan")), INV),
    (dict(B=-1), INV),
    (dict(D=60), UNS), (dict(D=2048), UNS), (dict(rot=8), UNS), (dict(rot=24), UNS),
    (dict(rot=80), UNS), (dict(S=1 << 41), UNS),
    (dict(q=H(70000), q_out=H(70000)), UNS),
    (dict(), INV),                                             # not device memory
])
def test_rope_refusals(kw, status, back):
    a = dict(q=H(), q_out=H())
    a.update(kw)
    assert _rope(back=back, **a) == status, up.upipe_last_error_message()
    assert up.upipe_last_error_message()


def test_calls_without_rows_do_nothing():
    assert _rope(q=H(), q_out=H(), S=0) == up.UPIPE_OK
    assert _append(B=0) == up.UPIPE_OK
    assert _attend(S=0, workspace=None) == up.UPIPE_OK


def _append(q=None, q_out=None, k=H(2), v=H(2), cache=None, table=FAKE, ts=4, mp=4, lens=FAKE,
            cu=None, pos=None, phase=FAKE, mscale=1.0, B=2, S=1, rot=64, inter=0):
    return up._lib.upipe_kv_append(q, q_out, k, v, cache if cache is not None else C(), table, ts,
                                   mp, lens, cu, pos, 0, phase, mscale, B, S, rot, inter, None)


@pytest.mark.parametrize("kw,status", [
    (dict(k=None), INV), (dict(v=None), INV), (dict(k=H(4)), INV), (dict(v=H(1)), INV),
    (dict(q=H(4)), INV), (dict(q=H(4), q_out=H(3)), INV),
    (dict(cache=C(n_pages=0)), INV), (dict(cache=C(page_size=0)), INV),
    (dict(cache=C(stride_slot=32)), INV), (dict(cache=C(stride_head=68)), INV),
    (dict(cache=C(k=None)), INV), (dict(cache=C(v=FAKE + 8)), INV),
    (dict(cache=C(D=60, stride_head=64)), UNS), (dict(rot=24), UNS), (dict(rot=128), UNS),
    (dict(phase=None, cache=C(D=4, stride_head=64)), UNS),
    (dict(mp=0), INV), (dict(ts=3), INV), (dict(table=None), INV), (dict(lens=None), INV),
    (dict(lens=FAKE + 2), INV), (dict(cu=FAKE + 1), INV), (dict(inter=-1), INV),
    (dict(mscale=float("inf")), INV), (dict(S=1 << 32), UNS), (dict(B=-2), INV), (dict(), INV),
])
def test_append_refusals(kw, status):
    assert _append(**kw) == status, up.upipe_last_error_message()
    assert up.upipe_last_error_message()


def _attend(q=H(4), o=H(4), lse=None, cache=None, table=FAKE, ts=4, mp=4, lens=FAKE, cu=None,
            ptable=FAKE, prefix=16, B=2, S=1, max_q=1, max_len=64, workspace=FAKE, wb=1 << 30):
    return up._lib.upipe_attn_paged_fwd(q, o, lse, cache if cache is not None else C(), table, ts,
                                        mp, lens, cu, ptable, prefix, B, S, max_q, max_len,
                                        workspace, wb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), INV), (dict(o=None), INV), (dict(o=H(2)), INV), (dict(q=H(3), o=H(3)), INV),
    (dict(cache=C(page_size=8)), UNS), (dict(cache=C(page_size=24)), UNS),
    (dict(cache=C(D=80, stride_head=80, stride_slot=160)), UNS),
    (dict(cache=C(stride_page=0)), INV), (dict(cache=C(stride_page=1 << 39)), INV),
    (dict(prefix=-1), INV), (dict(ptable=None), INV), (dict(prefix=1 << 31), UNS),
    (dict(cu=FAKE, max_q=0), INV), (dict(max_len=0), INV),
    (dict(workspace=None), INV), (dict(workspace=FAKE + 16), INV),
    (dict(wb=16), up.UPIPE_ERR_WORKSPACE_TOO_SMALL),
    (dict(lse=FAKE + 2), INV), (dict(table=FAKE + 2), INV), (dict(mp=0), INV),
    (dict(o=H(4, sh=32)), INV),
    (dict(S=1 << 25), UNS), (dict(B=-1), INV), (dict(), INV),
])
def test_attend_refusals(kw, status):
    assert _attend(**kw) == status, up.upipe_last_error_message()
    assert up.upipe_last_error_message()


@pytest.mark.parametrize("pages,status", [
    (2045 * 4, UNS),                              # (2^21 + 1) row tiles, each 2045 + 3: 2^32 and more
    (2044 * 4, up.UPIPE_ERR_WORKSPACE_TOO_SMALL)  # below: the next check
])
def test_tiles_are_counted_in_32_bits(pages, status):
    """2^24 rows of 8 q-heads on one kv-head: 64-row tiles, 64-key tiles; each row tile counts two
    tiles more than its keys fill, and the table's last tile may be a part of one."""
    assert _attend(q=H(8), o=H(8), cache=C(heads=1), B=1, S=1 << 24, mp=pages, prefix=0,
                   max_len=1) == status, up.upipe_last_error_message()


def test_append_refuses_more_heads_than_a_launch_counts():
    assert _append(k=H(40000), v=H(40000), cache=C(heads=40000)) == UNS


@pytest.mark.parametrize("args", [
    (0, 4, 8, 2, 64, 0, 1, 64), (1, 0, 8, 2, 64, 0, 1, 64), (1, 4, 6, 4, 64, 0, 1, 64),
    (1, 4, 8, 2, 96, 0, 1, 64), (1, 4, 8, 2, 64, -1, 1, 64), (1, 4, 8, 2, 64, 0, 0, 64),
    (1, 4, 8, 2, 64, 0, 1, 0), (1, 1 << 25, 8, 2, 64, 0, 1, 64),
])
def test_workspace_zero_for_invalid(args):
    assert up.upipe_attn_paged_workspace_bytes(*args) == 0


def test_workspace_is_bounded_by_the_rows_and_the_blocks():
    """Pieces: a tile of rows each for every sequence's and kv-head's rows and every block, at
    most 304; prefix parts: rows x Hq each, at most 160 splits of two. D + 4 floats a row, and
    16 bytes a row and head for the descriptors. Nothing grows with the lengths beyond that."""
    for B, rows, Hq, Hkv, D, P, mq, ml in [(1, 1, 32, 8, 128, 0, 1, 131072),
                                           (64, 64, 32, 8, 128, 32768, 1, 1500),
                                           (96, 240, 64, 8, 128, 131000, 5, 700),
                                           (1, 1, 4, 4, 64, 0, 1, 1)]:
        ws = up.upipe_attn_paged_workspace_bytes(B, rows, Hq, Hkv, D, P, mq, ml)
        mt = 64
        segs = (rows * Hq // Hkv // mt + B + 1) * Hkv * (2 if P else 1)
        most = ((segs + 304) * mt + (320 * rows * Hq if P else 0)) * (D + 4) * 4
        assert 0 < ws <= most + 16 * rows * Hq + 5 * 256
        assert up.upipe_attn_paged_workspace_bytes(B, rows, Hq, Hkv, D, P, mq, 1 << 30) <= \
            most + 16 * rows * Hq + 5 * 256


@pytest.mark.parametrize("hint", [1 << 31, 1 << 40, 1 << 58, (1 << 63) - 1])
def test_length_hints_of_any_size(hint):
    for args in [(64, 64, 32, 8, 128, 1000, 1), (1, 1, 32, 8, 64, 0, 1 << 62), (3, 40, 8, 8, 64, 0, 40)]:
        assert up.upipe_attn_paged_workspace_bytes(*args, hint) == \
            up.upipe_attn_paged_workspace_bytes(*args, (1 << 31) - 1) > 0


def _t(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def test_binding_refusals():
    ph = torch.zeros(32, dtype=torch.int64)
    q, k = _t(1, 3, 4, 64), _t(1, 3, 2, 64)
    for bad in (lambda: up.rope_forward(None, None, ph),
                lambda: up.rope_forward(q, _t(1, 4, 2, 64), ph),
                lambda: up.rope_forward(q[0], None, ph),
                lambda: up.rope_forward(q.transpose(2, 3), None, ph),
                lambda: up.rope_forward(q, k, ph.int()),
                lambda: up.rope_forward(q, k, ph, positions=torch.zeros(3, dtype=torch.int64)),
                lambda: up.rope_forward(q, k, ph, positions=torch.zeros(1, 3)),
                lambda: up.rope_phases(32, inv_freq=[1.0], device="cpu")):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        up.rope_forward(q.float(), None, ph)
    with pytest.raises(up.UpipeError):  # host memory
        up.rope_forward(q, k, ph)

    kp, vp = _t(6, 16, 2, 64), _t(6, 16, 2, 64)
    table, lens = torch.zeros((1, 2), dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    for bad in (lambda: up.kv_append(k[:, :1], k[:, :1], kp, vp, table, lens.long()),
                lambda: up.kv_append(k[:, :1], k[:, :1], kp, vp, table.long(), lens),
                lambda: up.kv_append(k[:, :1], k, kp, vp, table, lens),
                lambda: up.kv_append(k[0], k[0], kp, vp, table, lens),
                lambda: up.kv_append(k, k, kp, vp, table, lens, cu_seqlens=lens),
                lambda: up.kv_append(k, k, kp, vp.transpose(1, 2), table, lens),
                lambda: up.kv_append(k, k, kp, vp[:5], table, lens),
                lambda: up.paged_attention(q, kp, vp, table, lens, prefix_len=3),
                lambda: up.paged_attention(q, kp, vp, table, lens, prefix_table=table[0],
                                           prefix_len=33),
                lambda: up.paged_attention(_t(1, 3, 4, 128), kp, vp, table, lens),
                lambda: up.paged_attention(q, kp, vp, table, lens, out=q[:, :1]),
                lambda: up.paged_attention(q, kp, vp, table, lens, lse=torch.zeros(4, 3))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        up.paged_attention(q.half(), kp, vp, table, lens)


def test_status_string_of_missing_pages():
    assert up.upipe_status_string(up.UPIPE_ERR_PAGE) == "UPIPE_ERR_PAGE"
    assert ctypes.sizeof(up.Heads) == 40 and ctypes.sizeof(up.Pages) == 64
