"""Written tensors that overlap (themselves, or each other) are refused: two threads would write the
same element, in place even read what the other wrote. No GPU: addresses are made up, and a call that
passes every check before the device says that they are no device memory."""
import pytest
import torch

import context_parallelism_gb300 as up
from tests.test_paged_api import C, FAKE, H, _append, _attend, _rope

D, S, HEADS = 64, 8, 4


def _said(status):
    assert status == up.UPIPE_ERR_INVALID_ARG
    return up.upipe_last_error_message()


# strides of [B = 2, S = 8, heads = 4, D = 64]
FINE = [(2048, 256, 64),            # dense
        (2048, 64, 512),            # head-major
        (256, 512, 64),             # token-major over the batch
        (8192, 1024, 128),          # heads with gaps, as between keys and values
        (64, 128, 1024)]            # batch innermost
MEET = [(2048, 64, 64),             # windows over a sequence
        (2048, 128, 64),            # neighbouring tokens share half their heads
        (64, 256, 64),              # batch rows one head apart
        (2040, 256, 64),            # the last features of a row
        (1 << 62, 1 << 62, 64)]     # as far apart as batch rows


@pytest.mark.parametrize("st", FINE + MEET)
def test_self_overlap(st):
    t, dense = H(HEADS, *st), H(HEADS, 2048, 256, 64, data=FAKE * 64)
    meets = st in MEET
    cache = C(n_pages=2, page_size=16, heads=2)
    for said in (_said(_rope(q=t, q_out=t, B=2, S=S)),
                 _said(_rope(q=dense, q_out=t, B=2, S=S, back=True)),
                 _said(_append(q=dense, q_out=t, k=H(2, 1024, 128, 64), v=H(2, 1024, 128, 64),
                               cache=cache, B=2, S=S)),
                 _said(_attend(q=dense, o=t, cache=cache, B=2, S=S))):
        assert ("overlap" in said) == meets, said
    # inputs may overlap
    assert "overlap" not in _said(_rope(q=t, q_out=dense, B=2, S=S))


def test_extents_of_one_do_not_count():
    t = H(1, 0, 64, 8)
    assert "overlap" not in _said(_rope(q=t, q_out=t, B=1, S=S))


@pytest.mark.parametrize("kw", [dict(stride_slot=64), dict(stride_page=1024),
                                dict(stride_head=128, stride_slot=64, stride_page=128 * 8)])
def test_cache_slots_that_meet(kw):
    assert "overlap" in _said(_append(cache=C(**kw)))
    assert "overlap" not in _said(_attend(cache=C(**kw)))  # reading them is fine
    assert "overlap" not in _said(_append(cache=C(stride_head=16 * 64, stride_slot=64)))


def test_q_and_k_in_one_place():
    t, u = H(HEADS, 2048, 256, 64), H(HEADS, 2048, 256, 64, data=FAKE * 2)
    assert "one tensor" in _said(_rope(q=t, k=t, q_out=t, k_out=t, B=2, S=S))
    assert "one tensor" in _said(_rope(q=t, k=u, q_out=u, k_out=u, B=2, S=S, back=True))
    assert "one tensor" not in _said(_rope(q=t, k=t, q_out=t, k_out=u, B=2, S=S))


@pytest.mark.gpu
def test_one_tensor_as_q_and_k():
    x = torch.randn((2, 8, 4, 64), device="cuda").bfloat16()
    ph, _ = up.rope_phases(64)
    q, k = up.rope_forward(x, x, ph)
    torch.cuda.synchronize()
    assert torch.equal(q, k)
    x0 = x.clone()
    with pytest.raises(up.UpipeError):
        up.rope_forward(x, x, ph, inplace=True)
    torch.cuda.synchronize()
    assert torch.equal(x, x0)
