"""Arguments of the calls with head norms that would be ignored are refused, and refusals of gradients name
them (no GPU)."""
import pytest
import torch

import context_parallelism_gb300 as up
from tests.test_norm_api import _bwd, _fwd
from tests.test_paged_api import FAKE, H, _rope


def test_an_offset_without_its_norm():
    k, w = torch.zeros((1, 3, 2, 64), dtype=torch.bfloat16), torch.zeros(64, dtype=torch.bfloat16)
    kp = torch.zeros((4, 16, 2, 64), dtype=torch.bfloat16)
    table, lens = torch.zeros((1, 2), dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    for norm in (dict(offset=1.0), dict(offset=1.0, k_weight=w), dict(q_weight=w)):
        with pytest.raises(ValueError, match="eps"):
            up.kv_append(k, k, kp, kp.clone(), table, lens, **norm)
    for norm in (dict(offset=0.0), dict(), dict(offset=1.0, eps=1e-6)):
        with pytest.raises(up.UpipeError):  # host memory
            up.kv_append(k, k, kp, kp.clone(), table, lens, **norm)


@pytest.mark.parametrize("kw,name", [
    (dict(dqo=H(data=FAKE + 2)), "dq_out is not"), (dict(dq=H(data=FAKE + 2)), "dq is not"),
    (dict(dqo=H(ss=260)), "dq_out: strides"), (dict(dq=H(ss=0)), "dq: a written"),
    (dict(dq=H(3)), "dq_out and dq differ"), (dict(dko=H(), k=H(), dk=H()), "dq and dk are one"),
    (dict(dko=H(data=FAKE + 2), k=H(), dk=H()), "dk_out is not"),
    (dict(dko=H(), k=H(), dk=H(data=FAKE + 2)), "dk is not"),
    (dict(q=H(data=FAKE + 2)), "the forward's q is not"),
])
def test_gradients_by_their_names(kw, name):
    assert _bwd(**kw) == up.UPIPE_ERR_INVALID_ARG
    assert up.upipe_last_error_message().startswith(name)


def test_the_others_by_theirs():
    bad, good = H(data=FAKE + 2), H()
    for call, name in ((lambda: _rope(q=bad, q_out=good, back=True), "dq_out is not"),
                       (lambda: _rope(k=good, k_out=bad, back=True), "dk is not"),
                       (lambda: _rope(q=bad, q_out=good), "q is not"),
                       (lambda: _rope(k=good, k_out=bad), "k_out is not"),
                       (lambda: _fwd(q_out=bad), "q_out is not"),
                       (lambda: _fwd(k=good, k_out=good), "q_out and k_out are one")):
        assert call() == up.UPIPE_ERR_INVALID_ARG
        assert up.upipe_last_error_message().startswith(name)
