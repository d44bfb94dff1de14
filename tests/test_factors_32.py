"""Factors that 64 bits hold and 32 bits do not are refused, as infinite ones are (no GPU): a kernel would
take them as infinite, and the zeros of a padded token, times that, are NaN.
"""
import pytest

import context_parallelism_gb300 as up
from tests.test_embed_api import _bwd as embed_bwd
from tests.test_embed_api import _fwd as embed_fwd
from tests.test_norm_api import N, _append
from tests.test_norm_api import _bwd as norm_bwd
from tests.test_norm_api import _fwd as norm_fwd
from tests.test_paged_api import C, FAKE, H, _rope

INV, OK = up.UPIPE_ERR_INVALID_ARG, up.UPIPE_OK


def _plain_append(mscale):
    return up._lib.upipe_kv_append(None, None, H(2), H(2), C(), FAKE, 4, 4, FAKE, None, None, 0, FAKE, mscale,
                                   0, 1, 64, 0, None)


@pytest.mark.parametrize("f,status", [(3e38, OK), (-3e38, OK), (1e39, INV), (-1e39, INV), (1e300, INV)])
def test_factors(f, status):
    calls = [embed_fwd(S=0, scale=f), embed_bwd(S=0, add=1, scale=f), norm_fwd(S=0, norm=N(offset=f)),
             norm_bwd(S=0, dqw=None, norm=N(offset=f)), _append(B=0, norm=N(offset=f)),
             norm_fwd(S=0, mscale=f), norm_bwd(S=0, dqw=None, mscale=f), _plain_append(f),
             _rope(S=0, q=H(), q_out=H(), mscale=f), _rope(S=0, q=H(), q_out=H(), mscale=f, back=True)]
    if f > 0:
        calls += [norm_fwd(S=0, norm=N(eps=f)), norm_bwd(S=0, dqw=None, norm=N(eps=f)),
                  _append(B=0, norm=N(eps=f))]
    assert calls == [status] * len(calls)
    assert status == OK or "finite" in up.upipe_last_error_message()
