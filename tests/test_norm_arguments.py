"""Arguments of the calls with head norms that would be ignored are refused (no GPU)."""
import pytest
import torch

import context_parallelism_gb300 as up


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
