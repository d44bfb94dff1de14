"""A workspace of any type counts by its bytes (no GPU: past the check of its size the call refuses host
memory)."""
import pytest
import torch

import context_parallelism_gb300 as up


@pytest.mark.parametrize("dtype", [torch.uint8, torch.bfloat16, torch.float32, torch.int64])
def test_bytes_not_elements(dtype):
    t, dh = torch.zeros(6, dtype=torch.int64), torch.zeros((6, 16), dtype=torch.bfloat16)
    need = up.upipe_embed_workspace_bytes(6, 16, 9)
    size = torch.empty(0, dtype=dtype).element_size()
    for n, status in ((need // size, up.UPIPE_ERR_INVALID_ARG), (need // size - 1, up.UPIPE_ERR_WORKSPACE_TOO_SMALL)):
        with pytest.raises(up.UpipeError) as e:
            up.embed_backward(t, dh, 9, workspace=torch.empty(n, dtype=dtype))
        assert e.value.status == status
