"""Both norms' gradients where a workgroup takes two and three tokens one after
the other: the next token's rows loaded in place of the ones at work, the slots of
LDS that take turns, the gates' dots added up a token later, d_weight's part over
several tokens.  The checks are test_gpu_norm's, against FP64."""
import pytest
import torch

import fp8_block_scaled_bias_amd as M
import test_gpu_norm as N

pytestmark = pytest.mark.gpu


def workgroups(T, H):
    """(each has a part of d_weight in the workspace)"""
    return M.moe_norm_backward_workspace_bytes(T, H) // (4 * H)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,H", [(4101, 64), (2500, 1032), (1027, 7168), (1027, 8192), (1029, 8200)])
def test_norm_backward(T, H, dtype):
    P = workgroups(T, H)
    assert 2 * P < T < 3 * P or H == 1032 and P < T
    N.test_norm_backward(T, H, dtype)


@pytest.mark.parametrize("T,k,H,shared,norm,dtypes", [
    (4101, 8, 64, 1, 1, "both"), (4101, 1, 64, 0, 0, "both"), (4099, 3, 128, 1, 1, "both"), (1027, 8, 4224, 1, 1, "bf16"),
    (1027, 2, 7168, 1, 1, "both"), (1027, 1, 8192, 1, 1, "bf16"), (1027, 1, 8192, 0, 1, "f32"), (1029, 2, 8200, 1, 1, "bf16")])
def test_combine_norm_backward(T, k, H, shared, norm, dtypes):
    P = workgroups(T, H)
    assert P == M.moe_combine_norm_backward_workspace_bytes(T, H) // (4 * H) and 2 * P < T < 3 * P
    for dtype in dict(both=(torch.float32, torch.bfloat16), bf16=(torch.bfloat16,), f32=(torch.float32,))[dtypes]:
        N.test_combine_norm_backward(T, k, H, shared, norm, dtype)
