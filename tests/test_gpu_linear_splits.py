"""Weight gradients whose tiles are split into six to eight shares: the partial sums stay in their part of the
workspace, and dz, which lies behind them, is whole while dW reads it."""
import pytest
import torch

import output_head_kl_b200 as K
from tests import test_gpu_linear as TL

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
# widths at which the shares of 192-wide tiles take more room than those of 256-wide ones
CASES = [(2048, 256, 8, 80192), (3503, 248, 64, 80192), (2048, 256, 256, 80192), (2048, 512, 768, 80192),
         (1536, 256, 512, 60192), (1800, 456, 264, 70192), (2048, 1024, 200, 80192)]


@pytest.mark.parametrize("M,d_in,d_out,plan", CASES)
def test_shares_stay_in_the_workspace(M, d_in, d_out, plan):
    dy, pre, x, W = TL._grad_data(M, d_in, d_out, seed=30)
    size = K.kdkl_linear_workspace_bytes(M, d_in, d_out, True)
    room = torch.full((size + (4 << 20),), 0x5A, dtype=torch.uint8, device="cuda")
    dW = torch.empty(d_out, d_in, dtype=BF, device="cuda")
    K.kdkl_linear_backward(dy, x, None, None, dW, room[:size], pre=pre, activation="silu", dw_plan=plan)
    assert K.kdkl_read_device_flags(room[:size]) == 0
    assert bool((room[size:] == 0x5A).all())


@pytest.mark.parametrize("M,d_in,d_out,plan", CASES)
def test_weight_gradient_of_many_shares(M, d_in, d_out, plan):
    args = TL._grad_data(M, d_in, d_out, seed=31)
    TL._check_grad(*args, "silu", dw_plan=plan, want=("dW",))
    both = TL._grad(*args, "silu", dw_plan=plan)
    alone = TL._grad(*args, "silu", dw_plan=plan, want=("dW",))
    assert torch.equal(both[1], alone[1])      # dx, which uses the same workspace first, changes nothing
