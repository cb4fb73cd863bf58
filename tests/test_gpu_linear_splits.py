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


@pytest.fixture
def debug_lib(monkeypatch):
    monkeypatch.setattr(K, "_lib", None)
    monkeypatch.setattr(K, "LIB_PATH", K.DEBUG_LIB_PATH)
    yield
    monkeypatch.setattr(K, "_lib", None)


def test_bounds_checking_build(debug_lib):
    """The same plans, every kind of forward tile and the column sums through the library that checks shares,
    tickets, direct loads and stores: the results hold, and no check fails (TL._check and _check_grad read the flags)."""
    assert K.lib()._name == K.DEBUG_LIB_PATH
    for M, d_in, d_out, plan in CASES:
        TL._check_grad(*TL._grad_data(M, d_in, d_out, seed=32), "gelu", dw_plan=plan)
    for f8 in (False, True):
        for plan in (1016, 2064, 8128, 128, 20192, 40256):
            TL._check(TL._data(130, 2048, 136, f8, seed=33), "gelu", pre=True, plan=plan)
    TL._check(TL._data(5000, 576, 2088, seed=34), "silu", pre=True, plan=20256, rows=slice(4700, 5000))
