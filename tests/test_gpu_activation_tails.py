"""The linear layer's activations and their slopes far from zero, element by element against the float64 definition.

The pre-activation is exact: x holds bf16 values z, W is the identity.  Tolerances (U = 2^-24, half an fp32
step): the exponent z^2 / 2 of the normal tail and density carries up to 4 U, 2 z^2 U of the value; the exponential
(2 ulp), the other factors of the tail and the products add 16 U.  A bf16 output adds half a bf16 step, 2^-8 of the
value.
"""
import math

import pytest
import torch

import output_head_kl_b200 as K

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF = torch.bfloat16
D = 512
TAIL = -torch.linspace(3.0, 11.0, D, dtype=torch.float64)
HUGE = torch.tensor([s * v for v in (1e3, 1e5, 1e10, 1e18, 6e18, 1e19, 7e19, 1e20, 1e25, 1e30, 1e38, 3.3e38)
                     for s in (1.0, -1.0)], dtype=torch.float64)


def _cdf(z):
    return 0.5 * torch.special.erfc(-z / math.sqrt(2.0))


def _forward(z, act, rows, plan):
    """act of `rows` rows that all hold z."""
    x = z.to("cuda", BF).repeat(rows, 1)
    d = z.numel()
    W = torch.eye(d, device="cuda", dtype=BF)
    y = torch.empty(rows, d, dtype=BF, device="cuda")
    ws = torch.empty(K.kdkl_linear_workspace_bytes(rows, d, d), dtype=torch.uint8, device="cuda")
    K.kdkl_linear_forward(x, W, y, ws, activation=act, plan=plan)
    return y.double().cpu()


def _slopes(z, act):
    """act'(z) in fp32: the column sums of one row with dy = 1."""
    d = z.numel()
    db = torch.empty(d, device="cuda")
    ws = torch.empty(K.kdkl_linear_workspace_bytes(1, 8, d, True), dtype=torch.uint8, device="cuda")
    K.kdkl_linear_backward(torch.ones(1, d, dtype=BF, device="cuda"), None, None, None, None, ws,
                           pre=z.to("cuda", BF).view(1, d), dbias=db, activation=act)
    return db.double().cpu()


@pytest.mark.parametrize("rows,plan", [(1, 0), (300, 256), (600, 20128)])
def test_gelu_of_negative_values(rows, plan):
    z = TAIL.to(BF).double()
    y = _forward(z, "gelu", rows, plan)
    want = (z * _cdf(z)).expand_as(y)
    assert bool(((y - want).abs() <= (2.0 ** -8 + (2 * z * z + 16) * U) * want.abs()).all())


def test_gelu_slope_of_negative_values():
    z = TAIL.to(BF).double()
    a, b = _cdf(z), z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    assert bool(((_slopes(z, "gelu") - (a + b)).abs() <= (2 * z * z + 16) * U * (a.abs() + b.abs())).all())


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu", "relu"])
def test_slopes_of_huge_values(act):
    """0 or 1 and never NaN, as far as bf16 reaches."""
    z = HUGE.to(BF).double()
    assert bool(torch.isfinite(z).all())
    assert torch.equal(_slopes(z, act), (z > 0).double())


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu", "relu"])
@pytest.mark.parametrize("rows,plan", [(1, 0), (300, 256)])
def test_huge_values(act, rows, plan):
    z = HUGE.to(BF).double()
    y = _forward(z, act, rows, plan)
    assert torch.equal(y, torch.where(z > 0, z, 0.0).expand_as(y))


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu", "relu"])
def test_nan_passes(act):
    z = torch.full((8,), float("nan"), dtype=torch.float64)
    assert bool(torch.isnan(_slopes(z, act)).all()) and bool(torch.isnan(_forward(z, act, 1, 0)).all())
