"""Rows of zeros (padding) with eps = 0: y, the e4m3 scale and the row's share of the gradient are zero, and the
rows around them are what they are alone.  Tolerances as in test_gpu_rmsnorm.py."""
import pytest
import torch

import output_head_kl_b200 as K
from oracle import layers as L
from tests import test_gpu_rmsnorm as TN

pytestmark = pytest.mark.gpu

BF, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
ZERO = (0, 3, 4, 11)
# a warp per row, a block per row with and without asynchronous copies
SHAPES = [(1300, 256), (12, 4096), (12, 8200), (300, 2880)]


def _rows(N, d, t, seed):
    x, _, gamma = TN._data(N, d, t, t, t, seed)
    x[list(ZERO)] = 0
    keep = [n for n in range(N) if n not in ZERO]
    return x, gamma, keep


@pytest.mark.parametrize("N,d", SHAPES)
@pytest.mark.parametrize("t", [BF, F32], ids=["bf16", "f32"])
def test_forward(N, d, t):
    x, gamma, keep = _rows(N, d, t, seed=21)
    _, y, _ = TN._forward(x, None, gamma, BF, eps=0.0)
    _, q, s = TN._forward(x, None, gamma, F8, eps=0.0)
    assert bool((y[list(ZERO)] == 0).all()) and bool((s[list(ZERO)] == 0).all())
    assert bool((q.float()[list(ZERO)] == 0).all())
    _, yo = L.rmsnorm(TN._f64(x[keep]), None, TN._f64(gamma), 0.0)
    yo = torch.from_numpy(yo)
    assert bool(((y[keep].double().cpu() - yo).abs() <= (2.0 ** -8 + TN.C * TN.U) * yo.abs() + TN.TINY).all())
    so = yo.abs().amax(dim=1) / 448
    assert bool(((s[keep].double().cpu() - so).abs() <= TN.C * TN.U * so).all())


@pytest.mark.parametrize("N,d", SHAPES)
@pytest.mark.parametrize("t", [BF, F32], ids=["bf16", "f32"])
def test_backward(N, d, t):
    h, gamma, keep = _rows(N, d, t, seed=22)
    dy = torch.randn(N, d, device="cuda").to(BF)
    dh = torch.randn(N, d, device="cuda").to(t)
    dx, dg = TN._grad(dy, h, gamma, dh, eps=0.0)
    assert torch.equal(dx[list(ZERO)], dh[list(ZERO)])
    ho, dyo = TN._f64(h[keep]), TN._f64(dy[keep])
    dxo, dgo = (torch.from_numpy(v) for v in L.rmsnorm_grad(dyo, ho, TN._f64(gamma), 0.0, TN._f64(dh[keep])))
    assert bool(torch.isfinite(dx).all())
    a, r = dyo * TN._f64(gamma), 1 / (ho * ho).mean(axis=1, keepdims=True) ** 0.5
    terms = torch.from_numpy(abs(r * a) + abs(ho) * r ** 3 * abs(a * ho).mean(axis=1, keepdims=True)) \
        + dh[keep].double().cpu().abs()
    tol = TN.HALF[t] * dxo.abs() + 2 * TN.C * TN.U * terms + TN.TINY
    assert bool(((dx[keep].double().cpu() - dxo).abs() <= tol).all())
    share = torch.from_numpy(abs(dyo * ho * r).sum(axis=0))
    assert bool(((dg.double().cpu() - dgo).abs() <= (TN.C + 128) * TN.U * share).all())


def test_zero_rows_through_the_8bit_layer():
    """The scale of a row of zeros is a number: the 8-bit layer fed by it gives the bias."""
    N, d, n = 5, 256, 64
    x, gamma = torch.zeros(N, d, dtype=BF, device="cuda"), torch.ones(d, dtype=BF, device="cuda")
    _, q, s = TN._forward(x, None, gamma, F8, eps=0.0)
    W = torch.randn(n, d, device="cuda").to(F8)
    bias = torch.randn(n, device="cuda").to(BF)
    y = torch.empty(N, n, dtype=BF, device="cuda")
    ws = torch.empty(K.kdkl_linear_workspace_bytes(N, d, n), dtype=torch.uint8, device="cuda")
    K.kdkl_linear_forward(q, W, y, ws, bias=bias, x_scale=s, w_scale=torch.ones(n, device="cuda"))
    assert torch.equal(y, bias.expand(N, n))
