"""RMS norm with residual (bf16 and e4m3 output) and its gradient on the GPU vs the float64 oracle.

Tolerances (U = 2^-24, half an fp32 step).  The sum of squares of a row adds at most 64 terms in
sequence in a thread, five shuffle steps in the warp and five across warps, each within U of a sum
of non-negative terms, so its relative error is below 80 U and that of 1 / sqrt(.), with its own roundings,
below 50 U; C = 128 covers it and the products that follow.  A bf16 output adds half a bf16 step, 2^-8 of the
value; an e4m3 one half a step, 2^-4 of the value or, below 2^-6 of the scale, 2^-10 of the scale.
"""
import numpy as np
import pytest
import torch

import output_head_kl_b200 as K
from oracle import layers as L

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
C = 128
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 0.0}
TINY = 2.0 ** -133        # half the smallest bf16 step
BF, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
EPS = 1e-5


def _f64(t):
    return t.double().cpu().numpy()


def _data(N, d, xt, ht, gt, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    chan = torch.exp(torch.randn(d, generator=g, device="cuda"))
    x = torch.randn(N, d, generator=g, device="cuda").to(xt)
    r = (torch.randn(N, d, generator=g, device="cuda") * chan).to(ht)
    gamma = (1 + 0.3 * torch.randn(d, generator=g, device="cuda")).to(gt)
    return x, r, gamma


def _forward(x, r, gamma, yt, with_h=True, eps=EPS):
    N, d = x.shape
    y = torch.full((N, d), float("nan"), device="cuda").to(yt)
    ht = r.dtype if r is not None else x.dtype
    h = torch.full((N, d), float("nan"), device="cuda").to(ht) if with_h else None
    scale = torch.full((N,), float("nan"), device="cuda") if yt == F8 else None
    K.kdkl_rmsnorm_forward(x, gamma, y, residual=r, h=h, y_scale=scale, eps=eps)
    torch.cuda.synchronize()
    return h, y, scale


def _check_forward(x, r, gamma, yt, with_h=True):
    h, y, scale = _forward(x, r, gamma, yt, with_h)
    ho, yo = L.rmsnorm(_f64(x), _f64(r) if r is not None else None, _f64(gamma), EPS)
    if h is not None:
        assert np.all(np.abs(_f64(h) - ho) <= (HALF[h.dtype] + U) * np.abs(ho) + TINY)
    if yt == BF:
        assert np.all(np.abs(_f64(y) - yo) <= (2.0 ** -8 + C * U) * np.abs(yo) + TINY)
        return
    so = np.abs(yo).max(axis=1) / 448.0
    s = _f64(scale)
    assert np.all(np.abs(s - so) <= C * U * so)
    err = np.abs(_f64(y) * s[:, None] - yo)
    assert np.all(err <= (2.0 ** -4 + 2 * C * U) * np.abs(yo) + (2.0 ** -10 + 2 * C * U) * so[:, None])
    # away from rounding borders the stored value is the nearest e4m3 value itself
    q, _ = L.e4m3_rows(yo)
    assert np.mean(_f64(y) != q) < 2e-4


# every way a row is held: a warp per row (d <= 1024 and rows enough), a block per row with 1 to 8 steps a
# thread, few and many rows, rows that end inside a step
SHAPES = [(1, 8), (1, 4096), (3, 24), (700, 8), (700, 264), (333, 520), (1003, 896), (150, 1024), (151, 1032),
          (600, 2880), (299, 4096), (320, 8192), (5, 8200), (400, 16384), (2, 32768), (300, 32768)]


@pytest.mark.parametrize("N,d", SHAPES)
@pytest.mark.parametrize("out", [BF, F8], ids=["bf16", "e4m3"])
def test_forward(N, d, out):
    _check_forward(*_data(N, d, BF, BF, BF, seed=N + d), out)


@pytest.mark.parametrize("xt,ht,gt", [(BF, F32, BF), (F32, F32, F32), (F32, BF, F32), (BF, BF, F32)])
@pytest.mark.parametrize("out", [BF, F8], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("N,d", [(77, 2880), (500, 264)])
def test_forward_types(N, d, xt, ht, gt, out):
    _check_forward(*_data(N, d, xt, ht, gt, seed=5), out)


@pytest.mark.parametrize("out", [BF, F8], ids=["bf16", "e4m3"])
def test_forward_without_residual_and_without_h(out):
    x, r, gamma = _data(300, 640, BF, BF, BF, seed=6)
    _check_forward(x, None, gamma, out, with_h=True)
    _check_forward(x, None, gamma, out, with_h=False)
    _check_forward(x, r, gamma, out, with_h=False)


@pytest.mark.parametrize("d", [64, 4096])
def test_forward_special_rows(d):
    """A row of zeros, a tiny row, rows with a NaN and an infinity; their neighbours are not touched."""
    x, _, gamma = _data(200, d, F32, F32, F32, seed=7)
    x[3] = 0
    x[5] = 1e-38
    x[7, 1] = float("nan")
    x[9, 2] = float("inf")
    _, y, _ = _forward(x, None, gamma, BF)
    _, q, s = _forward(x, None, gamma, F8)
    y, q, s = _f64(y), _f64(q), _f64(s)
    assert np.all(y[3] == 0) and s[3] == 0 and np.all(q[3] == 0)
    _, yo = L.rmsnorm(_f64(x[5:6]), None, _f64(gamma), EPS)          # 1e-38 / sqrt(eps) * gamma
    assert np.all(np.abs(q[5] * s[5] - yo[0]) <= 2.0 ** -3 * np.abs(yo[0]))
    assert np.all(np.isnan(y[7])) and np.isnan(s[7]) and np.all(np.isnan(q[7]))
    assert np.isnan(y[9, 2]) and np.all(y[9, 3:] == 0) and np.isnan(s[9])
    for n in (2, 4, 6, 8, 10):
        _, yo = L.rmsnorm(_f64(x[n:n + 1]), None, _f64(gamma), EPS)
        assert np.all(np.abs(y[n] - yo[0]) <= (2.0 ** -8 + C * U) * np.abs(yo[0]) + TINY)


def test_forward_in_place():
    """h over residual, h over x, and y over x: the documented overlaps give the same bits."""
    for d in (512, 4096):
        x, r, gamma = _data(300, d, BF, BF, BF, seed=8)
        h, y, _ = _forward(x, r, gamma, BF)
        r2, y2 = r.clone(), torch.empty_like(y)
        K.kdkl_rmsnorm_forward(x, gamma, y2, residual=r2, h=r2, eps=EPS)
        assert torch.equal(r2, h) and torch.equal(y2, y)
        x2 = x.clone()
        K.kdkl_rmsnorm_forward(x2, gamma, y2, residual=r, h=x2, eps=EPS)
        assert torch.equal(x2, h) and torch.equal(y2, y)
        x3, h3 = x.clone(), torch.empty_like(h)
        K.kdkl_rmsnorm_forward(x3, gamma, x3, residual=r, h=h3, eps=EPS)
        assert torch.equal(h3, h) and torch.equal(x3, y)


def test_rows_behind_the_last_are_left():
    x, r, gamma = _data(260, 1032, BF, BF, BF, seed=9)
    y = torch.full((261, 1032), 7.0, dtype=BF, device="cuda")
    h = torch.full((261, 1032), 7.0, dtype=BF, device="cuda")
    K.kdkl_rmsnorm_forward(x, gamma, y[:260], residual=r, h=h[:260], eps=EPS)
    assert bool((y[260] == 7).all()) and bool((h[260] == 7).all())


# ------------------------------------------------------------------ gradient
def _grad(dy, h, gamma, dh, eps=EPS):
    N, d = h.shape
    dx = torch.full_like(h, float("nan"))
    dg = torch.full((d,), float("nan"), device="cuda")
    ws = torch.full((K.kdkl_rmsnorm_workspace_bytes(N, d),), 255, dtype=torch.uint8, device="cuda")
    K.kdkl_rmsnorm_backward(dy, h, gamma, dx, dg, ws, dh=dh, eps=eps)
    torch.cuda.synchronize()
    return dx, dg


def _check_grad(dy, h, gamma, dh):
    dx, dg = _grad(dy, h, gamma, dh)
    dyo, ho, go = _f64(dy), _f64(h), _f64(gamma)
    dho = _f64(dh) if dh is not None else np.zeros_like(ho)
    dxo, dgo = L.rmsnorm_grad(dyo, ho, go, EPS, dho)
    r = 1 / np.sqrt((ho * ho).mean(axis=1, keepdims=True) + EPS)
    a = dyo * go
    # what the fp32 arithmetic adds up for one element: r a, h r^3 mean|a h|, dh
    terms = np.abs(r * a) + np.abs(ho) * r ** 3 * np.abs(a * ho).mean(axis=1, keepdims=True) + np.abs(dho)
    assert np.all(np.abs(_f64(dx) - dxo) <= HALF[dx.dtype] * np.abs(dxo) + 2 * C * U * terms + TINY)
    # dgamma: at most N / 592 + 1 <= 4 rows in sequence (64 for the row counts here with few blocks), four warps,
    # 37 partial sums and 16 groups, on top of each term's own error
    assert np.all(np.abs(_f64(dg) - dgo) <= (C + 128) * U * np.abs(dyo * ho * r).sum(axis=0) + 1e-30)


@pytest.mark.parametrize("N,d", SHAPES)
def test_backward(N, d):
    h, dh, gamma = _data(N, d, BF, BF, BF, seed=N + d + 1)
    dy = torch.randn(N, d, device="cuda").mul_(1e-3).to(BF)
    _check_grad(dy, h, gamma, dh)


@pytest.mark.parametrize("ht,gt", [(F32, F32), (F32, BF), (BF, F32)])
@pytest.mark.parametrize("N,d", [(1003, 896), (161, 2880), (2000, 72), (40, 7680), (40, 7688), (3, 8192), (70, 8200),
                                 (5, 16392), (2, 32768)])
def test_backward_types(N, d, ht, gt):
    h, dh, gamma = _data(N, d, ht, ht, gt, seed=11)
    dy = torch.randn(N, d, device="cuda").to(BF)
    _check_grad(dy, h, gamma, dh)
    _check_grad(dy, h, gamma, None)


def test_backward_against_differences():
    """dx and dgamma against central differences of the GPU forward itself (fp32 stream, e4m3-free)."""
    x, r, gamma = _data(4, 16, F32, F32, F32, seed=12)
    r = torch.randn_like(r)
    w = torch.randn(4, 16, device="cuda").to(BF)
    dx, dg = _grad(w, x + r, gamma, None)
    ho = _f64(x) + _f64(r)

    def f(hv, gv):
        return (_f64(w) * L.rmsnorm(hv, None, gv, EPS)[1]).sum()
    for i in np.ndindex(4, 16):
        a, b = ho.copy(), ho.copy()
        a[i] += 1e-5
        b[i] -= 1e-5
        num = (f(a, _f64(gamma)) - f(b, _f64(gamma))) / 2e-5
        assert abs(_f64(dx)[i] - num) <= 1e-4 * np.abs(_f64(dx)).max()
    for j in range(16):
        a, b = _f64(gamma), _f64(gamma)
        a[j] += 1e-5
        b[j] -= 1e-5
        num = (f(ho, a) - f(ho, b)) / 2e-5
        assert abs(_f64(dg)[j] - num) <= 1e-4 * np.abs(_f64(dg)).max()


def test_backward_in_place_and_repeatable():
    for N, d in ((900, 512), (700, 4096)):
        h, dh, gamma = _data(N, d, BF, BF, BF, seed=13)
        dy = torch.randn(N, d, device="cuda").to(BF)
        dx, dg = _grad(dy, h, gamma, dh)
        dx2, dg2 = _grad(dy, h, gamma, dh)
        assert torch.equal(dx, dx2) and torch.equal(dg, dg2)
        acc, dg3 = dh.clone(), torch.empty_like(dg)
        ws = torch.empty(K.kdkl_rmsnorm_workspace_bytes(N, d), dtype=torch.uint8, device="cuda")
        K.kdkl_rmsnorm_backward(dy, h, gamma, acc, dg3, ws, dh=acc, eps=EPS)
        assert torch.equal(acc, dx) and torch.equal(dg3, dg)


def test_offsets_past_32_bits():
    """More than 2^31 elements: the last rows land where they belong (all others are zero)."""
    N, d, last = 262300, 8192, 40
    free, _ = torch.cuda.mem_get_info()
    assert N * d > 2 ** 31 and free > 24 << 30
    h, dh, gamma = _data(last, d, BF, BF, BF, seed=15)
    dy = torch.randn(last, d, device="cuda").to(BF)
    big = [torch.zeros(N, d, dtype=BF, device="cuda") for _ in range(3)]
    big[0][-last:], big[1][-last:] = h, dy
    K.kdkl_rmsnorm_forward(big[0], gamma, big[2], eps=EPS)
    _, want, _ = _forward(h, None, gamma, BF, with_h=False)
    assert torch.equal(big[2][-last:], want) and not bool(big[2][:-last].any())
    dg = torch.empty(d, device="cuda")
    ws = torch.empty(K.kdkl_rmsnorm_workspace_bytes(N, d), dtype=torch.uint8, device="cuda")
    K.kdkl_rmsnorm_backward(big[1], big[0], gamma, big[2], dg, ws, eps=EPS)
    dx, dgw = _grad(dy, h, gamma, None)
    assert torch.equal(big[2][-last:], dx) and not bool(big[2][:-last].any())
    scale = (dy.float().abs() * h.float().abs()).sum(0) / h.float().square().mean(1).sqrt().min()
    assert bool(((dg - dgw).abs() <= 256 * U * scale).all())      # the same terms in another order


def test_empty_batch():
    e = torch.empty(0, 64, dtype=BF, device="cuda")
    gamma = torch.ones(64, dtype=BF, device="cuda")
    dg = torch.full((64,), 3.0, device="cuda")
    ws = torch.empty(K.kdkl_rmsnorm_workspace_bytes(0, 64), dtype=torch.uint8, device="cuda")
    buf = torch.full((1, 64), 5.0, dtype=BF, device="cuda")
    lib = K.lib()
    s = torch.cuda.current_stream().cuda_stream
    assert lib.kdkl_rmsnorm_forward(buf.data_ptr(), None, gamma.data_ptr(), 0, 64, EPS, 0, 0, 0, 0, None,
                                    buf.data_ptr(), None, s) == 0
    assert lib.kdkl_rmsnorm_backward(buf.data_ptr(), buf.data_ptr(), gamma.data_ptr(), None, 0, 64, EPS, 0, 0,
                                     buf.data_ptr(), dg.data_ptr(), ws.data_ptr(), ws.numel(), s) == 0
    torch.cuda.synchronize()
    assert bool((buf == 5).all()) and bool((dg == 0).all())
    # empty tensors, which torch gives no address, through the binding
    dg.fill_(3)
    K.kdkl_rmsnorm_forward(e, gamma, e, residual=e, h=e)
    K.kdkl_rmsnorm_forward(e, gamma, e.to(F8), y_scale=torch.empty(0, device="cuda"))
    K.kdkl_rmsnorm_backward(e, e, gamma, e, dg, ws, dh=e)
    torch.cuda.synchronize()
    assert bool((dg == 0).all())


def test_binding_refusals():
    x, r, gamma = _data(10, 64, BF, BF, BF, seed=14)
    y = torch.empty_like(x)

    def refused(match, **kw):
        a = dict(x=x, gamma=gamma, y=y, residual=r)
        a.update(kw)
        with pytest.raises(K.KDKLError, match=match):
            K.kdkl_rmsnorm_forward(a["x"], a["gamma"], a["y"], residual=a["residual"], h=a.get("h"),
                                   y_scale=a.get("y_scale"))
    refused("residual has shape", residual=r[:9])
    refused("gamma has shape", gamma=gamma[:63])
    refused("dense", x=torch.empty(10, 128, dtype=BF, device="cuda")[:, ::2])
    refused("h is torch.float32", h=torch.empty(10, 64, device="cuda"))
    refused("x is torch.float16", x=x.half())
    refused("residual is on cpu", residual=r.cpu())
    refused("y_scale goes with", y=y.to(F8))
    refused("y_scale goes with", y_scale=torch.empty(10, device="cuda"))
    with pytest.raises(K.KDKLError, match="KDKL_ERR_ALIGN"):
        odd = torch.empty(10 * 64 + 1, dtype=BF, device="cuda")[1:].view(10, 64)
        K.kdkl_rmsnorm_forward(odd, gamma, y)
    dg = torch.empty(64, device="cuda")
    with pytest.raises(K.KDKLError, match="KDKL_ERR_WORKSPACE"):
        K.kdkl_rmsnorm_backward(y, x, gamma, y, dg, torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(K.KDKLError, match="dx is torch.float32"):
        K.kdkl_rmsnorm_backward(y, x, gamma, x.float(), dg, torch.empty(1 << 20, dtype=torch.uint8, device="cuda"))
