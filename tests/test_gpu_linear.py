"""Linear layer (bias, activation, residual; bf16 and e4m3 operands) and its gradient on the GPU vs the
float64 oracle, through every kind of tile.

Tolerances (U = 2^-24, half an fp32 step).  A product of len terms is summed in fp32 in an order of the
tensor core's choosing, with at most one step (2 U, allowing for truncation) of the partial sums' magnitude
per addition, bounded by 2 len U S with S = sum |x w|.  The activations have slopes of at most 1.13 in
magnitude, and their own error (hardware exponential and reciprocal, 2 ulp each, argument rounding
|z| U) is below |z| (|z| + 16) 2 U.  A bf16 output adds 2^-8 of its value.
"""
import ctypes

import numpy as np
import pytest
import torch

import output_head_kl_b200 as K
from oracle import layers as L

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
TINY = 2.0 ** -133
PAIR_PLANS = (128, 192, 256)
SMALL_PLANS = tuple(1000 * s + n for s in (1, 2, 4, 8) for n in (16, 32, 64, 128))


def _f64(t):
    return None if t is None else t.double().cpu().numpy()


def _e4m3_rows(t):
    s = t.abs().amax(dim=1) / 448.0
    return (t / s[:, None]).to(F8), s


def _data(M, d_in, d_out, f8=False, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + M * 31 + d_in + d_out)

    def rn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")
    x, W = rn(M, d_in), rn(d_out, d_in) * d_in ** -0.5
    o = dict(bias=rn(d_out).to(BF), residual=rn(M, d_out).to(BF), x_scale=None, w_scale=None)
    if f8:
        o["x"], o["x_scale"] = _e4m3_rows(x)
        o["W"], o["w_scale"] = _e4m3_rows(W)
    else:
        o["x"], o["W"] = x.to(BF), W.to(BF)
    return o


def _call(o, act="none", bias=True, residual=True, pre=False, plan=0):
    M, d_out = o["x"].shape[0], o["W"].shape[0]
    # one row more than asked for, to see that it is left as it was
    y = torch.full((M + 1, d_out), 9.0, dtype=BF, device="cuda")
    p = torch.full((M + 1, d_out), 9.0, dtype=BF, device="cuda") if pre else None
    ws = torch.full((K.kdkl_linear_workspace_bytes(M, o["x"].shape[1], d_out),), 255, dtype=torch.uint8, device="cuda")
    K.kdkl_linear_forward(o["x"], o["W"], y[:M], ws, bias=o["bias"] if bias else None,
                          residual=o["residual"] if residual else None, pre=p[:M] if pre else None, activation=act,
                          x_scale=o["x_scale"], w_scale=o["w_scale"], plan=plan)
    assert K.kdkl_read_device_flags(ws) == 0
    assert bool((y[M] == 9).all()) and (p is None or bool((p[M] == 9).all()))
    return y[:M], (p[:M] if pre else None)


def _check(o, act="none", bias=True, residual=True, pre=False, plan=0, rows=None):
    y, p = _call(o, act, bias, residual, pre, plan)
    sel = slice(None) if rows is None else rows
    x, W = _f64(o["x"][sel]), _f64(o["W"])
    if o["x_scale"] is not None:
        x, W = x * _f64(o["x_scale"])[sel, None], W * _f64(o["w_scale"])[:, None]
    b, r = (_f64(o["bias"]) if bias else None), (_f64(o["residual"][sel]) if residual else None)
    yo, zo = L.linear(x, W, b, r, act)
    S = np.abs(x) @ np.abs(W).T + (np.abs(b) if bias else 0)
    dz = (2 * x.shape[1] + 8) * U * S
    if pre:
        assert np.all(np.abs(_f64(p[sel]) - zo) <= dz + 2.0 ** -8 * np.abs(zo) + TINY)
    own = 2 * U * np.abs(zo) * (np.abs(zo) + 16) if act not in ("none", "relu") else 0
    tol = 1.13 * dz + own + 2.0 ** -8 * np.abs(yo) + 2 * U * (np.abs(yo) + np.abs(zo)) + TINY
    err = np.abs(_f64(y[sel]) - yo)
    assert np.all(err <= tol), f"max err {err.max():.3e} at {np.unravel_index(err.argmax(), err.shape)}"


@pytest.mark.parametrize("f8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("M,d_in,d_out", [(1, 16, 8), (1, 4096, 4096), (2, 64, 128), (7, 80, 136), (16, 2048, 264),
                                          (17, 208, 120), (77, 2048, 2880), (128, 512, 512), (200, 1024, 392),
                                          (257, 144, 520), (700, 2880, 896), (1500, 272, 1032)])
def test_forward(M, d_in, d_out, f8):
    _check(_data(M, d_in, d_out, f8), act="silu", pre=True)


@pytest.mark.parametrize("f8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("act", L.ACTIVATIONS)
@pytest.mark.parametrize("M", [9, 300])
def test_activations(act, M, f8):
    o = _data(M, 256, 328, f8, seed=1)
    _check(o, act, bias=True, residual=True, pre=True)
    _check(o, act, bias=False, residual=False)
    _check(o, act, bias=False, residual=True)
    _check(o, act, bias=True, residual=False, pre=True)


@pytest.mark.parametrize("f8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("plan", PAIR_PLANS + SMALL_PLANS)
def test_every_plan(plan, f8):
    """Ragged in rows, columns and reduction, with more tiles than one per CTA pair for the large ones."""
    d_in = 1040 if f8 else 536          # 9 reduction blocks, the last one partly filled
    o = _data(300, d_in, 712, f8, seed=2)
    _check(o, "gelu", pre=True, plan=plan)
    _check(_data(1, d_in, 8, f8, seed=3), "none", plan=plan)


def test_many_tiles_per_pair():
    """More output tiles than CTA pairs, so that accumulators, stages and staging buffers turn over."""
    o = _data(5000, 192, 2088, seed=4)
    for plan in PAIR_PLANS:
        _check(o, "gelu_tanh", pre=True, plan=plan, rows=slice(4700, 5000))
    y0, p0 = _call(o, "silu", pre=True, plan=256)
    y1, p1 = _call(o, "silu", pre=True, plan=128)
    assert torch.equal(p0, p1) and torch.equal(y0, y1)   # each output is one fp32 reduction in the same order


@pytest.mark.parametrize("f8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("plan", [20128, 20192, 20256, 40128, 40192, 40256])
def test_split_last_wave(plan, f8):
    """Tiles whose reduction is shared by a cluster of CTA pairs and joined over their shared memory."""
    o = _data(300, 4112 if f8 else 2088, 712, f8, seed=10)    # 33 reduction blocks, the last partly filled
    _check(o, "silu", pre=True, plan=plan)
    _check(o, "none", bias=False, residual=False, plan=plan)
    a, pa = _call(o, "gelu", pre=True, plan=plan)
    for _ in range(3):                                         # whichever share arrives last, the same bits
        b, pb = _call(o, "gelu", pre=True, plan=plan)
        assert torch.equal(a, b) and torch.equal(pa, pb)


def test_split_last_wave_after_full_waves():
    """180 tiles: two full waves of 74 pairs and 32 tiles in two shares each."""
    o = _data(5000, 576, 2088, seed=11)
    _check(o, "gelu_tanh", pre=True, plan=20256, rows=slice(0, 300))
    _check(o, "gelu_tanh", pre=True, plan=20256, rows=slice(4700, 5000))
    a, _ = _call(o, "silu", plan=20256)
    b, _ = _call(o, "silu", plan=256)
    assert (a.float() - b.float()).abs().max().item() <= 2.0 ** -6 * b.float().abs().max().item()


def test_splits_leave_rounding_only():
    """Splitting the reduction changes the order of one fp32 sum: results stay within its bound, and repeat."""
    o = _data(40, 2048, 512, seed=5)
    for plan in (1064, 2064, 4064, 8064):
        _check(o, "none", pre=True, plan=plan)
        a, _ = _call(o, "none", plan=plan)
        b, _ = _call(o, "none", plan=plan)
        assert torch.equal(a, b)


@pytest.mark.parametrize("M", [5, 400])
def test_extreme_preactivations(M):
    """|z| far beyond the exponentials' range: the activations saturate instead of overflowing."""
    o = _data(M, 64, 128, seed=6)
    o["x"] = (o["x"].float() * 1000).to(BF)
    for act in ("gelu", "gelu_tanh", "silu", "relu"):
        y, p = _call(o, act, residual=False, pre=True)
        z = _f64(p)
        yv = _f64(y)
        assert np.all(np.isfinite(yv))
        big = z > 100
        assert big.any() and np.all(np.abs(yv[big] - z[big]) <= 2.0 ** -7 * z[big])
        assert np.all(np.abs(yv[z < -150]) == 0)


@pytest.mark.parametrize("M", [6, 300])
def test_nonfinite_rows_stay_in_their_rows(M):
    o = _data(M, 128, 136, seed=7)
    clean, _ = _call(o, "silu")
    o["x"][2, 5] = float("nan")
    o["x"][4, 7] = float("inf")
    y, _ = _call(o, "silu")
    assert bool(torch.isnan(y[2]).all()) and not bool(torch.isfinite(y[4]).all())
    keep = [n for n in range(M) if n not in (2, 4)]
    assert torch.equal(y[keep], clean[keep])


@pytest.mark.parametrize("M", [5, 300])
def test_residual_in_place(M):
    o = _data(M, 256, 264, seed=8)
    ws = torch.empty(K.kdkl_linear_workspace_bytes(M, 256, 264), dtype=torch.uint8, device="cuda")
    for plan in (0, 256, 4032):
        y = o["residual"].clone()
        want, _ = _call(o, "gelu", plan=plan)
        K.kdkl_linear_forward(o["x"], o["W"], y, ws, bias=o["bias"], residual=y, activation="gelu", plan=plan)
        assert torch.equal(y, want)


def test_offsets_past_32_bits():
    """More than 2^31 output elements: the last rows of a tall product land where they belong."""
    M, d_in, d_out = 262400, 16, 8192
    free, _ = torch.cuda.mem_get_info()
    assert M * d_out > 2 ** 31 and free > 12 << 30
    g = torch.Generator(device="cuda").manual_seed(9)
    x = torch.randn(M, d_in, generator=g, device="cuda").to(BF)
    W = (torch.randn(d_out, d_in, generator=g, device="cuda") / 4).to(BF)
    y = torch.empty(M, d_out, dtype=BF, device="cuda")
    y[-300:].fill_(9)
    ws = torch.empty(K.kdkl_linear_workspace_bytes(M, d_in, d_out), dtype=torch.uint8, device="cuda")
    K.kdkl_linear_forward(x, W, y, ws, residual=y, activation="none")     # residual read at the same offsets
    want = _f64(x[-300:]) @ _f64(W).T + 9
    S = np.abs(_f64(x[-300:])) @ np.abs(_f64(W)).T + 9
    assert np.all(np.abs(_f64(y[-300:]) - want) <= 2.0 ** -8 * np.abs(want) + 48 * U * S)


# ------------------------------------------------------------------ gradient
def _grad_data(M, d_in, d_out, seed=0):
    o = _data(M, d_in, d_out, seed=seed)
    g = torch.Generator(device="cuda").manual_seed(seed + 77)
    dy = torch.randn(M, d_out, generator=g, device="cuda").to(BF)
    pre = (2 * torch.randn(M, d_out, generator=g, device="cuda")).to(BF)
    return dy, pre, o["x"], o["W"]


def _grad(dy, pre, x, W, act, dx_plan=0, dw_plan=0, want=("dx", "dW", "dbias")):
    M, d_out = dy.shape
    d_in = x.shape[1]
    nan = float("nan")
    dx = torch.full((M, d_in), nan, dtype=BF, device="cuda") if "dx" in want else None
    dW = torch.full((d_out, d_in), nan, dtype=BF, device="cuda") if "dW" in want else None
    db = torch.full((d_out,), nan, device="cuda") if "dbias" in want else None
    ws = torch.full((K.kdkl_linear_workspace_bytes(M, d_in, d_out, True),), 255, dtype=torch.uint8, device="cuda")
    K.kdkl_linear_backward(dy, x if dW is not None else None, W, dx, dW, ws, pre=pre, dbias=db, activation=act,
                           dx_plan=dx_plan, dw_plan=dw_plan)
    assert K.kdkl_read_device_flags(ws) == 0
    return dx, dW, db


def _check_grad(dy, pre, x, W, act, **kw):
    dx, dW, db = _grad(dy, pre, x, W, act, **kw)
    dyo, zo, xo, Wo = _f64(dy), _f64(pre), _f64(x), _f64(W)
    dxo, dWo, dbo, dz = L.linear_grad(dyo, zo if act != "none" else None, xo, Wo, act)
    # dz is rounded once to bf16 (not at all without an activation); the slopes' own error as the activations'
    own = np.abs(dyo) * (np.abs(zo) + 16) * 4 * U if act not in ("none", "relu") else np.zeros_like(dz)
    ez = own + (2.0 ** -8 * np.abs(dz) + TINY if act != "none" else 0)
    for got, ref, e, S, n in ((dx, dxo, ez @ np.abs(Wo), np.abs(dz) @ np.abs(Wo), dz.shape[1]),
                              (dW, dWo, ez.T @ np.abs(xo), np.abs(dz).T @ np.abs(xo), dz.shape[0])):
        if got is not None:
            err = np.abs(_f64(got) - ref)
            assert np.all(err <= e + (2 * n + 8) * U * S + 2.0 ** -8 * (np.abs(ref) + e) + TINY), err.max()
            # the bound above allows every rounding of dz the same sign; they are independent, so the
            # error's 2-norm stays near one bf16 rounding of the result
            if act != "none":
                assert np.linalg.norm(err) <= 2.0 ** -7 * np.linalg.norm(ref) + 1e-30
    if db is not None:
        tol = own.sum(axis=0) + (dz.shape[0] + 64) * U * np.abs(dz).sum(axis=0) + 1e-30
        assert np.all(np.abs(_f64(db) - dbo) <= tol)


@pytest.mark.parametrize("act", L.ACTIVATIONS)
@pytest.mark.parametrize("M,d_in,d_out", [(1, 8, 8), (3, 72, 136), (100, 200, 264), (1003, 456, 328)])
def test_backward(M, d_in, d_out, act):
    _check_grad(*_grad_data(M, d_in, d_out), act)


@pytest.mark.parametrize("M,d_in,d_out", [(1, 2048, 2880), (77, 2880, 1024), (1500, 1032, 520), (2050, 64, 72)])
def test_backward_shapes(M, d_in, d_out):
    _check_grad(*_grad_data(M, d_in, d_out, seed=1), "gelu")


@pytest.mark.parametrize("dx_plan", PAIR_PLANS + SMALL_PLANS)
def test_every_dx_plan(dx_plan):
    _check_grad(*_grad_data(300, 712, 536, seed=2), "silu", dx_plan=dx_plan, want=("dx",))
    _check_grad(*_grad_data(1, 8, 520, seed=3), "none", dx_plan=dx_plan, want=("dx",))


def test_split_gradient_products():
    dy, pre, x, W = _grad_data(2100, 712, 1096, seed=9)
    for dx_plan, dw_plan in ((20256, 20256), (40192, 30192), (20128, 20128), (40256, 20256)):
        _check_grad(dy[:300], pre[:300], x[:300], W, "silu", dx_plan=dx_plan, want=("dx",))
        _check_grad(dy, pre, x, W, "silu", dw_plan=dw_plan, want=("dW",))
    both = _grad(dy, pre, x, W, "gelu", dx_plan=20256, dw_plan=40256)
    for _ in range(2):
        again = _grad(dy, pre, x, W, "gelu", dx_plan=20256, dw_plan=40256)
        assert all(torch.equal(a, b) for a, b in zip(both, again))


@pytest.mark.parametrize("dw_plan", PAIR_PLANS)
def test_every_dw_plan(dw_plan):
    _check_grad(*_grad_data(300, 712, 536, seed=4), "silu", dw_plan=dw_plan, want=("dW",))
    dy, pre, x, W = _grad_data(257, 2088, 5000, seed=5)
    a = _grad(dy, pre, x, W, "relu", dw_plan=dw_plan, want=("dW",))[1]
    b = _grad(dy, pre, x, W, "relu", dw_plan=256, want=("dW",))[1]
    assert torch.equal(a, b)


def test_backward_outputs_one_by_one():
    args = _grad_data(130, 200, 264, seed=6)
    full = _grad(*args, "gelu_tanh")
    for i, name in enumerate(("dx", "dW", "dbias")):
        one = _grad(*args, "gelu_tanh", want=(name,))
        assert torch.equal(one[i], full[i])
    plain = _grad(*args, "none", want=("dbias",))
    np.testing.assert_allclose(_f64(plain[2]), _f64(args[0]).sum(axis=0), atol=1e-4)


def test_relu_gradient_is_zero_at_zero():
    dy = torch.ones(4, 8, dtype=BF, device="cuda")
    pre = torch.tensor([[-1.0, -0.0, 0.0, 1e-30, 1.0, 2.0, -2.0, float("nan")]] * 4, dtype=BF, device="cuda")
    db = torch.empty(8, device="cuda")
    ws = torch.empty(K.kdkl_linear_workspace_bytes(4, 8, 8, True), dtype=torch.uint8, device="cuda")
    K.kdkl_linear_backward(dy, None, None, None, None, ws, pre=pre, dbias=db, activation="relu")
    assert db[:7].tolist() == [0, 0, 0, 4, 4, 4, 0] and bool(torch.isnan(db[7]))


def test_empty_batch():
    """M = 0 leaves the outputs alone, or zeroes the sums over rows."""
    buf = torch.full((1, 64), 5.0, dtype=BF, device="cuda")
    W = torch.ones(64, 64, dtype=BF, device="cuda")
    dW = torch.full((64, 64), 5.0, dtype=BF, device="cuda")
    db = torch.full((64,), 5.0, device="cuda")
    ws = torch.full((K.kdkl_linear_workspace_bytes(0, 64, 64, True),), 255, dtype=torch.uint8, device="cuda")
    lib, s = K.lib(), torch.cuda.current_stream().cuda_stream
    b, w = buf.data_ptr(), W.data_ptr()
    assert lib.kdkl_linear_forward(b, w, None, None, 0, 64, 64, None, b, None, ws.data_ptr(), ws.numel(), s) == 0
    assert K.kdkl_read_device_flags(ws) == 0 and bool((buf == 5).all())
    assert lib.kdkl_linear_backward(b, None, b, w, 0, 64, 64, None, b, dW.data_ptr(), db.data_ptr(), ws.data_ptr(),
                                    ws.numel(), s) == 0
    torch.cuda.synchronize()
    assert bool((buf == 5).all()) and bool((dW == 0).all()) and bool((db == 0).all())
    # empty tensors, which torch gives no address, through the binding
    e, dW[:], db[:] = torch.empty(0, 64, dtype=BF, device="cuda"), 5, 5
    K.kdkl_linear_forward(e, W, e, ws, bias=W[0], residual=e, pre=e, activation="silu")
    K.kdkl_linear_backward(e, e, W, e, dW, ws, pre=e, dbias=db, activation="silu")
    torch.cuda.synchronize()
    assert bool((dW == 0).all()) and bool((db == 0).all())
    e8, s8 = e.to(F8), torch.empty(0, device="cuda")
    K.kdkl_linear_forward(e8, W.to(F8), e, ws, x_scale=s8, w_scale=torch.ones(64, device="cuda"))


def test_binding_refusals():
    o = _data(10, 64, 128)
    y = torch.empty(10, 128, dtype=BF, device="cuda")
    ws = torch.empty(K.kdkl_linear_workspace_bytes(10, 64, 128) + 256, dtype=torch.uint8, device="cuda")

    def refused(match, **kw):
        a = dict(x=o["x"], W=o["W"], y=y, ws=ws)
        a.update(kw)
        with pytest.raises(K.KDKLError, match=match):
            K.kdkl_linear_forward(a["x"], a["W"], a["y"], a["ws"], **{k: v for k, v in a.items()
                                                                      if k not in ("x", "W", "y", "ws")})
    refused("W has shape", W=o["W"][:, :56].contiguous())
    refused("W is torch", W=o["W"].float())
    refused("dense", x=torch.empty(64, 10, dtype=BF, device="cuda").t())
    refused("y has shape", y=y[:9])
    refused("unknown activation", activation="tanh")
    refused("unknown activation", activation=11)
    refused("is no plan", plan=64)
    refused("is no plan", plan=2016)          # d_in = 64 has one reduction block, not two
    refused("is no plan", plan=3016)
    refused("is no plan", plan=1048)
    refused("is no plan", plan=20256)         # one reduction block cannot be split
    refused("is no plan", plan=-256)
    refused("is no plan", plan=90256)
    refused("is no plan", plan=30256)
    refused("need x_scale", x=o["x"].to(F8), W=o["W"].to(F8))
    refused("KDKL_E4M3 operands only", x_scale=torch.ones(10, device="cuda"))
    refused("workspace is on cpu", ws=ws.cpu())
    refused("KDKL_ERR_WORKSPACE", ws=ws[:128])
    refused("KDKL_ERR_ALIGN", ws=ws[8:])
    dW = torch.empty(128, 64, dtype=BF, device="cuda")
    big = torch.empty(1 << 25, dtype=torch.uint8, device="cuda")
    with pytest.raises(K.KDKLError, match="is no plan"):
        K.kdkl_linear_backward(y, o["x"], o["W"], None, dW, big, dw_plan=1016)
    with pytest.raises(K.KDKLError, match="needs pre"):
        K.kdkl_linear_backward(y, o["x"], o["W"], None, dW, big, activation="silu")
    with pytest.raises(K.KDKLError, match="dW is torch.float32"):
        K.kdkl_linear_backward(y, o["x"], o["W"], None, dW.float(), big)
    assert ctypes.sizeof(K.LinearOptions) == 40
