"""Host-side checks of the operators ahead of the head: workspace sizes, plans and refusals.  Every bad
argument is caught before the device is touched, so no call here reaches a kernel."""
import ctypes

import pytest
import torch

import output_head_kl_b200 as K

NULL, SHAPE, ALIGN, UNSUPPORTED, WORKSPACE = 1, 2, 3, 4, 5


@pytest.fixture(scope="module")
def lib():
    from output_head_kl_b200 import build
    build.build()
    return K.lib()


def _norm(lib, **kw):
    a = dict(x=0x10000, residual=0x20000, gamma=0x30000, N=100, d=256, eps=1e-6, xt=K.BF16, ht=K.BF16, gt=K.BF16,
             yt=K.BF16, h=0x40000, y=0x50000, scale=None)
    a.update(kw)
    return lib.kdkl_rmsnorm_forward(a["x"], a["residual"], a["gamma"], a["N"], a["d"], a["eps"], a["xt"], a["ht"],
                                    a["gt"], a["yt"], a["h"], a["y"], a["scale"], None)


def test_rmsnorm_forward_refusals(lib):
    for name in ("x", "gamma", "y"):
        assert _norm(lib, **{name: None}) == NULL
    assert _norm(lib, yt=K.E4M3) == NULL and _norm(lib, scale=0x60000) == NULL
    assert _norm(lib, d=12) == SHAPE and _norm(lib, d=0) == SHAPE and _norm(lib, N=-1) == SHAPE
    assert _norm(lib, eps=-1.0) == SHAPE and _norm(lib, eps=float("nan")) == SHAPE
    assert _norm(lib, eps=float("inf")) == SHAPE
    assert _norm(lib, d=32776) == UNSUPPORTED and "32768" in K.kdkl_last_error()
    assert _norm(lib, xt=K.E4M3) == UNSUPPORTED and _norm(lib, ht=7) == UNSUPPORTED
    assert _norm(lib, gt=-1) == UNSUPPORTED and _norm(lib, yt=K.F32) == UNSUPPORTED
    for name in ("x", "residual", "gamma", "h", "y"):
        assert _norm(lib, **{name: 0x70008}) == ALIGN
    assert _norm(lib, yt=K.E4M3, scale=0x60002) == ALIGN


def test_rmsnorm_backward_refusals(lib):
    need = K.kdkl_rmsnorm_workspace_bytes(100, 256)
    assert need > 0 and K.kdkl_rmsnorm_workspace_bytes(100, 12) == 0
    assert K.kdkl_rmsnorm_workspace_bytes(0, 256) > 0
    # bounded: the partial sums do not grow with N
    assert K.kdkl_rmsnorm_workspace_bytes(1 << 20, 4096) == K.kdkl_rmsnorm_workspace_bytes(1 << 24, 4096)

    def bwd(**kw):
        a = dict(dy=0x10000, h=0x20000, gamma=0x30000, dh=0x40000, N=100, d=256, eps=1e-6, ht=K.BF16, gt=K.F32,
                 dx=0x50000, dgamma=0x60000, ws=0x70000, wsb=need)
        a.update(kw)
        return lib.kdkl_rmsnorm_backward(a["dy"], a["h"], a["gamma"], a["dh"], a["N"], a["d"], a["eps"], a["ht"],
                                         a["gt"], a["dx"], a["dgamma"], a["ws"], a["wsb"], None)
    for name in ("dy", "h", "gamma", "dx", "dgamma", "ws"):
        assert bwd(**{name: None}) == NULL
    for name in ("dy", "h", "gamma", "dh", "dx"):
        assert bwd(**{name: 0x80004}) == ALIGN
    assert bwd(dgamma=0x80002) == ALIGN and bwd(ws=0x80010) == ALIGN
    assert bwd(d=20) == SHAPE and bwd(ht=K.E4M3) == UNSUPPORTED
    assert bwd(wsb=need - 1) == WORKSPACE and "workspace" in K.kdkl_last_error()


def _fwd(lib, opt=None, **kw):
    a = dict(x=0x10000, W=0x20000, bias=0x30000, residual=0x40000, M=100, d_in=256, d_out=128, y=0x50000,
             pre=0x60000, ws=0x70000, wsb=1 << 40)
    a.update(kw)
    o = K.LinearOptions(**opt) if opt is not None else None
    return lib.kdkl_linear_forward(a["x"], a["W"], a["bias"], a["residual"], a["M"], a["d_in"], a["d_out"],
                                   ctypes.byref(o) if o is not None else None, a["y"], a["pre"], a["ws"], a["wsb"],
                                   None)


def test_linear_forward_refusals(lib):
    for name in ("x", "W", "y", "ws"):
        assert _fwd(lib, **{name: None}) == NULL
    assert _fwd(lib, M=-1) == SHAPE and _fwd(lib, d_in=12) == SHAPE and _fwd(lib, d_out=12) == SHAPE
    assert _fwd(lib, d_in=0) == SHAPE and _fwd(lib, d_out=0) == SHAPE
    assert _fwd(lib, d_out=(1 << 20) + 8) == UNSUPPORTED
    for name in ("x", "W", "bias", "residual", "y", "pre"):
        assert _fwd(lib, **{name: 0x80008}) == ALIGN
    assert _fwd(lib, ws=0x80010) == ALIGN and _fwd(lib, wsb=K.kdkl_linear_workspace_bytes(100, 256, 128) - 1) == WORKSPACE
    assert _fwd(lib, opt=dict(activation=5)) == UNSUPPORTED and _fwd(lib, opt=dict(activation=-1)) == UNSUPPORTED
    assert _fwd(lib, opt=dict(operands=K.F32)) == UNSUPPORTED
    f8 = dict(operands=K.E4M3, x_scale=0x90000, w_scale=0xA0000)
    assert _fwd(lib, opt=dict(f8, x_scale=None)) == NULL and _fwd(lib, opt=dict(f8, w_scale=None)) == NULL
    assert _fwd(lib, opt=dict(f8, w_scale=0xA0004)) == ALIGN and _fwd(lib, opt=dict(f8, x_scale=0x90002)) == ALIGN
    assert _fwd(lib, opt=f8, d_in=264) == SHAPE                       # e4m3 rows are multiples of 16
    assert _fwd(lib, opt=dict(x_scale=0x90000)) == UNSUPPORTED       # scales without e4m3 operands
    # the most rows a call may have, times too many columns: tiles are counted in 32 bits
    assert _fwd(lib, M=(1 << 31) - 256, d_out=1 << 20, d_in=8) == UNSUPPORTED
    assert _fwd(lib, M=(1 << 31) - 255) == SHAPE


def test_linear_backward_refusals(lib):
    need = K.kdkl_linear_workspace_bytes(100, 256, 128, True)
    assert need >= 100 * 128 * 2 and K.kdkl_linear_workspace_bytes(100, 12, 128) == 0

    def bwd(opt=None, **kw):
        a = dict(dy=0x10000, pre=0x20000, x=0x30000, W=0x40000, M=100, d_in=256, d_out=128, dx=0x50000, dW=0x60000,
                 dbias=0x70000, ws=0x80000, wsb=need)
        a.update(kw)
        o = K.LinearOptions(**(opt or {}))
        return lib.kdkl_linear_backward(a["dy"], a["pre"], a["x"], a["W"], a["M"], a["d_in"], a["d_out"],
                                        ctypes.byref(o), a["dx"], a["dW"], a["dbias"], a["ws"], a["wsb"], None)
    assert bwd(dx=None, dW=None, dbias=None) == NULL
    assert bwd(dy=None) == NULL and bwd(ws=None) == NULL and bwd(x=None) == NULL and bwd(W=None) == NULL
    assert bwd(opt=dict(activation=K.ACT_GELU), pre=None) == NULL
    assert bwd(opt=dict(operands=K.E4M3)) == UNSUPPORTED and bwd(opt=dict(activation=9)) == UNSUPPORTED
    for name in ("dy", "pre", "x", "W", "dx", "dW"):
        assert bwd(**{name: 0x90008}) == ALIGN
    assert bwd(dbias=0x90002) == ALIGN and bwd(ws=0x90010) == ALIGN
    assert bwd(wsb=need - 1) == WORKSPACE and bwd(d_out=100) == SHAPE


def test_linear_plans(lib):
    def plan(*a, **kw):
        return K.kdkl_linear_plan(*a, sm_count=148, **kw)
    # half the last wave's pairs idle: its tiles are split
    assert plan(1 << 14, 4096, 4096, product=K.LINEAR_DW) == 20256
    # few rows: small tiles, the reduction split; many rows: full 256 x 256 tiles
    assert plan(1, 4096, 4096) > 1000 and plan(1, 4096, 4096) % 1000 == 16
    assert plan(32768, 4096, 4096) == 256
    assert plan(1, 4096, 4096, product=K.LINEAR_DX) > 1000
    for M in (0, 1, 2, 17, 100, 255, 256, 257, 1000, 5000, 1 << 20):
        for d_in, d_out in ((16, 8), (64, 4096), (4096, 64), (2048, 2880), (4096, 4096), (1 << 20, 1 << 20)):
            for ops, prod in ((K.BF16, 0), (K.E4M3, 0), (K.BF16, 1), (K.BF16, 2)):
                p = plan(M, d_in, d_out, operands=ops, product=prod)
                if p % 10000 in (128, 192, 256):
                    # the last wave's tiles split 2 to 8 ways, each share of 4 reduction blocks at least
                    rows, cols, length = ((M, d_out, d_in), (M, d_in, d_out), (d_out, d_in, M))[prod]
                    tail = -(-rows // 256) * -(-cols // (p % 10000)) % 74
                    blocks = -(-length // (128 if ops == K.E4M3 else 64))
                    sp = p // 10000
                    full = -(-rows // 256) * -(-cols // (p % 10000)) >= 74
                    assert sp == 0 or 2 <= sp <= min(8, 74 // tail, blocks // 4)
                    assert sp in (0, 2, 4) or full or prod == 2
                else:
                    length = d_out if prod == 1 else d_in
                    assert prod != 2 and p % 1000 in (16, 32, 64, 128) and p // 1000 in (1, 2, 4, 8)
                    assert p // 1000 <= -(-length // (128 if ops == K.E4M3 else 64))
    out = ctypes.c_int32()
    assert lib.kdkl_linear_plan(1, 64, 64, 0, 0, 148, None) == NULL
    assert lib.kdkl_linear_plan(1, 60, 64, 0, 0, 148, ctypes.byref(out)) == SHAPE
    assert lib.kdkl_linear_plan(1, 64, 64, 0, 3, 148, ctypes.byref(out)) == UNSUPPORTED
    assert lib.kdkl_linear_plan(1, 64, 64, K.E4M3, 1, 148, ctypes.byref(out)) == UNSUPPORTED
    assert lib.kdkl_linear_plan(1, 64, 64, 0, 0, 1, ctypes.byref(out)) == SHAPE


def test_binding_refuses_tensors_off_the_device():
    """The Python binding checks tensors before it asks the library: a CPU tensor is refused by name."""
    x = torch.zeros(4, 16, dtype=torch.bfloat16)
    with pytest.raises(K.KDKLError, match="x is on cpu"):
        K.kdkl_rmsnorm_forward(x, x[0], x)
    with pytest.raises(K.KDKLError, match="x is on cpu"):
        K.kdkl_linear_forward(x, x, x, x)
    with pytest.raises(K.KDKLError, match="dy is on cpu"):
        K.kdkl_linear_backward(x, x, x, x, x, x)
    with pytest.raises(K.KDKLError, match="3 dimensions"):
        K.kdkl_rmsnorm_forward(x[None], x[0], x)


def test_binding_missing_fails_loudly(monkeypatch, tmp_path):
    monkeypatch.setattr(K, "_binding", None)
    monkeypatch.setattr(K, "BINDING_PATH", str(tmp_path / "nope.so"))
    x = torch.zeros(4, 16, dtype=torch.bfloat16)
    with pytest.raises(RuntimeError, match="not built"):
        K.kdkl_rmsnorm_forward(x, x[0], x)


def test_compiled_marshalling_declines_what_it_does_not_take():
    """None (and no crash) for arguments that are no tensors, off the device, or of the wrong kind; the Python
    path then raises, naming the argument."""
    b, x = K._fast(), torch.zeros(4, 16, dtype=torch.bfloat16)
    for bad in (x, None, 3, "x", torch.zeros(4, 16).to_sparse(), object()):
        assert b.rmsnorm_forward(0, bad, x[0], x, None, None, None, 1e-6, None) is None
        assert b.rmsnorm_backward(0, bad, bad, x[0], x, x[0], x, None, 1e-6, None) is None
        assert b.linear_forward(0, bad, x, x, x, None, None, None, 0, None, None, 0, None) is None
        assert b.linear_backward(0, bad, x, x, x, x, x, None, None, 0, 0, 0, None) is None
    with pytest.raises(TypeError):
        b.linear_forward(0, x)
    assert ctypes.cast(K.lib().kdkl_linear_forward, ctypes.c_void_p).value == K.lib().kdkl_addr["linear_forward"]
