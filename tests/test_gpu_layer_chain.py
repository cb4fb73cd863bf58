"""The operators ahead of the head together, as a training step and a decoding step use them: linear block ->
RMS norm -> fused KL loss and back, RMS norm -> 8-bit linear, in CUDA graphs, on several streams, and through
the bounds-checking build."""
import numpy as np
import pytest
import torch

import output_head_kl_b200 as K
import synth
from oracle import kl as O
from oracle import layers as L
from tests import gpu_harness as H
from tests import test_gpu_linear as TL
from tests import test_gpu_rmsnorm as TN

pytestmark = pytest.mark.gpu

BF, F8 = torch.bfloat16, torch.float8_e4m3fn
EPS = 1e-5


def _f64(t):
    return t.double().cpu().numpy()


def _u8(n):
    return torch.empty(n, dtype=torch.uint8, device="cuda")


class Step:
    """A residual block y = x + silu(x Wb^T + b), h = y + r, hidden = rmsnorm(h), the loss, and all gradients."""

    def __init__(self, N=700, d=256, V=3001, Kc=16, seed=1):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def rn(*s):
            return torch.randn(*s, generator=g, device="cuda")
        self.N, self.d = N, d
        self.x, self.r = rn(N, d).to(BF), rn(N, d).to(BF)
        self.Wb, self.b = (rn(d, d) * d ** -0.5).to(BF), rn(d).to(BF)
        self.gamma = (1 + 0.2 * rn(d)).to(BF)
        self.k = H.to_device(synth.custom_inputs(N, d, V, Kc, seed=seed, mask_frac=0.05, w_std=0.05))
        e = lambda *s, dt=BF: torch.empty(*s, dtype=dt, device="cuda")  # noqa: E731
        f = torch.float32
        self.y, self.pre, self.h, self.hidden = e(N, d), e(N, d), e(N, d), e(N, d)
        self.loss, self.lse = e(1, dt=f), e(N, dt=f)
        self.dhidden, self.dWh, self.dh = e(N, d), e(V, d, dt=f), e(N, d)
        self.dgamma, self.dx, self.dWb, self.db = e(d, dt=f), e(N, d), e(d, d), e(d, dt=f)
        self.ws = _u8(K.kdkl_workspace_bytes(N, d, V, Kc))
        self.ws_n = _u8(K.kdkl_rmsnorm_workspace_bytes(N, d))
        self.ws_l = _u8(K.kdkl_linear_workspace_bytes(N, d, d, backward=True))

    def run(self, stream=None):
        k, s = self.k, stream
        K.kdkl_linear_forward(self.x, self.Wb, self.y, self.ws_l, bias=self.b, residual=self.x, pre=self.pre,
                              activation="silu", stream=s)
        K.kdkl_rmsnorm_forward(self.y, self.gamma, self.hidden, residual=self.r, h=self.h, eps=EPS, stream=s)
        K.kdkl_forward(self.hidden, k.W, k.idx, k.logit, k.mask, k.tau, self.loss, self.lse, self.ws, stream=s)
        K.kdkl_backward(self.hidden, k.W, k.idx, k.logit, k.mask, k.tau, self.lse, None, self.dhidden, self.dWh,
                        self.ws, stream=s)
        K.kdkl_rmsnorm_backward(self.dhidden, self.h, self.gamma, self.dh, self.dgamma, self.ws_n, eps=EPS, stream=s)
        K.kdkl_linear_backward(self.dh, self.x, self.Wb, self.dx, self.dWb, self.ws_l, pre=self.pre, dbias=self.db,
                               activation="silu", stream=s)

    def outputs(self):
        return {n: getattr(self, n) for n in ("y", "pre", "h", "hidden", "loss", "lse", "dhidden", "dWh", "dh",
                                              "dgamma", "dx", "dWb", "db")}

    def snapshot(self):
        torch.cuda.synchronize()
        return {n: t.clone() for n, t in self.outputs().items()}


def test_training_step_matches_the_oracle():
    """Every gradient of the whole step against float64.  Each of the five bf16 tensors on the way back (hidden,
    dHidden, dh, pre, dz) is within 2^-8 of its value element by element, independently, so the gradients' 2-norm
    error stays well below 5 x 2^-8; a wrong term anywhere is of order 1."""
    s = Step()
    s.run()
    torch.cuda.synchronize()
    x, r, Wb, b, gamma = (_f64(t) for t in (s.x, s.r, s.Wb, s.b, s.gamma))
    y, z = L.linear(x, Wb, b, x, "silu")
    h, hidden = L.rmsnorm(y, r, gamma, EPS)
    # the loss oracle reads bf16 hidden states: the exact ones, rounded
    k = s.k
    W = k.W.view(torch.int16).cpu().numpy().view(np.uint16)
    ref = O.kl_loss(synth.f32_to_bf16_bits(hidden.astype(np.float32)), W, k.idx.cpu().numpy(), k.logit.cpu().numpy(),
                    k.mask.cpu().numpy(), k.tau)
    H.assert_loss(s.loss.item(), ref.loss)
    dh, dgamma = L.rmsnorm_grad(ref.dH, h, gamma, EPS)
    dx, dWb, db, _ = L.linear_grad(dh, z, x, Wb, "silu")
    for name, got, want in (("dhidden", s.dhidden, ref.dH), ("dWh", s.dWh, ref.dW), ("dh", s.dh, dh),
                            ("dgamma", s.dgamma, dgamma), ("dx", s.dx, dx), ("dWb", s.dWb, dWb), ("db", s.db, db)):
        rel = np.linalg.norm(_f64(got) - want) / np.linalg.norm(want)
        assert rel <= 5 * 2.0 ** -8, (name, rel)
    masked = k.mask.cpu().numpy() == 0
    assert masked.any() and bool((s.dh[torch.from_numpy(masked).cuda()] == 0).all())


@pytest.mark.parametrize("M", [1, 8, 300])
def test_norm_feeds_the_8bit_product(M):
    """RMS norm to e4m3 rows and scales, straight into the 8-bit linear layer: one decoding step, and a prompt.
    The product is exact up to fp32 summation and the bf16 output for the e4m3 values that the norm wrote; against
    the unquantised chain the rounding of x and W to 3 mantissa bits stays below 2^-4 in 2-norm."""
    g = torch.Generator(device="cuda").manual_seed(M)
    d, n = 1024, 520
    x = torch.randn(M, d, generator=g, device="cuda").to(BF)
    r = torch.randn(M, d, generator=g, device="cuda")
    gamma = (1 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(BF)
    W = torch.randn(n, d, generator=g, device="cuda") * d ** -0.5
    sw = W.abs().amax(1) / 448
    Wq = (W / sw[:, None]).to(F8)
    q = torch.empty(M, d, dtype=F8, device="cuda")
    sx, y = torch.empty(M, device="cuda"), torch.empty(M, n, dtype=BF, device="cuda")
    ws = _u8(K.kdkl_linear_workspace_bytes(M, d, n))
    K.kdkl_rmsnorm_forward(x, gamma, q, residual=r, h=r, y_scale=sx, eps=EPS)   # the fp32 stream, in place
    K.kdkl_linear_forward(q, Wq, y, ws, x_scale=sx, w_scale=sw)
    xq, Wd = _f64(q) * _f64(sx)[:, None], _f64(Wq) * _f64(sw)[:, None]
    want = xq @ Wd.T
    S = np.abs(xq) @ np.abs(Wd).T
    assert np.all(np.abs(_f64(y) - want) <= 2.0 ** -8 * np.abs(want) + 2 * (d + 8) * 2.0 ** -24 * S)
    full = L.rmsnorm(_f64(r), None, _f64(gamma), EPS)[1] @ _f64(W).T
    assert np.linalg.norm(_f64(y) - full) <= 2.0 ** -4 * np.linalg.norm(full)


def test_norm_feeds_the_topk_producer():
    """The norm's bf16 output is a teacher's hidden state: its top-K equals the top-K of the same bits uploaded."""
    s = Step(N=300, d=192, V=4000, seed=3)
    s.run()
    idx = [torch.empty(300, 32, dtype=torch.int32, device="cuda") for _ in range(2)]
    val = [torch.empty(300, 32, device="cuda") for _ in range(2)]
    ws = _u8(K.kdkl_teacher_topk_workspace_bytes(300, 192, 4000, 32))
    K.kdkl_teacher_topk(s.hidden, s.k.W, 32, idx[0], val[0], ws)
    K.kdkl_teacher_topk(s.hidden.cpu().cuda(), s.k.W, 32, idx[1], val[1], ws)
    assert torch.equal(*idx) and torch.equal(*val)


def test_graphs_replay_bit_identical():
    """Two captured steps with workspaces of their own, replayed in turn and on refilled inputs."""
    steps = [Step(seed=4), Step(N=300, seed=5)]
    want = []
    for s in steps:
        s.run()
        want.append(s.snapshot())
    graphs = []
    for s in steps:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s.run()
        graphs.append(g)
    for s in steps:
        for t in s.outputs().values():
            t.fill_(float("nan"))
        s.ws_l.fill_(255)
    for _ in range(3):
        for g in graphs:
            g.replay()
    for s, w in zip(steps, want):
        for n, t in s.snapshot().items():
            assert torch.equal(t, w[n]), n
    other = Step(seed=6)
    other.run()
    want = other.snapshot()
    for name in ("x", "r", "Wb", "b", "gamma"):
        getattr(steps[0], name).copy_(getattr(other, name))
    for name in ("W", "idx", "logit", "mask"):
        getattr(steps[0].k, name).copy_(getattr(other.k, name))
    graphs[0].replay()
    for n, t in steps[0].snapshot().items():
        assert torch.equal(t, want[n]), n


@pytest.mark.parametrize("plan,dw_plan", [(0, 0), (20256, 20128), (4032, 128)])
def test_graph_of_each_kind_of_tile(plan, dw_plan):
    """A captured forward and gradient through split, whole and small tiles: the tickets of split tiles and the
    flag word are cleared inside the graph, whatever the workspace holds."""
    M, d_in, d_out = 600, 1032, 712
    o = TL._data(M, d_in, d_out, seed=20)
    e = lambda *s: torch.empty(*s, dtype=BF, device="cuda")  # noqa: E731
    dy = torch.randn(M, d_out, device="cuda").to(BF)
    y, pre, dx, dW, db = e(M, d_out), e(M, d_out), e(M, d_in), e(d_out, d_in), torch.empty(d_out, device="cuda")
    ws = _u8(K.kdkl_linear_workspace_bytes(M, d_in, d_out, True))

    def call():
        K.kdkl_linear_forward(o["x"], o["W"], y, ws, bias=o["bias"], residual=o["residual"], pre=pre,
                              activation="gelu", plan=plan)
        K.kdkl_linear_backward(dy, o["x"], o["W"], dx, dW, ws, pre=pre, dbias=db, activation="gelu", dx_plan=plan,
                               dw_plan=dw_plan)
    call()
    torch.cuda.synchronize()
    want = [t.clone() for t in (y, pre, dx, dW, db)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for _ in range(3):
        ws.fill_(255)
        for t in (y, pre, dx, dW, db):
            t.fill_(float("nan"))
        g.replay()
        assert K.kdkl_read_device_flags(ws) == 0
        assert all(torch.equal(a, b) for a, b in zip((y, pre, dx, dW, db), want))


def test_streams_give_single_stream_results():
    """Independent steps on two streams at once, each with its own workspaces."""
    a, b = Step(N=900, seed=7), Step(N=500, d=192, V=2000, seed=8)
    a.run()
    b.run()
    wa, wb = a.snapshot(), b.snapshot()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for s in (s1, s2):
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(4):
        a.run(stream=s1)
        b.run(stream=s2)
    for step, want in ((a, wa), (b, wb)):
        for n, t in step.snapshot().items():
            assert torch.equal(t, want[n]), n


def test_current_stream_is_the_default():
    s = Step(N=200, seed=9)
    s.run()
    want = s.snapshot()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s.x.mul_(1.0)      # work on the side stream that the calls must follow
        s.run()
    side.synchronize()
    for n, t in s.snapshot().items():
        assert torch.equal(t, want[n]), n


@pytest.fixture
def debug_lib(monkeypatch):
    monkeypatch.setattr(K, "_lib", None)
    monkeypatch.setattr(K, "LIB_PATH", K.DEBUG_LIB_PATH)
    yield
    monkeypatch.setattr(K, "_lib", None)


def test_bounds_checking_build(debug_lib):
    """The ragged cases through the library whose kernels check their indexes: same results, no flag raised."""
    assert "debug" in K.lib()._name
    for f8 in (False, True):
        for plan in (128, 192, 256, 20256, 4016, 2064, 1128):
            TL._check(TL._data(300, 1040, 712, f8, seed=2), "gelu", pre=True, plan=plan)
        TL._check(TL._data(1, 16, 8, f8, seed=3), "silu", pre=True)
    for dx_plan, dw_plan in ((128, 192), (20256, 256), (4032, 20256)):
        TL._check_grad(*TL._grad_data(600, 712, 1064, seed=4), "silu", dx_plan=dx_plan, dw_plan=dw_plan)
    for N, d in ((3, 24), (1003, 896), (299, 4096), (2, 32768)):
        TN._check_forward(*TN._data(N, d, BF, BF, BF, seed=1), F8)
        h, dh, gamma = TN._data(N, d, BF, BF, BF, seed=2)
        TN._check_grad(torch.randn(N, d, device="cuda").to(BF), h, gamma, dh)


def test_kernel_times_are_reported():
    s = Step(N=200, seed=10)
    s.run()
    K.kdkl_timing_read(reset=True)
    K.kdkl_timing_enable(True)
    s.run()
    K.kdkl_timing_enable(False)
    kt = K.kdkl_timing_read(reset=True)
    for name in ("rmsnorm", "rmsnorm_grad", "linear_gemm", "linear_act_grad", "linear_dx_gemm", "linear_dw_gemm"):
        assert kt[name][0] == 1 and kt[name][1] > 0, name
