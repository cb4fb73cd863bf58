"""Cases of the operators that stand between a model's last layer and its output head.

``rmsnorm``      h = x + residual, y = h / rms(h) * gamma; y in bf16, or in e4m3 with one fp32 scale per row
``rmsnorm_grad`` its gradient: dx (of x and residual alike) and dgamma
``linear``       y = residual + act(x W^T + bias), bf16 operands or e4m3 operands with a scale per row of each
``linear_grad``  its gradient: dx, dW and dbias, from the saved pre-activation

``run`` computes each in a plain form of elementary torch operations, or, where ``own`` is true, by the
calls that a user of ``output_head_kl_b200`` makes.
"""
from __future__ import annotations

import math

import torch

own = False

EPS = 1e-6
E4M3_MAX = 448.0
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}


# ------------------------------------------------------------------ cases
def _norm(name, N, d, stream, out):
    return {"name": name, "op": "rmsnorm", "N": N, "d": d, "stream": stream, "out": out}


def _norm_grad(name, N, d, stream):
    return {"name": name, "op": "rmsnorm_grad", "N": N, "d": d, "stream": stream}


def _linear(name, M, d_in, d_out, act, operands="bf16", bias=True, residual=True, pre=False):
    return {"name": name, "op": "linear", "M": M, "d_in": d_in, "d_out": d_out, "act": act, "operands": operands,
            "bias": bias, "residual": residual, "pre": pre}


def _linear_grad(name, M, d_in, d_out, act):
    return {"name": name, "op": "linear_grad", "M": M, "d_in": d_in, "d_out": d_out, "act": act}


def listed():
    return [
        # the final norm of one decoded token, at the 8B-class head's width
        _norm("norm-one-token", 1, 4096, "bf16", "bf16"),
        # the final norm of a training batch of the 8B-class head, feeding the loss
        _norm("norm-train", 32768, 4096, "bf16", "bf16"),
        # a prompt whose rows feed an 8-bit product; fp32 residual stream, odd row count
        _norm("norm-8bit-ragged", 4099, 2880, "f32", "e4m3"),
        # the loss's dHidden taken back through the final norm
        _norm_grad("norm-grad-train", 32768, 4096, "bf16"),
        # the same for a short packed batch with an fp32 residual stream
        _norm_grad("norm-grad-ragged", 1003, 896, "f32"),
        # one decoded token through a residual block ahead of the head
        _linear("linear-one-token", 1, 4096, 4096, "silu"),
        # a small ragged batch through a width projection, pre-activation kept for the gradient
        _linear("linear-ragged", 77, 2048, 2880, "gelu", residual=False, pre=True),
        # a training batch through the residual block, pre-activation kept for the gradient
        _linear("linear-train", 16384, 4096, 4096, "silu", pre=True),
        # the same product in 8 bits: a teacher's pass over a long text
        _linear("linear-8bit", 8192, 4096, 4096, "gelu_tanh", operands="e4m3"),
        # eight sequences decoded together in 8 bits
        _linear("linear-8bit-decode", 8, 4096, 4096, "silu", operands="e4m3"),
        # the gradient of the training batch's block
        _linear_grad("linear-grad-train", 16384, 4096, 4096, "silu"),
        # the gradient of a short packed batch through a width projection
        _linear_grad("linear-grad-ragged", 1003, 2048, 2880, "gelu"),
    ]


def _log_int(rng, lo, hi, step=1):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return max(lo, min(hi, (v + step - 1) // step * step))


def draw(rng):
    op = rng.choice(["rmsnorm", "rmsnorm_grad", "linear", "linear", "linear", "linear_grad"])
    if op.startswith("rmsnorm"):
        d = _log_int(rng, 64, 8192, 8)
        N = _log_int(rng, 1, min(32768, 32768 * 4096 // d))
        c = {"op": op, "N": N, "d": d, "stream": rng.choice(["bf16", "f32"])}
        if c["stream"] == "f32":
            c["N"] = max(1, N // 2)
        if op == "rmsnorm":
            c["out"] = rng.choice(["bf16", "e4m3"])
        return c
    d_in, d_out = _log_int(rng, 64, 8192, 16), _log_int(rng, 64, 8192, 8)
    most = 16384 * 4096 * 4096
    M = _log_int(rng, 1, max(1, min(32768, most // (d_in * d_out))))
    act = rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"])
    if op == "linear_grad":
        return {"op": op, "M": M, "d_in": d_in, "d_out": d_out, "act": act}
    return {"op": op, "M": M, "d_in": d_in, "d_out": d_out, "act": act, "operands": rng.choice(["bf16", "e4m3"]),
            "bias": rng.random() < 0.7, "residual": rng.random() < 0.6, "pre": rng.random() < 0.3}


def work(case):
    op = case["op"]
    if op.startswith("rmsnorm"):
        N, d = case["N"], case["d"]
        s = 2 if case["stream"] == "bf16" else 4
        if op == "rmsnorm":
            out = N * d * 2 if case["out"] == "bf16" else N * d + 4 * N
            return {"bytes": N * d * (2 + 2 * s) + out + d * s, "flops": 6 * N * d}
        return {"bytes": N * d * (2 + 3 * s) + d * (s + 4), "flops": 10 * N * d}
    M, k, n = case["M"], case["d_in"], case["d_out"]
    if op == "linear":
        b = 2 if case["operands"] == "bf16" else 1
        by = b * (M * k + n * k) + 2 * M * n
        by += (4 * (M + n) if b == 1 else 0) + (2 * n if case["bias"] else 0)
        by += (2 * M * n if case["residual"] else 0) + (2 * M * n if case["pre"] else 0)
        return {"bytes": by, "flops": 2 * M * n * k}
    by = 2 * M * n * (2 if case["act"] != "none" else 1) + 2 * (M * k + n * k) + 2 * (M * k + n * k) + 4 * n
    return {"bytes": by, "flops": 4 * M * n * k}


# ------------------------------------------------------------------ inputs
def _rows_to_e4m3(t):
    """e4m3 rows and their fp32 scales of a matrix, as 8-bit checkpoints and caches hold them."""
    scale = t.abs().amax(dim=1) / E4M3_MAX
    return (t / scale[:, None]).to(torch.float8_e4m3fn), scale


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]

    def normal(*shape, std=1.0, dtype=torch.bfloat16):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)

    def empty(*shape, dtype=torch.bfloat16):
        return torch.empty(*shape, dtype=dtype, device="cuda")

    s = {"case": case}
    if op.startswith("rmsnorm"):
        N, d, st = case["N"], case["d"], DTYPES[case["stream"]]
        # residual streams carry a few channels far larger than the rest
        chan = torch.exp(torch.randn(d, generator=g, device="cuda"))
        s["gamma"] = (1.0 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(st)
        s["h"] = (torch.randn(N, d, generator=g, device="cuda") * chan).to(st)
        if op == "rmsnorm":
            s["x"], s["residual"] = normal(N, d), s["h"]
            s["h"] = empty(N, d, dtype=st)
            s["y"] = empty(N, d, dtype=DTYPES[case["out"]])
            s["y_scale"] = empty(N, dtype=torch.float32) if case["out"] == "e4m3" else None
        else:
            s["dy"] = normal(N, d, std=2.0 ** -8)
            s["dh"] = normal(N, d, std=2.0 ** -8, dtype=st)
            s["dx"], s["dgamma"] = empty(N, d, dtype=st), empty(d, dtype=torch.float32)
        return s
    M, k, n = case["M"], case["d_in"], case["d_out"]
    W = torch.randn(n, k, generator=g, device="cuda") / math.sqrt(k)
    x = torch.randn(M, k, generator=g, device="cuda")
    if op == "linear":
        s["x_scale"] = s["w_scale"] = None
        if case["operands"] == "e4m3":
            s["x"], s["x_scale"] = _rows_to_e4m3(x)
            s["W"], s["w_scale"] = _rows_to_e4m3(W)
        else:
            s["x"], s["W"] = x.bfloat16(), W.bfloat16()
        s["bias"] = normal(n, std=0.2) if case["bias"] else None
        s["residual"] = normal(M, n) if case["residual"] else None
        s["y"] = empty(M, n)
        s["pre"] = empty(M, n) if case["pre"] else None
        return s
    s["x"], s["W"] = x.bfloat16(), W.bfloat16()
    s["dy"] = normal(M, n, std=2.0 ** -8)
    s["pre"] = normal(M, n) if case["act"] != "none" else None
    s["dx"], s["dW"], s["dbias"] = empty(M, k), empty(n, k), empty(n, dtype=torch.float32)
    return s


# ------------------------------------------------------------------ plain forms (fp32)
def _act(z, kind):
    if kind == "relu":
        return torch.clamp(z, min=0.0)
    if kind == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if kind == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    if kind == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _act_grad(z, kind):
    if kind == "relu":
        return (z > 0).to(z.dtype)
    if kind == "gelu":
        cdf = 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5)))
        return cdf + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2.0 * math.pi))
    if kind == "gelu_tanh":
        c = math.sqrt(2.0 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * z * z)
    if kind == "silu":
        p = 1.0 / (1.0 + torch.exp(-z))
        return p * (1.0 + z * (1.0 - p))
    return torch.ones_like(z)


def _plain_norm(s):
    h = s["x"].float() + s["residual"].float()
    y = h * torch.rsqrt((h * h).mean(dim=1, keepdim=True) + EPS) * s["gamma"].float()
    out = {"h": h.to(s["h"].dtype)}
    if s["y_scale"] is None:
        out["y"] = y.bfloat16()
    else:
        scale = y.abs().amax(dim=1) / E4M3_MAX
        q = torch.where(scale[:, None] > 0, y / scale[:, None], torch.zeros_like(y))
        out["y"], out["y_scale"] = q.to(torch.float8_e4m3fn), scale
    return out


def _plain_norm_grad(s):
    h, dy, gamma = s["h"].float(), s["dy"].float(), s["gamma"].float()
    rstd = torch.rsqrt((h * h).mean(dim=1, keepdim=True) + EPS)
    xhat = h * rstd
    a = dy * gamma
    dx = rstd * (a - xhat * (a * xhat).mean(dim=1, keepdim=True)) + s["dh"].float()
    return {"dx": dx.to(s["dx"].dtype), "dgamma": (dy * xhat).sum(dim=0)}


def _plain_linear(s):
    c = s["case"]
    z = s["x"].float() @ s["W"].float().t()
    if s["x_scale"] is not None:
        z = z * s["x_scale"][:, None] * s["w_scale"][None, :]
    if s["bias"] is not None:
        z = z + s["bias"].float()
    y = _act(z, c["act"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    out = {"y": y.bfloat16()}
    if s["pre"] is not None:
        out["pre"] = z.bfloat16()
    return out


def _plain_linear_grad(s):
    dz = s["dy"].float()
    if s["pre"] is not None:
        dz = dz * _act_grad(s["pre"].float(), s["case"]["act"])
    dx = dz @ s["W"].float()
    dW = dz.t() @ s["x"].float()
    return {"dx": dx.bfloat16(), "dW": dW.bfloat16(), "dbias": dz.sum(dim=0)}


# ------------------------------------------------------------------ the framework's calls
def _own(s):
    import output_head_kl_b200 as K
    c = s["case"]
    op = c["op"]
    if op == "rmsnorm":
        K.kdkl_rmsnorm_forward(s["x"], s["gamma"], s["y"], residual=s["residual"], h=s["h"], y_scale=s["y_scale"],
                               eps=EPS)
        out = {"h": s["h"], "y": s["y"]}
        if s["y_scale"] is not None:
            out["y_scale"] = s["y_scale"]
        return out
    if op == "rmsnorm_grad":
        if "ws" not in s:
            s["ws"] = torch.empty(K.kdkl_rmsnorm_workspace_bytes(c["N"], c["d"]), dtype=torch.uint8, device="cuda")
        K.kdkl_rmsnorm_backward(s["dy"], s["h"], s["gamma"], s["dx"], s["dgamma"], s["ws"], dh=s["dh"], eps=EPS)
        return {"dx": s["dx"], "dgamma": s["dgamma"]}
    if "ws" not in s:
        size = K.kdkl_linear_workspace_bytes(c["M"], c["d_in"], c["d_out"], backward=op == "linear_grad")
        s["ws"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    if op == "linear":
        K.kdkl_linear_forward(s["x"], s["W"], s["y"], s["ws"], bias=s["bias"], residual=s["residual"], pre=s["pre"],
                              activation=c["act"], x_scale=s["x_scale"], w_scale=s["w_scale"])
        return {"y": s["y"]} if s["pre"] is None else {"y": s["y"], "pre": s["pre"]}
    K.kdkl_linear_backward(s["dy"], s["x"], s["W"], s["dx"], s["dW"], s["ws"], pre=s["pre"], dbias=s["dbias"],
                           activation=c["act"])
    return {"dx": s["dx"], "dW": s["dW"], "dbias": s["dbias"]}


def run(state):
    if own:
        return _own(state)
    return {"rmsnorm": _plain_norm, "rmsnorm_grad": _plain_norm_grad, "linear": _plain_linear,
            "linear_grad": _plain_linear_grad}[state["case"]["op"]](state)


# ------------------------------------------------------------------ the definitions in 64 bits
def _phi(z):
    """Standard normal distribution function."""
    return torch.special.ndtr(z)


def _sigmoid(z):
    return torch.special.expit(z)


def _f(z, kind):
    """(act(z), act'(z)) of the definition, fp64."""
    if kind == "none":
        return z, torch.ones_like(z)
    if kind == "relu":
        on = z > 0
        return torch.where(on, z, 0.0 * z), on.double()
    if kind == "gelu":
        return z * _phi(z), _phi(z) + z * torch.exp(-z.square() / 2) / math.sqrt(2 * math.pi)
    if kind == "silu":
        return z * _sigmoid(z), _sigmoid(z) + z * _sigmoid(z) * _sigmoid(-z)
    # 0.5 (1 + tanh u) = sigmoid(2 u)
    u2 = 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z.pow(3))
    du2 = 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z.square())
    return z * _sigmoid(u2), _sigmoid(u2) + z * _sigmoid(u2) * _sigmoid(-u2) * du2


def _e4m3_nearest(v):
    """The nearest e4m3 value (ties to even), by exponent: 3 mantissa bits, smallest step 2^-9."""
    _, e = torch.frexp(v)
    step = torch.exp2(torch.clamp(e - 1, min=-6).double() - 3)
    return torch.clamp(torch.round(v / step) * step, -E4M3_MAX, E4M3_MAX)


def exact(case, seed):
    s = prepare(case, seed)
    d = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor)}
    op = case["op"]
    if op == "rmsnorm":
        h = d["x"] + d["residual"]
        rms = torch.sqrt(h.square().sum(1) / case["d"] + EPS)
        y = d["gamma"] * (h / rms[:, None])
        if case["out"] == "bf16":
            return {"h": h, "y": y}
        top = y.abs().max(dim=1).values
        safe = torch.where(top > 0, top, torch.ones_like(top))
        return {"h": h, "y": _e4m3_nearest(y * (E4M3_MAX / safe)[:, None]), "y_scale": top / E4M3_MAX}
    if op == "rmsnorm_grad":
        h, dy = d["h"], d["dy"]
        n = case["d"]
        r2 = h.square().sum(1) / n + EPS
        gdy = dy * d["gamma"]
        dot = (gdy * h).sum(1) / n
        dx = gdy / r2.sqrt()[:, None] - h * (dot / r2.pow(1.5))[:, None] + d["dh"]
        return {"dx": dx, "dgamma": (dy * h / r2.sqrt()[:, None]).sum(0)}
    if op == "linear":
        if case["operands"] == "e4m3":
            x, W = d["x"] * d["x_scale"][:, None], d["W"] * d["w_scale"][:, None]
        else:
            x, W = d["x"], d["W"]
        z = torch.einsum("mk,nk->mn", x, W)
        if case["bias"]:
            z = z + d["bias"]
        y = _f(z, case["act"])[0]
        if case["residual"]:
            y = d["residual"] + y
        return {"y": y, "pre": z} if case["pre"] else {"y": y}
    dz = d["dy"]
    if case["act"] != "none":
        dz = dz * _f(d["pre"], case["act"])[1]
    return {"dx": torch.einsum("mn,nk->mk", dz, d["W"]), "dW": torch.einsum("mn,mk->nk", dz, d["x"]),
            "dbias": dz.sum(0)}
