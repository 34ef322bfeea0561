"""The transformer-block operators on their measured sizes: a product with its
epilogue (``linear``), its gradients (``linear_backward``), the root-mean-square
norm with the residual's addition (``rms_norm``) and its gradients
(``rms_norm_backward``).

A case is a dict: ``op`` names the operator, ``dtype`` its 16-bit type (or
``e4m3`` where the operands, or the norm's output, are 8-bit floats with scales).

linear:          C = act(s_a s_b (A @ B) + bias) + residual, A [M, K], B [K, N]
linear_backward: G [M, N] is C's gradient, P = A @ B + bias as it was saved;
                 D = G act'(P), dA = D B^T, dB = A^T D, dbias = column sums of D
rms_norm:        h = x + residual, y = w h / sqrt(mean(h^2) + eps); in 8 bits
                 q = round(448 y / a) with the scale a / 448, a = max|y| of the row
rms_norm_backward: gradients of x (and so of the residual) and of w
"""
import math

import torch

own = False

EPS = 1e-6
E4M3_MAX = 448.0
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    return [
        # one token of a decoding step enters a layer: latency
        dict(name="norm token", op="rms_norm", dtype="bf16", rows=1, width=4096, residual=True, out="16", rstd=False),
        # a prompt's tokens, the output quantised for an 8-bit product
        dict(name="norm prompt 8-bit", op="rms_norm", dtype="bf16", rows=4096, width=8192, residual=True, out="e4m3", rstd=False),
        # training forward, odd width: the reciprocal norms are kept for the backward pass
        dict(name="norm train odd", op="rms_norm", dtype="fp16", rows=1000, width=5000, residual=True, out="16", rstd=True),
        # training backward at a usual width, with the gradient that arrives on the residual path
        dict(name="norm backward", op="rms_norm_backward", dtype="bf16", rows=8192, width=4096, through=True),
        # the same where the row is no multiple of a vector and nothing arrives on the residual path
        dict(name="norm backward odd", op="rms_norm_backward", dtype="fp16", rows=513, width=4095, through=False),
        # one token through one projection: the weights are read once, latency
        dict(name="linear token", op="linear", dtype="bf16", M=1, N=4096, K=4096, act="silu", bias=True, residual=False, pre=False, weight="kn"),
        # a batch of decoding sequences through the projection back into the residual stream
        dict(name="linear batch", op="linear", dtype="fp16", M=48, N=4096, K=8192, act="none", bias=True, residual=True, pre=False, weight="nk"),
        # ragged in every size, weights stored column by column
        dict(name="linear ragged", op="linear", dtype="fp16", M=4000, N=5000, K=3000, act="gelu_tanh", bias=True, residual=False, pre=False, weight="nk"),
        # training forward of the widest projection: the values before the activation are kept
        dict(name="linear train", op="linear", dtype="bf16", M=8192, N=16384, K=4096, act="gelu", bias=True, residual=False, pre=True, weight="kn"),
        # a prompt through an 8-bit projection back into the residual stream
        dict(name="linear prompt 8-bit", op="linear", dtype="e4m3", M=4096, N=8192, K=8192, act="none", bias=False, residual=True, pre=False, weight="nk"),
        # gradients of a projection with its activation
        dict(name="linear backward", op="linear_backward", dtype="bf16", M=4096, N=8192, K=4096, act="gelu", bias=True, weight="kn"),
        # gradients for a short, odd sequence
        dict(name="linear backward odd", op="linear_backward", dtype="fp16", M=257, N=1000, K=513, act="relu", bias=True, weight="nk"),
    ]


def _size(rng, low, high):
    """Spread over the logarithm; a third of the sizes odd, a third multiples of 8, a third of 64."""
    n = math.exp(rng.uniform(math.log(low), math.log(high)))
    step = rng.choice((1, 8, 64))
    n = max(low, min(high, round(n / step) * step))
    if step == 1:
        n |= 1
    return int(n) + (8 if n == 3072 else 0)


def draw(rng):
    op = rng.choice(("rms_norm", "rms_norm_backward", "linear", "linear", "linear_backward"))
    dtype = rng.choice(("bf16", "fp16"))
    if op in ("rms_norm", "rms_norm_backward"):
        rows, width = _size(rng, 1, 16384), _size(rng, 64, 16384)
        rows = min(rows, max(1, (1 << 25) // width))
        if op == "rms_norm":
            out = rng.choice(("16", "e4m3"))
            return dict(op=op, dtype=dtype, rows=rows, width=width, residual=rng.random() < 0.7, out=out, rstd=rng.random() < 0.4)
        return dict(op=op, dtype=dtype, rows=rows, width=width, through=rng.random() < 0.6)
    M, N, K = _size(rng, 1, 8192), _size(rng, 128, 16384), _size(rng, 64, 8192)
    most = 8192 * 16384 * 4096 // (2 if op == "linear_backward" else 1)
    while M * N * K > most:
        M = max(1, M // 2 + 1)
    act = rng.choice(("none", "relu", "gelu", "gelu_tanh", "silu"))
    bias, weight = rng.random() < 0.6, rng.choice(("kn", "nk"))
    if op == "linear_backward":
        return dict(op=op, dtype=dtype, M=M, N=N, K=K, act=act, bias=bias, weight=weight)
    if rng.random() < 0.3:
        dtype, weight = "e4m3", "nk"
    return dict(op=op, dtype=dtype, M=M, N=N, K=K, act=act, bias=bias, residual=rng.random() < 0.5,
                pre=act != "none" and dtype != "e4m3" and rng.random() < 0.4, weight=weight)


# ------------------------------------------------------------------ inputs
def _normal(gen, *shape, scale=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dtype)


def _eight_bits(x):
    """Rows of x as 8-bit floats and one scale per row."""
    top = x.abs().amax(dim=1).clamp_min(1e-12)
    return (x * (E4M3_MAX / top)[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), top / E4M3_MAX


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    s = {"case": case}
    op = case["op"]
    if op in ("rms_norm", "rms_norm_backward"):
        t, rows, width = TYPES[case["dtype"]], case["rows"], case["width"]
        s["weight"] = _normal(gen, width, scale=0.1).add_(1.0).to(t)
        x = _normal(gen, rows, width)
        x[:, :: max(1, width // 8)] *= 8.0  # a residual stream has a few strong channels
        s["x"] = x.to(t)
        if op == "rms_norm":
            s["residual"] = _normal(gen, rows, width, scale=2.0, dtype=t) if case["residual"] else None
            return s
        s["rstd"] = torch.rsqrt(s["x"].float().square().mean(dim=1) + EPS)
        s["grad"] = _normal(gen, rows, width, scale=0.5, dtype=t)
        s["through"] = _normal(gen, rows, width, scale=0.5, dtype=t) if case["through"] else None
        return s
    M, N, K = case["M"], case["N"], case["K"]
    eight = case["dtype"] == "e4m3"
    t = torch.bfloat16 if eight else TYPES[case["dtype"]]
    if eight:
        s["A"], s["scale_a"] = _eight_bits(_normal(gen, M, K))
        W, s["scale_b"] = _eight_bits(_normal(gen, N, K, scale=K ** -0.5))
        s["B"] = W.t()
    else:
        s["A"] = _normal(gen, M, K, dtype=t)
        s["scale_a"] = s["scale_b"] = None
        s["B"] = _normal(gen, K, N, scale=K ** -0.5, dtype=t) if case["weight"] == "kn" else _normal(gen, N, K, scale=K ** -0.5, dtype=t).t()
    s["bias"] = _normal(gen, N, scale=0.5, dtype=t) if case["bias"] else None
    if op == "linear":
        s["residual"] = _normal(gen, M, N, scale=2.0, dtype=t) if case["residual"] else None
    else:
        s["grad"] = _normal(gen, M, N, dtype=t)
        s["P"] = _normal(gen, M, N, dtype=t) if case["act"] != "none" else None
    return s


# ------------------------------------------------------------------ plain forms
def _act(x, name):
    if name == "relu":
        return torch.where(x < 0, torch.zeros_like(x), x)
    if name == "silu":
        return x / (1 + torch.exp(-x))
    if name == "gelu":
        return 0.5 * x * (1 + torch.erf(x * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * x * (1 + torch.tanh(math.sqrt(2 / math.pi) * (x + 0.044715 * x * x * x)))
    return x


def _act_slope(x, name):
    if name == "relu":
        return (x > 0).to(x.dtype)
    if name == "silu":
        g = 1 / (1 + torch.exp(-x))
        return g * (1 + x * (1 - g))
    if name == "gelu":
        return 0.5 * (1 + torch.erf(x * math.sqrt(0.5))) + x * torch.exp(-0.5 * x * x) * (1 / math.sqrt(2 * math.pi))
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (x + 0.044715 * x * x * x))
    return 0.5 * (1 + t) + 0.5 * x * (1 - t * t) * c * (1 + 3 * 0.044715 * x * x)


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "rms_norm":
        h = s["x"].float()
        if s["residual"] is not None:
            h = h + s["residual"].float()
        rstd = torch.rsqrt((h * h).mean(dim=1) + EPS)
        y = h * rstd[:, None] * s["weight"].float()
        out = {}
        if case["out"] == "e4m3":
            top = y.abs().amax(dim=1)
            out["q"] = (y * (E4M3_MAX / top)[:, None]).to(torch.float8_e4m3fn)
            out["scale"] = top / E4M3_MAX
        else:
            out["y"] = y.to(s["x"].dtype)
        if s["residual"] is not None:
            out["h"] = h.to(s["x"].dtype)
        if case["rstd"]:
            out["rstd"] = rstd
        return out
    if op == "rms_norm_backward":
        dy, rstd = s["grad"].float(), s["rstd"][:, None]
        unit = s["x"].float() * rstd
        g = dy * s["weight"].float()
        dx = rstd * (g - unit * (g * unit).mean(dim=1, keepdim=True))
        if s["through"] is not None:
            dx = dx + s["through"].float()
        return {"dx": dx.to(s["x"].dtype), "dweight": (dy * unit).sum(dim=0)}
    A, B = s["A"].float(), s["B"].float()
    if op == "linear":
        P = A @ B
        if s["scale_a"] is not None:
            P = P * s["scale_a"][:, None] * s["scale_b"]
        if s["bias"] is not None:
            P = P + s["bias"].float()
        C = _act(P, case["act"])
        if s["residual"] is not None:
            C = C + s["residual"].float()
        t = torch.bfloat16 if case["dtype"] == "e4m3" else s["A"].dtype
        return {"C": C.to(t), "P": P.to(t)} if case["pre"] else {"C": C.to(t)}
    D = s["grad"].float()
    if case["act"] != "none":
        D = D * _act_slope(s["P"].float(), case["act"])
    out = {"dA": (D @ B.t()).to(s["A"].dtype), "dB": (A.t() @ D).to(s["B"].dtype)}
    if case["bias"]:
        out["dbias"] = D.sum(dim=0)
    return out


# ------------------------------------------------------------------ the framework's operators
def _own(s):
    import dense_gemm_gb300 as dg
    case = s["case"]
    op = case["op"]
    if op == "rms_norm":
        r = dg.rms_norm(s["x"], s["weight"], residual=s["residual"], eps=EPS, return_rstd=case["rstd"],
                        out_dtype=torch.float8_e4m3fn if case["out"] == "e4m3" else None)
        out = {"q": r.y, "scale": r.scale} if case["out"] == "e4m3" else {"y": r.y}
        if s["residual"] is not None:
            out["h"] = r.h
        if case["rstd"]:
            out["rstd"] = r.rstd
        return out
    if op == "rms_norm_backward":
        dx, dweight = dg.rms_norm_backward(s["grad"], s["x"], s["weight"], s["rstd"], grad_h=s["through"])
        return {"dx": dx, "dweight": dweight}
    if op == "linear":
        r = dg.linear(s["A"], s["B"], s["bias"], activation=case["act"], residual=s["residual"], scale_a=s["scale_a"],
                      scale_b=s["scale_b"], return_pre=case["pre"])
        return {"C": r[0], "P": r[1]} if case["pre"] else {"C": r}
    dA, dB, dbias = dg.linear_backward(s["grad"], s["A"], s["B"], pre=s["P"], activation=case["act"], need_bias=case["bias"])
    return {"dA": dA, "dB": dB, "dbias": dbias} if case["bias"] else {"dA": dA, "dB": dB}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    if case["op"] == "rms_norm":
        n, rows = case["rows"] * case["width"], case["rows"]
        read = n * 2 * (2 if case["residual"] else 1) + case["width"] * 2
        write = n * (1 if case["out"] == "e4m3" else 2) + (rows * 4 if case["out"] == "e4m3" else 0)
        write += n * 2 if case["residual"] else 0
        return {"bytes": read + write + (rows * 4 if case["rstd"] else 0), "flops": 5 * n}
    if case["op"] == "rms_norm_backward":
        n, rows, width = case["rows"] * case["width"], case["rows"], case["width"]
        return {"bytes": n * 2 * (4 if case["through"] else 3) + rows * 4 + width * 2 + width * 4, "flops": 9 * n}
    M, N, K = case["M"], case["N"], case["K"]
    e = 1 if case["dtype"] == "e4m3" else 2
    if case["op"] == "linear":
        moved = (M * K + K * N) * e + M * N * 2 * (1 + bool(case["residual"]) + bool(case["pre"])) + (N * 2 if case["bias"] else 0)
        return {"bytes": moved + ((M + N) * 4 if e == 1 else 0), "flops": 2 * M * N * K}
    moved = M * N * 2 * (2 if case["act"] != "none" else 1) + 2 * (M * K + K * N) * 2 + (N * 4 if case["bias"] else 0)
    return {"bytes": moved, "flops": 4 * M * N * K}


# ------------------------------------------------------------------ the definitions in 64 bits
def _phi(x):
    """The normal distribution's cumulative function."""
    return torch.special.erfc(x * -math.sqrt(0.5)) * 0.5


def _exact_act(x, name):
    if name == "relu":
        return x.clamp_min(0)
    if name == "silu":
        return x * torch.sigmoid(x)
    if name == "gelu":
        return x * _phi(x)
    if name == "gelu_tanh":
        return x * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (x + 0.044715 * x.pow(3)))
    return x


def _exact_slope(x, name):
    if name == "relu":
        return torch.heaviside(x, torch.zeros((), dtype=x.dtype, device=x.device))
    if name == "silu":
        g = torch.sigmoid(x)
        return g + x * g * torch.sigmoid(-x)
    if name == "gelu":
        return _phi(x) + x * torch.exp(-x * x / 2) / math.sqrt(2 * math.pi)
    c = 2 * math.sqrt(2 / math.pi)
    g = torch.sigmoid(c * (x + 0.044715 * x.pow(3)))
    return g + x * g * (1 - g) * c * (1 + 0.134145 * x.square())


def exact(case, seed):
    s = prepare(case, seed)
    wide = {k: v.to(torch.float64) if isinstance(v, torch.Tensor) else v for k, v in s.items()}
    op = case["op"]
    if op == "rms_norm":
        h = wide["x"] if wide["residual"] is None else wide["x"] + wide["residual"]
        norm = (h.square().sum(dim=1) / case["width"] + EPS).sqrt()
        y = h / norm[:, None] * wide["weight"]
        out = {}
        if case["out"] == "e4m3":
            scale = y.abs().max(dim=1).values / E4M3_MAX
            out["q"] = (y / scale[:, None]).to(torch.float8_e4m3fn).to(torch.float64)
            out["scale"] = scale
        else:
            out["y"] = y
        if wide["residual"] is not None:
            out["h"] = h
        if case["rstd"]:
            out["rstd"] = 1 / norm
        return out
    if op == "rms_norm_backward":
        h, r, dy = wide["x"], wide["rstd"], wide["grad"]
        dot = (dy * wide["weight"] * h).sum(dim=1)
        dx = dy * wide["weight"] * r[:, None] - h * (r.pow(3) * dot / case["width"])[:, None]
        if wide["through"] is not None:
            dx += wide["through"]
        return {"dx": dx, "dweight": torch.einsum("rw,rw,r->w", dy, h, r)}
    if op == "linear":
        P = torch.matmul(wide["A"], wide["B"])
        if wide["scale_a"] is not None:
            P = P * torch.outer(wide["scale_a"], wide["scale_b"])
        if wide["bias"] is not None:
            P += wide["bias"]
        C = _exact_act(P, case["act"])
        if wide["residual"] is not None:
            C = C + wide["residual"]
        return {"C": C, "P": P} if case["pre"] else {"C": C}
    D = wide["grad"] if case["act"] == "none" else wide["grad"] * _exact_slope(wide["P"], case["act"])
    out = {"dA": torch.matmul(D, wide["B"].mT), "dB": torch.matmul(wide["A"].mT, D)}
    if case["bias"]:
        out["dbias"] = torch.sum(D, 0)
    return out
