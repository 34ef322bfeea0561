"""The operators around a block's products in 8 bits on their measured sizes: layer
norm (``layer_norm``) and its gradients (``layer_norm_backward``), rows kept in
8-bit floats with a scale each (``quantize_rows``), the gradients of a product
whose operand and pre-activation values were kept so (``linear_backward``), and a
product of 8-bit integers with scales for each token and channel (``linear``).

A case is a dict: ``op`` names the operator, ``dtype`` the 16-bit type around it.

layer_norm:          h = x + residual, y = w (h - mean) / sqrt(var + eps) + b; in 8 bits
                     q = round(448 y / a) with the scale a / 448, a = max|y| of the row
layer_norm_backward: gradients of x (and so of the residual), of w and of b
quantize_rows:       q = round(448 x / a), scale a / 448, a = max|x| of the row
linear_backward:     A = act_a(s_a A8) [M, K], P = s_p P8 [M, N] as they were kept, G is C's
                     gradient; D = G act'(P), dA = D B^T, dB = A^T D, dbias = column sums of D
linear_int8:         C = act(s_a s_b (A @ B) + bias) + residual, A and B whole numbers in -127 .. 127
"""
import math

import torch

own = False

EPS = 1e-5
E4M3_MAX = 448.0
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    return [
        # one token of a decoding step enters a layer: latency
        dict(name="layer norm token", op="layer_norm", dtype="bf16", rows=1, width=4096, residual=True, out="16", stats=False),
        # a prompt's tokens, the output quantised for an 8-bit product
        dict(name="layer norm prompt 8-bit", op="layer_norm", dtype="bf16", rows=4096, width=8192, residual=True, out="e4m3", stats=False),
        # training forward, odd width: the rows' means and reciprocal deviations are kept for the backward pass
        dict(name="layer norm train odd", op="layer_norm", dtype="fp16", rows=1000, width=5000, residual=True, out="16", stats=True),
        # training backward at a usual width, with the gradient that arrives on the residual path
        dict(name="layer norm backward", op="layer_norm_backward", dtype="bf16", rows=8192, width=4096, through=True),
        # the same where the row is no multiple of a vector and nothing arrives on the residual path
        dict(name="layer norm backward odd", op="layer_norm_backward", dtype="fp16", rows=513, width=4095, through=False),
        # a feed-forward block's widest activation, kept for the backward pass
        dict(name="checkpoint", op="quantize_rows", dtype="bf16", rows=4096, width=16384),
        # a short, odd sequence's
        dict(name="checkpoint odd", op="quantize_rows", dtype="fp16", rows=999, width=5001),
        # gradients of the projection back: its operand is made again from the values before the activation
        dict(name="backward from checkpoint", op="linear_backward", dtype="bf16", M=4096, N=4096, K=8192, act="none", act_a="gelu", bias=True, weight="nk"),
        # gradients of the projection into the block for a short, odd sequence: operand and values before the activation
        dict(name="backward from checkpoint odd", op="linear_backward", dtype="fp16", M=257, N=1000, K=513, act="relu", act_a="none", bias=True, weight="nk"),
        # one token through one projection: the weights are read once, latency
        dict(name="integers token", op="linear_int8", dtype="bf16", M=1, N=4096, K=4096, act="silu", bias=True, residual=False),
        # a batch of decoding sequences through the projection back into the residual stream
        dict(name="integers batch", op="linear_int8", dtype="bf16", M=48, N=4096, K=8192, act="none", bias=True, residual=True),
        # a prompt, ragged in every size
        dict(name="integers prompt ragged", op="linear_int8", dtype="fp16", M=4000, N=5000, K=3000, act="gelu_tanh", bias=True, residual=False),
    ]


def _size(rng, low, high):
    """Spread over the logarithm; a third of the sizes odd, a third multiples of 8, a third of 64."""
    n = math.exp(rng.uniform(math.log(low), math.log(high)))
    step = rng.choice((1, 8, 64))
    n = max(low, min(high, round(n / step) * step))
    return int(n | 1 if step == 1 else n)


def draw(rng):
    op = rng.choice(("layer_norm", "layer_norm_backward", "quantize_rows", "linear_backward", "linear_int8", "linear_int8"))
    dtype = rng.choice(("bf16", "fp16"))
    if op in ("layer_norm", "layer_norm_backward", "quantize_rows"):
        rows, width = _size(rng, 1, 16384), _size(rng, 64, 16384)
        rows = min(rows, max(1, (1 << 25) // width))
        if op == "layer_norm":
            out = rng.choice(("16", "e4m3"))
            return dict(op=op, dtype=dtype, rows=rows, width=width, residual=rng.random() < 0.7, out=out, stats=rng.random() < 0.4)
        if op == "quantize_rows":
            return dict(op=op, dtype=dtype, rows=rows, width=width)
        return dict(op=op, dtype=dtype, rows=rows, width=width, through=rng.random() < 0.6)
    M, N, K = _size(rng, 1, 8192), _size(rng, 128, 8192), _size(rng, 64, 8192)
    most = 4096 * 4096 * 8192 // 2
    while M * N * K > most:
        M = max(1, M // 2 + 1)
    act, bias = rng.choice(("none", "relu", "gelu", "gelu_tanh", "silu")), rng.random() < 0.6
    if op == "linear_int8":
        return dict(op=op, dtype=dtype, M=M, N=N, K=K, act=act, bias=bias, residual=rng.random() < 0.5)
    # the projection into a block keeps P and its operand, the one back only what its operand was made from
    act_a = "none" if act != "none" else rng.choice(("relu", "gelu", "gelu_tanh", "silu"))
    return dict(op=op, dtype=dtype, M=M, N=N, K=K, act=act, act_a=act_a, bias=bias, weight=rng.choice(("kn", "nk")))


# ------------------------------------------------------------------ inputs
def _normal(gen, *shape, scale=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dtype)


def _eight_bits(x):
    """Rows of x as 8-bit floats and one scale per row."""
    top = x.abs().amax(dim=1).clamp_min(1e-12)
    return (x * (E4M3_MAX / top)[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), top / E4M3_MAX


def _integers(x):
    """Rows of x as whole numbers in -127 .. 127 and one scale per row."""
    scale = x.abs().amax(dim=1).clamp_min(1e-12) / 127
    return torch.round(x / scale[:, None]).clamp(-127, 127).to(torch.int8), scale


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    s = {"case": case}
    op, t = case["op"], TYPES[case["dtype"]]
    if op in ("layer_norm", "layer_norm_backward", "quantize_rows"):
        rows, width = case["rows"], case["width"]
        x = _normal(gen, rows, width)
        x[:, :: max(1, width // 8)] *= 8.0  # a residual stream has a few strong channels
        if op == "quantize_rows":
            s["x"] = x.to(t)
            return s
        x += _normal(gen, rows, 1, scale=0.5)  # and rows a mean
        s["x"] = x.to(t)
        s["weight"] = _normal(gen, width, scale=0.1).add_(1.0).to(t)
        if op == "layer_norm":
            s["bias"] = _normal(gen, width, scale=0.1, dtype=t)
            s["residual"] = _normal(gen, rows, width, scale=2.0, dtype=t) if case["residual"] else None
            return s
        h = s["x"].float()
        s["mean"] = h.mean(dim=1)
        s["rstd"] = torch.rsqrt((h - s["mean"][:, None]).square().mean(dim=1) + EPS)
        s["grad"] = _normal(gen, rows, width, scale=0.5, dtype=t)
        s["through"] = _normal(gen, rows, width, scale=0.5, dtype=t) if case["through"] else None
        return s
    M, N, K = case["M"], case["N"], case["K"]
    if op == "linear_int8":
        s["A"], s["scale_a"] = _integers(_normal(gen, M, K))
        W, s["scale_b"] = _integers(_normal(gen, N, K, scale=K ** -0.5))
        s["B"] = W.t()
        s["bias"] = _normal(gen, N, scale=0.5, dtype=t) if case["bias"] else None
        s["residual"] = _normal(gen, M, N, scale=2.0, dtype=t) if case["residual"] else None
        return s
    s["A"], s["scale_a"] = _eight_bits(_normal(gen, M, K))
    s["B"] = _normal(gen, K, N, scale=K ** -0.5, dtype=t) if case["weight"] == "kn" else _normal(gen, N, K, scale=K ** -0.5, dtype=t).t()
    s["P"], s["scale_p"] = _eight_bits(_normal(gen, M, N)) if case["act"] != "none" else (None, None)
    s["grad"] = _normal(gen, M, N, dtype=t)
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
    if op == "layer_norm":
        h = s["x"].float()
        if s["residual"] is not None:
            h = h + s["residual"].float()
        mean = h.mean(dim=1)
        centred = h - mean[:, None]
        rstd = torch.rsqrt((centred * centred).mean(dim=1) + EPS)
        y = centred * rstd[:, None] * s["weight"].float() + s["bias"].float()
        out = {}
        if case["out"] == "e4m3":
            top = y.abs().amax(dim=1)
            out["q"] = (y * (E4M3_MAX / top)[:, None]).to(torch.float8_e4m3fn)
            out["scale"] = top / E4M3_MAX
        else:
            out["y"] = y.to(s["x"].dtype)
        if s["residual"] is not None:
            out["h"] = h.to(s["x"].dtype)
        if case["stats"]:
            out["mean"], out["rstd"] = mean, rstd
        return out
    if op == "layer_norm_backward":
        dy, rstd = s["grad"].float(), s["rstd"][:, None]
        unit = (s["x"].float() - s["mean"][:, None]) * rstd
        g = dy * s["weight"].float()
        dx = rstd * (g - g.mean(dim=1, keepdim=True) - unit * (g * unit).mean(dim=1, keepdim=True))
        if s["through"] is not None:
            dx = dx + s["through"].float()
        return {"dx": dx.to(s["x"].dtype), "dweight": (dy * unit).sum(dim=0), "dbias": dy.sum(dim=0)}
    if op == "quantize_rows":
        x = s["x"].float()
        top = x.abs().amax(dim=1)
        return {"q": (x * (E4M3_MAX / top)[:, None]).to(torch.float8_e4m3fn), "scale": top / E4M3_MAX}
    if op == "linear_int8":
        x = (s["A"].float() @ s["B"].float()) * s["scale_a"][:, None] * s["scale_b"]
        if s["bias"] is not None:
            x = x + s["bias"].float()
        c = _act(x, case["act"])
        if s["residual"] is not None:
            c = c + s["residual"].float()
        return {"C": c.to(TYPES[case["dtype"]])}
    A, B, D = _act(s["A"].float() * s["scale_a"][:, None], case["act_a"]), s["B"].float(), s["grad"].float()
    if case["act"] != "none":
        D = D * _act_slope(s["P"].float() * s["scale_p"][:, None], case["act"])
    out = {"dA": (D @ B.t()).to(s["B"].dtype), "dB": (A.t() @ D).to(s["B"].dtype)}
    if case["bias"]:
        out["dbias"] = D.sum(dim=0)
    return out


# ------------------------------------------------------------------ the framework's operators
def _own(s):
    import dense_gemm_gb300 as dg
    case = s["case"]
    op = case["op"]
    if op == "layer_norm":
        r = dg.layer_norm(s["x"], s["weight"], s["bias"], residual=s["residual"], eps=EPS, return_stats=case["stats"],
                          out_dtype=torch.float8_e4m3fn if case["out"] == "e4m3" else None)
        out = {"q": r.y, "scale": r.scale} if case["out"] == "e4m3" else {"y": r.y}
        if s["residual"] is not None:
            out["h"] = r.h
        if case["stats"]:
            out["mean"], out["rstd"] = r.mean, r.rstd
        return out
    if op == "layer_norm_backward":
        dx, dweight, dbias = dg.layer_norm_backward(s["grad"], s["x"], s["weight"], s["mean"], s["rstd"], grad_h=s["through"])
        return {"dx": dx, "dweight": dweight, "dbias": dbias}
    if op == "quantize_rows":
        q, scale = dg.quantize_rows(s["x"], torch.float8_e4m3fn)
        return {"q": q, "scale": scale}
    if op == "linear_int8":
        return {"C": dg.linear(s["A"], s["B"], s["bias"], activation=case["act"], residual=s["residual"], scale_a=s["scale_a"],
                               scale_b=s["scale_b"], out_dtype=TYPES[case["dtype"]])}
    dA, dB, dbias = dg.linear_backward(s["grad"], s["A"], s["B"], scale_a=s["scale_a"], activation_a=case["act_a"], pre=s["P"],
                                       scale_pre=s["scale_p"], activation=case["act"], need_bias=case["bias"])
    return {"dA": dA, "dB": dB, "dbias": dbias} if case["bias"] else {"dA": dA, "dB": dB}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op = case["op"]
    if op in ("layer_norm", "layer_norm_backward", "quantize_rows"):
        rows, width = case["rows"], case["width"]
        n = rows * width
        if op == "quantize_rows":
            return {"bytes": n * 3 + rows * 4, "flops": 3 * n}
        if op == "layer_norm_backward":
            return {"bytes": n * 2 * (4 if case["through"] else 3) + rows * 8 + width * (2 + 8), "flops": 13 * n}
        eight = case["out"] == "e4m3"
        read = n * 2 * (2 if case["residual"] else 1) + width * 4
        write = n * (1 if eight else 2) + (rows * 4 if eight else 0) + (n * 2 if case["residual"] else 0)
        return {"bytes": read + write + (rows * 8 if case["stats"] else 0), "flops": 8 * n}
    M, N, K = case["M"], case["N"], case["K"]
    bias = N * (2 if op == "linear_int8" else 4) if case["bias"] else 0
    if op == "linear_int8":
        return {"bytes": M * K + K * N + M * N * 2 * (2 if case["residual"] else 1) + (M + N) * 4 + bias, "flops": 2 * M * N * K}
    kept = M * K + M * 4 + (M * N + M * 4 if case["act"] != "none" else 0)
    return {"bytes": M * N * 2 + kept + K * N * 2 + (M * K + K * N) * 2 + bias, "flops": 4 * M * N * K}


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


def _exact_rows(y):
    """8-bit floats of y's rows as the numbers they hold, and the scales."""
    scale = torch.linalg.vector_norm(y, ord=math.inf, dim=1) / E4M3_MAX
    return {"q": torch.div(y, scale.unsqueeze(1)).to(torch.float8_e4m3fn).to(torch.float64), "scale": scale}


def exact(case, seed):
    s = prepare(case, seed)
    wide = {k: v.to(torch.float64) if isinstance(v, torch.Tensor) else v for k, v in s.items()}
    op = case["op"]
    if op == "layer_norm":
        h = wide["x"] if wide["residual"] is None else wide["x"] + wide["residual"]
        variance, mean = torch.var_mean(h, dim=1, correction=0)
        deviation = torch.sqrt(variance + EPS)
        y = torch.addcmul(wide["bias"], wide["weight"], (h - mean.unsqueeze(1)) / deviation.unsqueeze(1))
        out = _exact_rows(y) if case["out"] == "e4m3" else {"y": y}
        if wide["residual"] is not None:
            out["h"] = h
        if case["stats"]:
            out["mean"], out["rstd"] = mean, deviation.reciprocal()
        return out
    if op == "layer_norm_backward":
        h, r, dy, width = wide["x"], wide["rstd"], wide["grad"], case["width"]
        centred = h - wide["mean"].unsqueeze(1)
        g = dy * wide["weight"]
        first, second = g.sum(dim=1) / width, (g * centred).sum(dim=1) * r.pow(2) / width
        dx = (g - first.unsqueeze(1) - centred * second.unsqueeze(1)) * r.unsqueeze(1)
        if wide["through"] is not None:
            dx += wide["through"]
        return {"dx": dx, "dweight": torch.einsum("rw,rw,r->w", dy, centred, r), "dbias": torch.einsum("rw->w", dy)}
    if op == "quantize_rows":
        return _exact_rows(wide["x"])
    if op == "linear_int8":
        x = torch.matmul(wide["A"], wide["B"]) * torch.outer(wide["scale_a"], wide["scale_b"])
        if wide["bias"] is not None:
            x += wide["bias"]
        c = _exact_act(x, case["act"])
        return {"C": c if wide["residual"] is None else c + wide["residual"]}
    A = _exact_act(wide["A"].mul(wide["scale_a"].unsqueeze(1)), case["act_a"])
    D = wide["grad"]
    if case["act"] != "none":
        D = D * _exact_slope(wide["P"].mul(wide["scale_p"].unsqueeze(1)), case["act"])
    out = {"dA": torch.matmul(D, wide["B"].mT), "dB": torch.matmul(A.mT, D)}
    if case["bias"]:
        out["dbias"] = torch.sum(D, 0)
    return out
