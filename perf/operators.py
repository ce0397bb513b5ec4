"""What is measured of the decoder-layer operators: the RMS norm with the
residual's addition, the gated feed-forward product and the linear layer with
bias, activation and residual.

``own`` chooses between the framework's calls and the operators' plain form,
elementary torch operations in 32 bits rounded once at the end.  Types are
named "bf16", "f16", "f32" and "e4m3" (8-bit operands with one fp32 scale per
row).  T: tokens, H: the norm's row width, K: a product's inner size, N: a
linear layer's outputs, n: a gated layer's outputs (its weight has 2n rows,
gate then up).
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32,
       "e4m3": torch.float8_e4m3fn}
_SIZE = {"bf16": 2, "f16": 2, "f32": 4, "e4m3": 1}
_EPS = 1e-5


def listed():
    return [
        # one generated token: the norm before a layer's MLP, residual stream updated
        {"name": "norm-1-bf16", "op": "norm_fwd", "dtype": "bf16", "T": 1, "H": 4096, "quant": False},
        # a training batch's norm at the hidden size of the fused linear CE workload, feeding 8-bit products
        {"name": "norm-8192-bf16-e4m3", "op": "norm_fwd", "dtype": "bf16", "T": 8192, "H": 6656, "quant": True},
        # the same norm's backward, the residual stream's gradient joining it
        {"name": "normbwd-8192-bf16", "op": "norm_bwd", "dtype": "bf16", "T": 8192, "H": 6656},
        # fp32 with a row width that no vector load divides, a ragged number of rows
        {"name": "normbwd-333-f32-odd", "op": "norm_bwd", "dtype": "f32", "T": 333, "H": 1001},
        # one generated token through the gated layer: the weights are read once
        {"name": "glu-1-bf16", "op": "glu_fwd", "dtype": "bf16", "act": "silu", "T": 1, "K": 4096, "n": 12288,
         "preact": False},
        # a serving batch between the one-token and the training sizes, 8-bit operands
        {"name": "glu-300-e4m3", "op": "glu_fwd", "dtype": "e4m3", "act": "silu", "T": 300, "K": 4096, "n": 10240,
         "preact": False},
        # the training batch of the fused linear CE workload, the pre-activations kept for the backward pass
        {"name": "glu-4096-bf16", "op": "glu_fwd", "dtype": "bf16", "act": "silu", "T": 4096, "K": 6656, "n": 16384,
         "preact": True},
        # its backward pass
        {"name": "glubwd-4096-bf16", "op": "glu_bwd", "dtype": "bf16", "act": "silu", "T": 4096, "K": 6656,
         "n": 16384},
        # a serving batch through the layer that closes the MLP, added to the residual stream, 8-bit operands
        {"name": "linear-64-e4m3-res", "op": "linear_fwd", "dtype": "e4m3", "act": "none", "T": 64, "K": 16384,
         "N": 6656, "bias": False, "residual": True, "preact": False},
        # ragged everything, fp16: bias and gelu, pre-activations kept
        {"name": "linear-1007-f16-gelu", "op": "linear_fwd", "dtype": "f16", "act": "gelu", "T": 1007, "K": 1000,
         "N": 777, "bias": True, "residual": False, "preact": True},
        # a prompt's closing layer: bias and residual in the epilogue
        {"name": "linear-8192-bf16-res", "op": "linear_fwd", "dtype": "bf16", "act": "none", "T": 8192, "K": 16384,
         "N": 4096, "bias": True, "residual": True, "preact": False},
        # backward of a linear layer with a gelu and a bias
        {"name": "linearbwd-2048-bf16", "op": "linear_bwd", "dtype": "bf16", "act": "gelu_tanh", "T": 2048, "K": 4096,
         "N": 16384, "bias": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    most = max(work(c)["flops"] for c in listed())
    while True:
        op = rng.choice(["norm_fwd", "norm_bwd", "glu_fwd", "glu_bwd", "linear_fwd", "linear_bwd"])
        T = _log(rng, 1, 8192)
        if op in ("norm_fwd", "norm_bwd"):
            c = {"op": op, "dtype": rng.choice(["bf16", "f16", "f32"]), "T": T, "H": _log(rng, 100, 8192)}
            if op == "norm_fwd":
                c["quant"] = rng.random() < 0.4
            return c
        # rows of the operands of a product are whole 16-byte units
        dtype = rng.choice(["bf16", "f16", "e4m3"] if op.endswith("fwd") else ["bf16", "f16"])
        K = 16 * _log(rng, 16, 1024) if dtype == "e4m3" else 8 * _log(rng, 32, 2048)
        c = {"op": op, "dtype": dtype, "T": T, "K": K}
        if op.startswith("glu"):
            c["act"] = rng.choice(["silu", "gelu", "gelu_tanh", "relu"])
            c["n"] = _log(rng, 100, 16384)
            if op == "glu_fwd":
                c["preact"] = dtype != "e4m3" and rng.random() < 0.5
        else:
            c["act"] = rng.choice(["none", "silu", "gelu", "gelu_tanh", "relu"])
            c["N"] = _log(rng, 100, 16384)
            c["bias"] = rng.random() < 0.5
            if op == "linear_fwd":
                c["residual"] = rng.random() < 0.5
                c["preact"] = dtype != "e4m3" and c["act"] != "none" and rng.random() < 0.5
        if work(c)["flops"] <= most:
            return c


def _operand(g, dev, rows, cols, dtype, sigma):
    """A matrix of rows ~ N(0, sigma^2) and, in e4m3, its rows' scales max / 448."""
    v = torch.randn((rows, cols), generator=g, device=dev) * sigma
    if dtype != "e4m3":
        return v.to(_DT[dtype]), None
    scale = v.abs().amax(dim=1) / 448.0
    return (v / scale[:, None]).to(torch.float8_e4m3fn), scale


def _outputs(case):
    return case["n"] if case["op"].startswith("glu") else case["N"]


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def randn(*shape, sigma=1.0, dt=None):
        return (torch.randn(shape, generator=g, device=dev) * sigma).to(dt or _DT[case["dtype"]])

    s = {"case": case}
    op, T = case["op"], case["T"]
    if op in ("norm_fwd", "norm_bwd"):
        H = case["H"]
        s["weight"] = 1 + randn(H, sigma=0.1)
        if op == "norm_fwd":
            s["x"], s["residual"] = randn(T, H), randn(T, H, sigma=3.0)
        else:
            s["x"] = randn(T, H, sigma=3.0)  # the stored sum
            s["rstd"] = (s["x"].float().square().mean(dim=1) + _EPS).rsqrt()
            s["dy"], s["dresidual"] = randn(T, H, sigma=0.1), randn(T, H, sigma=0.1)
        return s
    K, m = case["K"], _outputs(case)
    rows = 2 * m if op.startswith("glu") else m
    s["x"], s["x_scale"] = _operand(g, dev, T, K, case["dtype"], 1.0)
    s["weight"], s["weight_scale"] = _operand(g, dev, rows, K, case["dtype"], K ** -0.5)
    wide = torch.bfloat16 if case["dtype"] == "e4m3" else _DT[case["dtype"]]  # the type of everything else
    s["bias"] = randn(m, sigma=0.5, dt=wide) if case.get("bias") else None
    s["residual"] = randn(T, m, sigma=2.0, dt=wide) if case.get("residual") else None
    if op.endswith("bwd"):
        s["dy"] = randn(T, m, sigma=0.1)
        s["preact"] = randn(T, rows) if op == "glu_bwd" or case["act"] != "none" else None
    return s


# ---------------------------------------------------------------- the framework's calls
def _run_own(s):
    import vocabulary_lm_cross_gb300 as v

    case = s["case"]
    op = case["op"]
    if op == "norm_fwd":
        r = v.rmsnorm_fwd(s["x"], s["weight"], s["residual"], eps=_EPS, fp8=case["quant"])
        out = {"y": r.y, "residual": r.residual, "rstd": r.rstd}
        if case["quant"]:
            out["scale"] = r.scale
        return out
    if op == "norm_bwd":
        r = v.rmsnorm_bwd(s["dy"], s["x"], s["weight"], s["rstd"], dresidual=s["dresidual"])
        return {"dx": r.dx, "dweight": r.dweight}
    if op == "glu_fwd":
        r = v.glu_fwd(s["x"], s["weight"], act=case["act"], preact=case["preact"], x_scale=s["x_scale"],
                      weight_scale=s["weight_scale"])
        return {"y": r.y, "preact": r.preact} if case["preact"] else {"y": r.y}
    if op == "linear_fwd":
        r = v.linear_fwd(s["x"], s["weight"], s["bias"], s["residual"], act=case["act"], preact=case["preact"],
                         x_scale=s["x_scale"], weight_scale=s["weight_scale"])
        return {"y": r.y, "preact": r.preact} if case["preact"] else {"y": r.y}
    if op == "glu_bwd":
        r = v.glu_bwd(s["dy"], s["x"], s["weight"], s["preact"], act=case["act"],
                      dweight_dtype=s["weight"].dtype)
        return {"dx": r.dx, "dweight": r.dweight}
    r = v.linear_bwd(s["dy"], s["x"], s["weight"], s["preact"], act=case["act"], bias_grad=case["bias"],
                     dweight_dtype=s["weight"].dtype)
    out = {"dx": r.dx, "dweight": r.dweight}
    if case["bias"]:
        out["dbias"] = r.dbias
    return out


# ---------------------------------------------------------------- the plain form
_C0, _C1 = math.sqrt(2.0 / math.pi), 0.044715


def _act(a, act):
    if act == "none":
        return a
    if act == "silu":
        return a * torch.sigmoid(a)
    if act == "gelu":
        return 0.5 * a * (1 + torch.erf(a * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * a * (1 + torch.tanh(_C0 * (a + _C1 * a * a * a)))
    return torch.clamp(a, min=0)


def _dact(a, act):
    if act == "silu":
        q = torch.sigmoid(a)
        return q * (1 + a * (1 - q))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(a * math.sqrt(0.5))) + a * torch.exp(-0.5 * a * a) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        t = torch.tanh(_C0 * (a + _C1 * a * a * a))
        return 0.5 * (1 + t) + 0.5 * a * (1 - t * t) * _C0 * (1 + 3 * _C1 * a * a)
    return (a > 0).to(a.dtype)


def _wide(v, scale):
    v = v.float()
    return v if scale is None else v * scale[:, None]


def _run_plain(s):
    case = s["case"]
    op, x = case["op"], s["x"]
    if op == "norm_fwd":
        v = x.float() + s["residual"].float()
        rstd = torch.rsqrt((v * v).mean(dim=1) + _EPS)
        y = v * rstd[:, None] * s["weight"].float()
        out = {"residual": v.to(x.dtype), "rstd": rstd}
        if case["quant"]:
            out["scale"] = y.abs().amax(dim=1) / 448.0
            out["y"] = (y / out["scale"][:, None]).to(torch.float8_e4m3fn)
        else:
            out["y"] = y.to(x.dtype)
        return out
    if op == "norm_bwd":
        dy = s["dy"].float()
        xhat = x.float() * s["rstd"][:, None]
        gw = dy * s["weight"].float()
        dx = (gw - xhat * (gw * xhat).mean(dim=1, keepdim=True)) * s["rstd"][:, None] + s["dresidual"].float()
        return {"dx": dx.to(x.dtype), "dweight": (dy * xhat).sum(dim=0)}
    xf, w = _wide(x, s["x_scale"]), _wide(s["weight"], s["weight_scale"])
    wide = torch.bfloat16 if case["dtype"] == "e4m3" else x.dtype
    if op == "glu_fwd":
        z = xf @ w.t()
        out = {"y": (_act(z[:, :case["n"]], case["act"]) * z[:, case["n"]:]).to(wide)}
        if case["preact"]:
            out["preact"] = z.to(wide)
        return out
    if op == "linear_fwd":
        z = xf @ w.t()
        if s["bias"] is not None:
            z = z + s["bias"].float()
        y = _act(z, case["act"])
        if s["residual"] is not None:
            y = y + s["residual"].float()
        out = {"y": y.to(wide)}
        if case["preact"]:
            out["preact"] = z.to(wide)
        return out
    dy = s["dy"].float()
    if op == "glu_bwd":
        z = s["preact"].float()
        a, u = z[:, :case["n"]], z[:, case["n"]:]
        dz = torch.cat([dy * u * _dact(a, case["act"]), dy * _act(a, case["act"])], dim=1)
    else:
        dz = dy if case["act"] == "none" else dy * _dact(s["preact"].float(), case["act"])
    out = {"dx": (dz @ w).to(wide), "dweight": (dz.t() @ xf).to(wide)}
    if op == "linear_bwd" and case["bias"]:
        out["dbias"] = dz.sum(dim=0)
    return out


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------- work and the 64-bit values
def work(case):
    op, T, e = case["op"], case["T"], _SIZE[case["dtype"]]
    if op == "norm_fwd":
        H = case["H"]
        q = 1 if case["quant"] else e
        return {"bytes": T * H * (3 * e + q) + H * e + T * (8 if case["quant"] else 4), "flops": 6 * T * H}
    if op == "norm_bwd":
        H = case["H"]
        return {"bytes": 4 * T * H * e + H * (e + 4) + 4 * T, "flops": 10 * T * H}
    K, m = case["K"], _outputs(case)
    rows = 2 * m if op.startswith("glu") else m
    o = 2  # bytes of an output value
    if op.endswith("fwd"):
        b = (T + rows) * K * e + T * m * o
        if case["dtype"] == "e4m3":
            b += 4 * (T + rows)
        if case["preact"]:
            b += T * rows * o
        if case.get("residual"):
            b += T * m * o
        if case.get("bias"):
            b += m * o
        return {"bytes": b, "flops": 2 * T * K * rows}
    b = 2 * (T + rows) * K * e + T * m * e
    if case["act"] != "none":
        b += T * rows * e
    if case.get("bias"):
        b += 4 * m
    return {"bytes": b, "flops": 4 * T * K * rows}


def _gate64(a, act):
    """(act(a), act'(a)) in 64 bits."""
    one = torch.ones_like(a)
    if act == "none":
        return a, one
    if act == "relu":
        return torch.where(a > 0, a, 0 * one), torch.where(a > 0, one, 0 * one)
    if act == "silu":
        q = torch.special.expit(a)
        return a * q, q + a * q * torch.special.expit(-a)
    if act == "gelu":
        cdf = torch.special.ndtr(a)
        return a * cdf, cdf + a * torch.exp(-a * a / 2) * (2 * math.pi) ** -0.5
    inner = 2 * _C0 * a * (1 + _C1 * a ** 2)  # (1 + tanh(v)) / 2 = expit(2 v)
    q = torch.special.expit(inner)
    return a * q, q + a * q * torch.special.expit(-inner) * 2 * _C0 * (1 + 3 * _C1 * a ** 2)


def exact(case, seed):
    s = prepare(case, seed)
    d = {k: (v.to(torch.float64) if isinstance(v, torch.Tensor) else v) for k, v in s.items()}
    op = case["op"]
    if op == "norm_fwd":
        h = d["residual"] + d["x"]
        inv = 1 / torch.sqrt(torch.linalg.vector_norm(h, dim=1) ** 2 / case["H"] + _EPS)
        y = torch.einsum("th,t,h->th", h, inv, d["weight"])
        out = {"y": y, "residual": h, "rstd": inv}
        if case["quant"]:
            out["scale"] = torch.linalg.vector_norm(y, ord=math.inf, dim=1) / 448
            out["y"] = y / out["scale"].unsqueeze(1)
        return out
    if op == "norm_bwd":
        inv = d["rstd"].unsqueeze(1)
        h, up = d["x"], d["dy"] * d["weight"]
        along = torch.linalg.vecdot(up, h).unsqueeze(1) / case["H"]
        return {"dx": d["dresidual"] + inv * up - inv ** 3 * along * h,
                "dweight": torch.einsum("th,th,t->h", d["dy"], h, d["rstd"])}
    x, w = d["x"], d["weight"]
    if d["x_scale"] is not None:
        x, w = torch.diag_embed(d["x_scale"]) @ x if x.shape[0] < 512 else x * d["x_scale"].unsqueeze(1), \
            w * d["weight_scale"].unsqueeze(1)
    if op.endswith("fwd"):
        z = torch.nn.functional.linear(x, w, d["bias"])
        if op == "glu_fwd":
            gate, up = z.chunk(2, dim=1)
            y = _gate64(gate, case["act"])[0] * up
        else:
            y = _gate64(z, case["act"])[0]
            if d["residual"] is not None:
                y = y + d["residual"]
        return {"y": y, "preact": z} if case["preact"] else {"y": y}
    if op == "glu_bwd":
        gate, up = d["preact"].chunk(2, dim=1)
        f, df = _gate64(gate, case["act"])
        dz = torch.hstack([d["dy"] * df * up, d["dy"] * f])
    else:
        dz = d["dy"] * (_gate64(d["preact"], case["act"])[1] if d["preact"] is not None else 1.0)
    out = {"dx": torch.einsum("tm,mk->tk", dz, w), "dweight": torch.einsum("tm,tk->mk", dz, x)}
    if op == "linear_bwd" and case["bias"]:
        out["dbias"] = torch.einsum("tm->m", dz)
    return out
