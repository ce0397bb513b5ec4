"""What is measured of the experts' operators: tokens sorted by expert and brought
back with weights, quantisation to e4m3 by blocks of 128, and the product of
operands quantised so, dense and by experts.

``own`` chooses between the framework's calls and the operators' plain form,
elementary torch operations in 32 bits rounded once at the end.  T: tokens, k:
experts of a token, E: experts, H: a row's width, R: rows, K: a product's inner
size, N: its outputs.  A block is 128 values along the inner size (and, of a
weight, 128 rows too) that share one fp32 scale.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f16": 2, "f32": 4}
_B = 128
_TINY = 2.0 ** -100  # the least maximum that a block is scaled by


def listed():
    return [
        # a serving batch of 64 tokens, each to 8 of 128 experts
        {"name": "sort-64x8", "op": "sort", "T": 64, "k": 8, "E": 128, "align": 1, "dropped": False, "wide": True},
        # a training batch; experts' rows start at multiples of 128 for the weights' gradient
        {"name": "sort-16384x8", "op": "sort", "T": 16384, "k": 8, "E": 256, "align": 128, "dropped": False,
         "wide": False},
        # a training batch to its experts' rows, quantised on the way
        {"name": "gather-8192x4-bf16-e4m3", "op": "gather", "dtype": "bf16", "T": 8192, "k": 4, "E": 64, "H": 4096,
         "fp8": True},
        # the gradient of a gather, fp16, at a width that no vector load divides
        {"name": "gatherbwd-1007x3-f16-odd", "op": "gather_bwd", "dtype": "f16", "T": 1007, "k": 3, "E": 16,
         "H": 1001},
        # a few generated tokens brought back with their weights, added to the residual stream
        {"name": "combine-16x8-bf16-res", "op": "combine", "dtype": "bf16", "T": 16, "k": 8, "E": 64, "H": 4096,
         "residual": True, "dropped": False},
        # its gradient in a training batch: the experts' rows and the weights
        {"name": "combinebwd-8192x4-bf16", "op": "combine_bwd", "dtype": "bf16", "T": 8192, "k": 4, "E": 64,
         "H": 4096},
        # a training batch's activations (the hidden size of the fused linear CE workload): for the forward product,
        # and transposed for the weight's gradient
        {"name": "quant-8192-bf16-both", "op": "quantize", "dtype": "bf16", "R": 8192, "C": 6656, "square": False,
         "rows": True, "transposed": True},
        # an fp32 master weight of odd sizes in 128 x 128 blocks
        {"name": "quant-1001-f32-square", "op": "quantize", "dtype": "f32", "R": 1001, "C": 2000, "square": True,
         "rows": True, "transposed": True},
        # one generated token through a dense projection: the weight is read once
        {"name": "product-1", "op": "product", "T": 1, "K": 4096, "N": 12288, "by_row": False, "residual": True,
         "out": "bf16"},
        # a serving batch of 64 tokens, each through 8 of 32 experts: about 16 rows an expert
        {"name": "experts-64x8", "op": "experts", "T": 64, "k": 8, "E": 32, "K": 4096, "N": 4096, "out": "bf16"},
        # a training batch of 8192 tokens, each through 2 of 16 experts
        {"name": "experts-8192x2", "op": "experts", "T": 8192, "k": 2, "E": 16, "K": 4096, "N": 4096, "out": "bf16"},
        # the gradient of those experts' second weight
        {"name": "dweight-8192x2", "op": "dweight", "T": 8192, "k": 2, "E": 16, "K": 2048, "N": 4096, "out": "f32"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    most = {"flops": max(work(c)["flops"] for c in listed()), "bytes": max(work(c)["bytes"] for c in listed())}
    while True:
        op = rng.choice(["sort", "gather", "gather_bwd", "combine", "combine_bwd", "quantize", "product", "experts",
                         "experts", "dweight"])
        if op == "product":
            c = {"op": op, "T": _log(rng, 1, 8192), "K": 16 * _log(rng, 8, 1024), "N": _log(rng, 100, 16384),
                 "by_row": rng.random() < 0.25, "residual": rng.random() < 0.5, "out": rng.choice(["bf16", "f16"])}
        elif op == "quantize":
            c = {"op": op, "dtype": rng.choice(["bf16", "f16", "f32"]), "R": _log(rng, 1, 8192),
                 "C": _log(rng, 64, 8192), "square": rng.random() < 0.3}
            c["rows"], c["transposed"] = rng.choice([(True, False), (True, True), (False, True)])
        else:
            E = _log(rng, 4, 256)
            c = {"op": op, "T": _log(rng, 1, 16384 if op == "sort" else 8192), "k": rng.randint(1, min(8, E)), "E": E}
            if op == "sort":
                c.update(align=rng.choice([1, 16, 128]), dropped=rng.random() < 0.3, wide=rng.random() < 0.5)
            elif op in ("experts", "dweight"):
                c.update(K=16 * _log(rng, 8, 512), N=_log(rng, 100, 8192),
                         out="f32" if op == "dweight" else rng.choice(["bf16", "f16"]))
            else:
                c.update(dtype=rng.choice(["bf16", "f16", "f32"]), H=_log(rng, 100, 8192))
                if op == "gather":
                    c["fp8"] = rng.random() < 0.5
                elif op == "combine":
                    c.update(residual=rng.random() < 0.5, dropped=rng.random() < 0.3)
        w = work(c)
        if w["flops"] <= most["flops"] and w["bytes"] <= most["bytes"]:
            return c


# ---------------------------------------------------------------- inputs
def _experts(g, dev, case):
    """[T, k] distinct experts a token, some more popular than others; -1: dropped."""
    T, k, E = case["T"], case["k"], case["E"]
    favour = torch.randn(E, generator=g, device=dev) * 0.5
    noise = -torch.log(-torch.log(torch.rand((T, E), generator=g, device=dev).clamp(1e-7, 1 - 1e-7)))
    ids = torch.topk(favour + noise, k, dim=1).indices
    if case.get("dropped"):
        ids = torch.where(torch.rand((T, k), generator=g, device=dev) < 0.2, -1, ids)
    return ids


def _capacity(T, k, E, align):
    """Rows that any routing of T tokens fits in."""
    n = T * k + min(E, T * k) * (align - 1)
    return n // align * align


def _order(ids, E, align):
    """position [T, k], offsets [E + 1], counts [E] of a routing, in 32-bit integers."""
    flat = ids.reshape(-1).long()
    key = torch.where(flat < 0, E, flat)
    counts = torch.zeros(E + 1, dtype=torch.int64, device=ids.device).scatter_add_(0, key, torch.ones_like(key))
    counts[E] = 0
    padded = (counts + align - 1) // align * align
    start = torch.cumsum(padded, 0) - padded          # start[E]: the end of the rows in use
    order = torch.argsort(key, stable=True)
    first = torch.cumsum(torch.bincount(key, minlength=E + 1), 0) - torch.bincount(key, minlength=E + 1)
    rank = torch.empty_like(key)
    rank[order] = torch.arange(key.numel(), device=ids.device) - first[key[order]]
    position = torch.where(flat < 0, -1, start[key] + rank)
    return position.reshape(ids.shape).int(), start.int(), counts[:E].int()


def _blocks(v):
    """v [R, C] to e4m3 by blocks of 128 columns: (q, scale [R, C / 128])."""
    R, C = v.shape
    pad = -C % _B
    w = torch.nn.functional.pad(v, (0, pad)).reshape(R, -1, _B)
    amax = w.abs().amax(dim=2).clamp(min=_TINY)
    q = (w * (448.0 / amax)[:, :, None]).to(torch.float8_e4m3fn)
    return _pitched(q.reshape(R, -1)[:, :C]), amax / 448.0


def _square(v):
    """v [R, C] to e4m3 by blocks of 128 x 128: (q, scale [R / 128, C / 128])."""
    R, C = v.shape
    w = torch.nn.functional.pad(v, (0, -C % _B, 0, -R % _B))
    w = w.reshape(w.shape[0] // _B, _B, w.shape[1] // _B, _B)
    amax = w.abs().amax(dim=(1, 3)).clamp(min=_TINY)
    q = (w * (448.0 / amax)[:, None, :, None]).to(torch.float8_e4m3fn)
    return _pitched(q.reshape(q.shape[0] * _B, -1)[:R, :C]), amax / 448.0


def _pitched(q):
    """The same values in rows of whole 16-byte units."""
    out = torch.zeros((q.shape[0], q.shape[1] + -q.shape[1] % 16), dtype=q.dtype, device=q.device)
    out[:, :q.shape[1]] = q
    return out[:, :q.shape[1]]


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def randn(*shape, sigma=1.0, dt=None):
        return (torch.randn(shape, generator=g, device=dev) * sigma).to(dt or _DT[case.get("dtype", "f32")])

    s = {"case": case}
    op = case["op"]
    if op == "quantize":
        # rows of unlike sizes, as activations have them
        s["x"] = (randn(case["R"], case["C"]).float() * torch.exp(randn(case["R"], 1).float())).to(_DT[case["dtype"]])
        return s
    if op == "product":
        s["x"], s["x_scale"] = _blocks(randn(case["T"], case["K"]))
        s["weight"], s["weight_scale"] = (_blocks if case["by_row"] else _square)(
            randn(case["N"], case["K"], sigma=case["K"] ** -0.5))
        s["residual"] = randn(case["T"], case["N"], dt=_DT[case["out"]]) if case["residual"] else None
        return s
    T, k, E = case["T"], case["k"], case["E"]
    ids = _experts(g, dev, case)
    if op == "sort":
        s["experts"] = ids if case["wide"] else ids.int()
        return s
    align = _B if op == "dweight" else 1
    s["position"], s["offsets"], s["counts"] = _order(ids, E, align)
    R = s["rows"] = _capacity(T, k, E, align)
    if op in ("experts", "dweight"):
        s["host_offsets"] = s["offsets"].tolist()
        K, N = case["K"], case["N"]
        if op == "experts":
            s["x"], s["x_scale"] = _blocks(randn(R, K))
            s["weight"] = torch.empty((E, N, K), dtype=torch.float8_e4m3fn, device=dev)
            s["weight_scale"] = torch.empty((E, -(-N // _B), -(-K // _B)), device=dev)
            for e in range(E):
                s["weight"][e], s["weight_scale"][e] = _square(randn(N, K, sigma=K ** -0.5))
            return s
        held = torch.zeros(R, device=dev)
        held[s["position"].reshape(-1).long()] = 1.0  # the rows between the experts' are zero
        s["dyt"], s["dyt_scale"] = _blocks(randn(N, R, sigma=0.1) * held)
        s["xt"], s["xt_scale"] = _blocks(randn(K, R) * held)
        return s
    H = case["H"]
    if op == "gather":
        s["x"] = randn(T, H)
        return s
    s["data"] = randn(R, H)  # the experts' rows, or their gradient
    if op.startswith("combine"):
        w = torch.rand((T, k), generator=g, device=dev) + 0.1
        s["weights"] = w / w.sum(dim=1, keepdim=True)
        s["residual"] = randn(T, H, sigma=3.0) if case.get("residual") else None
        s["dy"] = randn(T, H, sigma=0.1) if op == "combine_bwd" else None
    return s


# ---------------------------------------------------------------- the framework's calls
def _run_own(s):
    import vocabulary_lm_cross_gb300 as v

    case = s["case"]
    op = case["op"]
    if op == "sort":
        r = v.moe_sort(s["experts"], case["E"], align=case["align"])
        return {"position": r.position, "offsets": r.offsets, "counts": r.counts}
    if op == "quantize":
        r = v.quantize_blocks(s["x"], square=case["square"], rows=case["rows"], transposed=case["transposed"])
        out = {}
        if case["rows"]:
            out.update(q=r.q, scale=r.scale)
        if case["transposed"]:
            out.update(qt=r.qt, scale_t=r.scale_t)
        return out
    if op == "product":
        return v.block_linear_fwd(s["x"], s["x_scale"], s["weight"], s["weight_scale"], s["residual"],
                                  out_dtype=_DT[case["out"]])
    if op == "experts":
        return v.block_linear_fwd(s["x"], s["x_scale"], s["weight"], s["weight_scale"], offsets=s["offsets"],
                                  out_dtype=_DT[case["out"]])
    if op == "dweight":
        return v.block_linear_dweight(s["dyt"], s["dyt_scale"], s["xt"], s["xt_scale"], offsets=s["offsets"])
    order = v.MoEOrder(s["position"], s["offsets"], s["counts"], s["rows"])
    if op == "gather":
        r = v.moe_gather(s["x"], order, fp8=case["fp8"])
        return {"rows": r.rows, "scale": r.scale} if case["fp8"] else {"rows": r.rows}
    if op == "gather_bwd":
        return v.moe_gather_bwd(s["data"], order)
    if op == "combine":
        return v.moe_combine(s["data"], order, s["weights"], s["residual"])
    r = v.moe_combine_bwd(s["dy"], s["data"], order, s["weights"])
    return {"drows": r.drows, "dweights": r.dweights}


# ---------------------------------------------------------------- the plain form
def _widen(q, scale, by_row=True):
    """The values a quantised matrix stands for, in fp32."""
    f = scale.repeat_interleave(_B, dim=-1)[..., :q.shape[-1]]
    if not by_row:
        f = f.repeat_interleave(_B, dim=-2)[..., :q.shape[-2], :]
    return q.float() * f


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    if op == "sort":
        p, o, c = _order(s["experts"], case["E"], case["align"])
        return {"position": p, "offsets": o, "counts": c}
    if op == "quantize":
        x = s["x"].float()
        out = {}
        if case["square"]:
            q, scale = _square(x)
            if case["rows"]:
                out.update(q=q, scale=scale)
            if case["transposed"]:
                out.update(qt=q.t().contiguous(), scale_t=scale.t().contiguous())
            return out
        if case["rows"]:
            out["q"], out["scale"] = _blocks(x)
        if case["transposed"]:
            out["qt"], out["scale_t"] = _blocks(x.t())
        return out
    if op == "product":
        y = _widen(s["x"], s["x_scale"]) @ _widen(s["weight"], s["weight_scale"], case["by_row"]).t()
        if s["residual"] is not None:
            y = y + s["residual"].float()
        return y.to(_DT[case["out"]])
    if op == "experts":
        y = torch.empty((s["rows"], case["N"]), dtype=_DT[case["out"]], device=s["x"].device)
        at = s["host_offsets"]
        for e in range(case["E"]):
            a, b = at[e], at[e + 1]
            if b > a:
                y[a:b] = _widen(s["x"][a:b], s["x_scale"][a:b]) @ \
                    _widen(s["weight"][e], s["weight_scale"][e], False).t()
        return y
    if op == "dweight":
        out = torch.zeros((case["E"], case["N"], case["K"]), device=s["xt"].device)
        at = s["host_offsets"]
        for e in range(case["E"]):
            a, b = at[e], at[e + 1]
            if b > a:
                f = slice(a // _B, b // _B)
                out[e] = _widen(s["dyt"][:, a:b], s["dyt_scale"][:, f]) @ _widen(s["xt"][:, a:b], s["xt_scale"][:, f]).t()
        return out
    at = s["position"].reshape(-1).long()
    if op == "gather":
        rows = torch.empty((s["rows"], case["H"]), device=at.device)
        rows[at] = s["x"].float().repeat_interleave(case["k"], dim=0)
        if case["fp8"]:
            q, scale = _blocks(rows)
            return {"rows": q, "scale": scale}
        return {"rows": rows.to(s["x"].dtype)}
    T, k, H = case["T"], case["k"], case["H"]
    held = (at >= 0).float()[:, None]
    rows = (s["data"][at.clamp(min=0)].float() * held).reshape(T, k, H)
    if op == "gather_bwd":
        return rows.sum(dim=1).to(s["data"].dtype)
    if op == "combine":
        y = (rows * s["weights"][:, :, None]).sum(dim=1)
        if s["residual"] is not None:
            y = y + s["residual"].float()
        return y.to(s["data"].dtype)
    dy = s["dy"].float()
    each = (dy[:, None, :] * s["weights"][:, :, None]).reshape(T * k, H)
    drows = torch.zeros((s["rows"], H), device=at.device)
    drows[at] = each
    return {"drows": drows.to(s["data"].dtype), "dweights": (rows * dy[:, None, :]).sum(dim=2)}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------- work and the 64-bit values
def work(case):
    op = case["op"]
    if op == "quantize":
        R, C = case["R"], case["C"]
        n = case["rows"] + case["transposed"]
        return {"bytes": R * C * (_SIZE[case["dtype"]] + n) + n * 4 * R * C // (_B * (_B if case["square"] else 1)),
                "flops": 3 * R * C * n}
    if op == "product":
        T, K, N = case["T"], case["K"], case["N"]
        scales = 4 * (T + (N if case["by_row"] else N / _B)) * K / _B
        return {"bytes": int((T + N) * K + scales + 2 * T * N * (2 if case["residual"] else 1)), "flops": 2 * T * K * N}
    T, k, E = case["T"], case["k"], case["E"]
    R = T * k
    if op == "sort":
        return {"bytes": R * ((8 if case["wide"] else 4) + 4) + 4 * (2 * E + 1), "flops": R}
    if op == "experts":
        K, N = case["K"], case["N"]
        used = min(E, R)  # experts that have rows, at most
        return {"bytes": int((R + used * N) * K * (1 + 4 / _B) + 2 * R * N), "flops": 2 * R * K * N}
    if op == "dweight":
        K, N = case["K"], case["N"]
        return {"bytes": int(R * (K + N) * (1 + 4 / _B) + 4 * E * K * N), "flops": 2 * R * K * N}
    H, e = case["H"], _SIZE[case["dtype"]]
    if op == "gather":
        out = R * H * (1 + 4 / _B) if case["fp8"] else R * H * e
        return {"bytes": int(T * H * e + out + 4 * R), "flops": 3 * T * H if case["fp8"] else T * H}
    if op == "gather_bwd":
        return {"bytes": (T + R) * H * e + 4 * R, "flops": R * H}
    if op == "combine":
        return {"bytes": (T * (2 if case["residual"] else 1) + R) * H * e + 8 * R, "flops": 2 * R * H}
    return {"bytes": (T + 2 * R) * H * e + 12 * R, "flops": 3 * R * H}


def _exact_blocks(x, rows, cols):
    """Blocks of rows x cols of a 64-bit matrix: (values over scale, scale)."""
    R, C = x.shape
    scale = torch.nn.functional.max_pool2d(x.abs()[None], (rows, cols), ceil_mode=True)[0].clamp(min=_TINY) / 448
    i = torch.arange(R, device=x.device) // rows
    j = torch.arange(C, device=x.device) // cols
    return x / scale[i[:, None], j[None, :]], scale


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "sort":
        ids = s["experts"].cpu().tolist()
        where, counts = [], [0] * case["E"]
        for row in ids:
            where.append([])
            for e in row:
                where[-1].append(counts[e] if e >= 0 else None)
                if e >= 0:
                    counts[e] += 1
        start = [0]
        for c in counts:
            start.append(start[-1] + -(-c // case["align"]) * case["align"])
        pos = [[-1 if r is None else start[e] + r for e, r in zip(row, rk)] for row, rk in zip(ids, where)]
        dev = s["experts"].device
        return {"position": torch.tensor(pos, dtype=torch.int32, device=dev),
                "offsets": torch.tensor(start, dtype=torch.int32, device=dev),
                "counts": torch.tensor(counts, dtype=torch.int32, device=dev)}
    d = {n: (t.to(torch.float64) if isinstance(t, torch.Tensor) and t.dtype in
             (torch.float32, torch.float16, torch.bfloat16, torch.float8_e4m3fn) else t) for n, t in s.items()}
    if op == "quantize":
        out = {}
        if case["rows"]:
            out["q"], out["scale"] = _exact_blocks(d["x"], _B if case["square"] else 1, _B)
        if case["transposed"]:
            q, scale = _exact_blocks(d["x"], _B, _B if case["square"] else 1)
            out["qt"], out["scale_t"] = q.t().contiguous(), scale.t().contiguous()
        return out

    def split(a, blocks):  # [rows, K] -> [rows, blocks, 128]
        return torch.nn.functional.pad(a, (0, blocks * _B - a.shape[1])).unflatten(1, (blocks, _B))

    def product(a, fa, b, fb):  # factors fa [rows of a, blocks], fb [rows of b, blocks]
        n = fa.shape[1]
        return torch.einsum("tbk,tb,nbk->tn", split(a, n), fa, split(b, n) * fb[:, :, None])

    def per_row(f, rows):  # one factor for 128 rows -> one for each
        return f[torch.arange(rows, device=f.device) // _B]

    if op == "product":
        f = d["weight_scale"] if case["by_row"] else per_row(d["weight_scale"], case["N"])
        y = product(d["x"], d["x_scale"], d["weight"], f)
        return y if d["residual"] is None else y + d["residual"]
    if op in ("experts", "dweight"):
        at = s["host_offsets"]
        parts = []
        for e in range(case["E"]):
            rows = slice(at[e], at[e + 1])
            if op == "experts":
                parts.append(product(d["x"][rows], d["x_scale"][rows], d["weight"][e],
                                     per_row(d["weight_scale"][e], case["N"])))
            else:
                b = slice(at[e] // _B, at[e + 1] // _B)
                parts.append(product(d["dyt"][:, rows], d["dyt_scale"][:, b], d["xt"][:, rows], d["xt_scale"][:, b]))
        return torch.cat(parts) if op == "experts" else torch.stack(parts)
    at = s["position"].long()
    held = at >= 0
    R, H = s["rows"], case["H"]
    if op == "gather":
        rows = d["x"].new_zeros((R, H)).index_put_((at[held],), d["x"][held.nonzero()[:, 0]])
        if case["fp8"]:
            q, scale = _exact_blocks(rows, 1, _B)
            return {"rows": q, "scale": scale}
        return {"rows": rows}
    T, k = at.shape
    token, slot = held.nonzero(as_tuple=True)
    w = d["weights"] if op.startswith("combine") else torch.ones((T, k), dtype=torch.float64, device=at.device)
    rows = d["data"][at[held]]
    if op == "combine_bwd":
        up = d["dy"][token]
        dw = torch.zeros((T, k), dtype=torch.float64, device=at.device)
        dw[token, slot] = torch.linalg.vecdot(rows, up)
        drows = d["data"].new_zeros((R, H))
        drows[at[held]] = w[token, slot].unsqueeze(1) * up
        return {"drows": drows, "dweights": dw}
    y = d["data"].new_zeros((T, H)).index_add_(0, token, rows * w[token, slot].unsqueeze(1))
    return y + d["residual"] if d.get("residual") is not None else y
