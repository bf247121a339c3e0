"""The operators around a training step of the layer, as measured cases.

Three operators of the library, each in its plain form and as the library's call:

  norm          y = (s - mean) rstd weight + bias of every row (layer norm), or y = s rstd weight (RMS norm), with
                s = x, or x + residual as stored; bf16, fp32, or e4m3 codes with one scale per 128 columns
  norm_backward the gradients of the rows, the weight and the bias
  orthogonalize steps of X <- a X + (b A + c A A) X, A = X X^T, on X = g / (|g| + eps): a matrix near the orthogonal
                factor of every expert's weight gradient

`own` chooses the library's calls; the plain forms are elementary torch operations in 32 bits, rounded once.
"""
import math

import torch

own = False

COEFFS = (3.4445, -4.775, 2.0315)
EPS_NORM = 1e-5
EPS_ORTH = 1e-7
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn}
BYTES = {"f32": 4, "bf16": 2, "fp8": 1}


def _norm(name, T, H, kind, x, y, bias, residual):
    return {"name": name, "op": "norm", "T": T, "H": H, "kind": kind, "x": x, "y": y, "bias": bias,
            "residual": residual}


def _back(name, T, H, kind, x, bias, residual):
    return {"name": name, "op": "norm_backward", "T": T, "H": H, "kind": kind, "x": x, "bias": bias,
            "residual": residual}


def _orth(name, B, m, n, out, rank):
    return {"name": name, "op": "orthogonalize", "B": B, "m": m, "n": n, "out": out, "rank": rank}


def listed():
    return [
        # one decode step of 64 tokens in front of a bf16 layer: launch latency
        _norm("norm decode", 64, 7168, "rms", "bf16", "bf16", False, True),
        # the input of an fp8 layer of 8192 tokens: bf16 rows in, e4m3 rows with their scales out
        _norm("norm to fp8", 8192, 7168, "rms", "bf16", "fp8", False, True),
        # a long bf16 batch, layer norm with bias
        _norm("norm long", 16384, 4096, "layer", "bf16", "bf16", True, False),
        # an odd token count and a width that no vector divides
        _norm("norm odd", 1001, 1537, "layer", "f32", "f32", True, True),
        # the small fp32 layer's backward: launch latency
        _back("backward small", 256, 128, "layer", "f32", True, False),
        # the training step of 2048 tokens, with the gradient that the residual stream brings
        _back("backward train", 2048, 4096, "rms", "bf16", False, True),
        # a long bf16 batch, layer norm with bias
        _back("backward long", 16384, 4096, "layer", "bf16", True, False),
        # the small fp32 layer's gate gradients
        _orth("orthogonalize small", 8, 128, 256, "f32", 0),
        # odd sizes, fp32 update
        _orth("orthogonalize odd", 3, 1001, 333, "f32", 0),
        # down-projection gradients of a few experts, some seen by few tokens (their gradients have a low rank)
        _orth("orthogonalize low rank", 4, 1536, 4096, "bf16", 24),
        # down-projection gradients of many narrow experts
        _orth("orthogonalize experts", 8, 2048, 7168, "bf16", 0),
        # up-projection gradients of wide experts
        _orth("orthogonalize wide", 4, 4096, 14336, "bf16", 0),
    ]


def _spread(rng, lo, hi):
    """A size between lo and hi, even over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_backward", "orthogonalize"])
    if op == "orthogonalize":
        out = rng.choice(["bf16", "f32"])
        while True:
            B, m, n = _spread(rng, 1, 16), _spread(rng, 40, 4096), _spread(rng, 40, 8192)
            if B * m * n <= 4 * 4096 * 7168 and min(m, n) <= (4096 if out == "bf16" else 2048):
                break
        # a low rank's small directions are rounding noise that the steps magnify: 32 bits do not hold them to 32 bits
        rank = rng.choice([0, 0, 0, _spread(rng, 2, 64)]) if out == "bf16" else 0
        return {"op": op, "B": B, "m": m, "n": n, "out": out, "rank": rank if rank < min(m, n) else 0}
    x = rng.choice(["bf16", "bf16", "f32"])
    while True:
        T, H = _spread(rng, 1, 32768), _spread(rng, 64, 16384)
        if T * H <= 16384 * 4096:
            break
    if rng.random() < 0.6:
        H = (H + 127) // 128 * 128
    kind = rng.choice(["layer", "rms"])
    case = {"op": op, "T": T, "H": H, "kind": kind, "x": x, "bias": kind == "layer" and rng.random() < 0.7,
            "residual": rng.random() < 0.5}
    if op == "norm":
        case["y"] = "fp8" if H % 128 == 0 and rng.random() < 0.35 else x
    return case


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)

    if case["op"] == "orthogonalize":
        B, m, n, r = case["B"], case["m"], case["n"], case["rank"]
        if r:  # the sum of r tokens' outer products
            grad = torch.matmul(normal(B, m, r), normal(B, r, n)) * (1e-3 / math.sqrt(r))
        else:
            grad = normal(B, m, n) * 1e-3
        return {"case": case, "g": grad, "out": torch.empty((B, m, n), dtype=TYPES[case["out"]], device="cuda")}

    T, H, dt = case["T"], case["H"], TYPES[case["x"]]
    # a residual stream: rows of different sizes about a common offset per column, a few large columns
    col = 0.3 * normal(H)
    col[:: max(1, H // 7)] += 4.0
    s = {"case": case, "weight": (1.0 + 0.2 * normal(H)).to(dt),
         "bias": (0.2 * normal(H)).to(dt) if case["bias"] else None}
    size = torch.exp(0.5 * normal(T, 1))
    s["x"] = (normal(T, H) * size + col).to(dt)
    s["mean"] = torch.empty(T, dtype=torch.float32, device="cuda") if case["kind"] == "layer" else None
    s["rstd"] = torch.empty(T, dtype=torch.float32, device="cuda")
    if case["op"] == "norm":
        s["residual"] = (0.5 * normal(T, H)).to(dt) if case["residual"] else None
        s["sum"] = torch.empty((T, H), dtype=dt, device="cuda") if case["residual"] else None
        s["y"] = torch.empty((T, H), dtype=TYPES[case["y"]], device="cuda")
        s["y_scales"] = torch.empty((T, H // 128), dtype=torch.float32, device="cuda") if case["y"] == "fp8" else None
        return s
    x = s["x"].float()
    if case["kind"] == "layer":
        s["mean"].copy_(x.mean(1))
        x = x - s["mean"][:, None]
    s["rstd"].copy_(torch.rsqrt((x * x).mean(1) + EPS_NORM))
    s["dy"] = normal(T, H).to(dt)
    s["dsum"] = normal(T, H).to(dt) if case["residual"] else None
    s["out"] = {"dx": torch.empty((T, H), dtype=dt, device="cuda"),
                "dweight": torch.empty(H, dtype=torch.float32, device="cuda"),
                "dbias": torch.empty(H, dtype=torch.float32, device="cuda") if case["bias"] else None}
    return s


def _own_run(s):
    import grouped_expert_ffn_router_amd as m

    case = s["case"]
    if case["op"] == "norm":
        r = m.moe_norm(s["x"], s["weight"], bias=s["bias"], residual=s["residual"], kind=case["kind"], eps=EPS_NORM,
                       y=s["y"], y_scales=s["y_scales"], sum=s["sum"], mean=s["mean"], rstd=s["rstd"])
        return {"y": r.y, "y_scales": r.y_scales, "sum": s["sum"], "mean": r.mean, "rstd": r.rstd}
    if case["op"] == "norm_backward":
        if "workspace" not in s:  # kept beside the buffers, as the layer keeps its own
            s["workspace"] = torch.empty(m.moe_norm_backward_workspace_bytes(case["T"], case["H"]),
                                         dtype=torch.uint8, device="cuda")
        return m.moe_norm_backward(s["dy"], s["x"], s["weight"], s["mean"], s["rstd"], kind=case["kind"],
                                   dsum=s["dsum"], want_bias=case["bias"], out=s["out"], workspace=s["workspace"])
    if "workspace" not in s:
        s["workspace"] = torch.empty(
            m.moe_orthogonalize_workspace_bytes(case["B"], case["m"], case["n"], TYPES[case["out"]]),
            dtype=torch.uint8, device="cuda")
    return m.moe_orthogonalize(s["g"], coeffs=COEFFS, eps=EPS_ORTH, out=s["out"], workspace=s["workspace"])


def _plain_norm(s):
    case = s["case"]
    x = s["x"].float()
    total = None
    if s["residual"] is not None:
        total = (x + s["residual"].float()).to(s["x"].dtype)
        x = total.float()
    mean = None
    if case["kind"] == "layer":
        mean = x.mean(1)
        x = x - mean[:, None]
    rstd = torch.rsqrt((x * x).mean(1) + EPS_NORM)
    y = x * rstd[:, None] * s["weight"].float()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    scales = None
    if case["y"] == "fp8":
        blocks = y.view(case["T"], case["H"] // 128, 128)
        amax = blocks.abs().amax(2)
        scales = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
        y = (blocks / scales[:, :, None]).clamp(-448.0, 448.0).view(case["T"], case["H"])
    return {"y": y.to(TYPES[case["y"]]), "y_scales": scales, "sum": total, "mean": mean, "rstd": rstd}


def _plain_backward(s):
    x, dy, rstd = s["x"].float(), s["dy"].float(), s["rstd"][:, None]
    layer = s["case"]["kind"] == "layer"
    xhat = (x - s["mean"][:, None]) * rstd if layer else x * rstd
    t = dy * s["weight"].float()
    dx = t - xhat * (t * xhat).mean(1, keepdim=True)
    if layer:
        dx = dx - t.mean(1, keepdim=True)
    dx = dx * rstd
    if s["dsum"] is not None:
        dx = dx + s["dsum"].float()
    return {"dx": dx.to(s["x"].dtype), "dweight": (dy * xhat).sum(0),
            "dbias": dy.sum(0) if s["bias"] is not None else None}


def _orthogonal(g):
    """The definition, in the type of g."""
    a, b, c = COEFFS
    x = g / (torch.sqrt((g * g).sum((1, 2), keepdim=True)) + EPS_ORTH)
    flip = x.shape[1] > x.shape[2]
    if flip:
        x = x.transpose(1, 2).contiguous()
    for _ in range(5):
        A = torch.matmul(x, x.transpose(1, 2))
        x = a * x + torch.matmul(b * A + c * torch.matmul(A, A), x)
    return x.transpose(1, 2).contiguous() if flip else x


def run(state):
    if own:
        return _own_run(state)
    op = state["case"]["op"]
    if op == "norm":
        return _plain_norm(state)
    if op == "norm_backward":
        return _plain_backward(state)
    return _orthogonal(state["g"]).to(TYPES[state["case"]["out"]])


def work(case):
    if case["op"] == "orthogonalize":
        B, p, q = case["B"], min(case["m"], case["n"]), max(case["m"], case["n"])
        # a step: X X^T and A A are symmetric (half of each), then the product with X
        return {"bytes": B * p * q * (4 + BYTES[case["out"]]), "flops": 5 * B * (p * p * q + p * p * p + 2 * p * p * q)}
    T, H, e = case["T"], case["H"], BYTES[case["x"]]
    stats = 4 * T * (2 if case["kind"] == "layer" else 1)
    params = H * e * (2 if case["bias"] else 1)
    if case["op"] == "norm":
        b = T * H * (e * (3 if case["residual"] else 1) + BYTES[case["y"]]) + stats + params
        return {"bytes": b + (T * H // 32 if case["y"] == "fp8" else 0), "flops": 8 * T * H}
    return {"bytes": T * H * e * (4 if case["residual"] else 3) + stats + params + 4 * H * (2 if case["bias"] else 1),
            "flops": 14 * T * H}


def _exact_norm(s):
    case = s["case"]
    x = s["x"].double()
    total = None
    if s["residual"] is not None:
        total = x + s["residual"].double()
        x = total.to(s["x"].dtype).double()  # the stored sum is what is normalised
    H = case["H"]
    if case["kind"] == "layer":
        mean = x.sum(1) / H
        var = (x * x).sum(1) / H - mean * mean  # 53 bits leave enough of the difference here
    else:
        mean, var = None, (x * x).sum(1) / H
    rstd = 1.0 / torch.sqrt(var + EPS_NORM)
    w = s["weight"].double() * rstd[:, None]
    y = x * w if mean is None else x * w - mean[:, None] * w
    if s["bias"] is not None:
        y += s["bias"].double()
    scales = None
    if case["y"] == "fp8":
        y = y.view(case["T"], -1, 128)
        big = y.abs().amax(2)
        scales = torch.where(big > 0, big / 448.0, torch.ones_like(big))
        y = (y / scales[:, :, None]).view(case["T"], H)  # the value that a code stands for
    return {"y": y, "y_scales": scales, "sum": total, "mean": mean, "rstd": rstd}


def _exact_backward(s):
    # z = (x - m) r has dz/dx = r (1 - 1/H - z z^T / H) (without the 1/H for the RMS form)
    H = s["case"]["H"]
    x, dy, r = s["x"].double(), s["dy"].double(), s["rstd"].double()[:, None]
    layer = s["case"]["kind"] == "layer"
    z = (x - s["mean"].double()[:, None]) * r if layer else x * r
    u = dy * s["weight"].double()
    along = (u * z).sum(1, keepdim=True) / H
    dx = r * (u - z * along - (u.sum(1, keepdim=True) / H if layer else 0.0))
    if s["dsum"] is not None:
        dx += s["dsum"].double()
    return {"dx": dx, "dweight": (dy * z).sum(0), "dbias": dy.sum(0) if s["bias"] is not None else None}


def _exact_orthogonal(s):
    # matrix by matrix, the step taken as a X + b (A X) + c (A (A X)): no product A A, no sum of matrices before X
    a, b, c = COEFFS
    out = []
    for g in s["g"].double():
        x = g / (g.norm() + EPS_ORTH)
        if x.shape[0] > x.shape[1]:
            x = x.T
        x = x.contiguous()
        for _ in range(5):
            gram = x @ x.T
            y = gram @ x
            x = a * x + b * y + c * (gram @ y)
        out.append(x if g.shape[0] <= g.shape[1] else x.T)
    return torch.stack([o.contiguous() for o in out])


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(s)
    if case["op"] == "norm_backward":
        return _exact_backward(s)
    return _exact_orthogonal(s)
