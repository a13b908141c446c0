"""Operators of a quantised linear layer: what is measured, with plain forms.

Five calls that stand around a product in a language model: the
root-mean-square norm with the residual's addition ("norm"), its training step
("norm_train"), the same norm with an 8-bit output and a scale per row
("norm_quant"), the product of 8-bit rows with their scales ("linear_f8") and
the product with 4-bit weights and group scales ("linear_w4").

``own = False`` computes them with elementary torch operations in 32 bits;
``own = True`` makes the calls of invariant_matmul_amd.torch_ops.
"""
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn,
          "e5m2": torch.float8_e5m2}
FMAX = {"e4m3": 448.0, "e5m2": 57344.0}
EPS = 1e-6
MIN_SCALE = 2.0 ** -120  # scale of a row that holds only zeros


def listed():
    return [
        # one token through a layer: latency alone
        {"name": "norm_token", "op": "norm", "rows": 1, "cols": 4096, "dtype": "bf16", "residual": True},
        # a long prompt, odd number of rows
        {"name": "norm_prefill", "op": "norm", "rows": 8191, "cols": 8192, "dtype": "f16", "residual": True},
        # norm of every head's query or key, no residual
        {"name": "norm_heads", "op": "norm", "rows": 32776, "cols": 128, "dtype": "bf16", "residual": False},
        # a training step's norm: forward and gradients of input, residual and weight
        {"name": "norm_train", "op": "norm_train", "rows": 4096, "cols": 4096, "dtype": "bf16", "residual": True},
        {"name": "norm_train_ragged", "op": "norm_train", "rows": 777, "cols": 1040, "dtype": "f16", "residual": False},
        # what feeds an 8-bit product: a decode batch, and a prompt
        {"name": "quant_decode", "op": "norm_quant", "rows": 32, "cols": 4096, "dtype": "bf16", "residual": True, "out": "e4m3"},
        {"name": "quant_prefill", "op": "norm_quant", "rows": 4099, "cols": 14336, "dtype": "f16", "residual": True, "out": "e4m3"},
        # fused query, key and value projection of a decode batch in 8 bits
        {"name": "f8_decode", "op": "linear_f8", "M": 16, "N": 6144, "K": 4096, "in": "e4m3", "dtype": "bf16", "bias": False},
        # a prompt through the down projection in 8 bits
        {"name": "f8_prefill", "op": "linear_f8", "M": 2051, "N": 4096, "K": 14336, "in": "e4m3", "dtype": "bf16", "bias": True},
        # one token with 4-bit weights: the stream of the weights
        {"name": "w4_token", "op": "linear_w4", "M": 1, "N": 14336, "K": 4096, "group": 128, "zeros": False, "dtype": "bf16", "bias": False},
        # a decode batch on the down projection, small groups with zero points
        {"name": "w4_batch", "op": "linear_w4", "M": 29, "N": 4096, "K": 14336, "group": 64, "zeros": True, "dtype": "f16", "bias": True},
        # a prompt with 4-bit weights: the matrix rate
        {"name": "w4_prefill", "op": "linear_w4", "M": 2048, "N": 6144, "K": 4096, "group": 128, "zeros": True, "dtype": "bf16", "bias": False},
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of step in [lo, hi], spread over its logarithm."""
    v = lo * (hi / lo) ** rng.random()
    return min(hi, max(lo, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["norm", "norm_train", "norm_quant", "linear_f8", "linear_w4"])
    dtype = rng.choice(["bf16", "f16"])
    if op.startswith("norm"):
        cols = _log(rng, 64, 16384, 16)
        most = {"norm": 8191 * 8192, "norm_train": 4096 * 4096, "norm_quant": 4099 * 14336}[op]
        rows = _log(rng, 1, min(40000, most // cols))
        case = {"op": op, "rows": rows, "cols": cols, "dtype": dtype, "residual": rng.random() < 0.6}
        if op == "norm_quant":
            case["out"] = "e4m3"
        return case
    N = _log(rng, 256, 14336, 16)
    if op == "linear_f8":
        K = _log(rng, 256, 14336, 16)
        M = _log(rng, 1, min(4096, 2051 * 4096 * 14336 // (N * K)))
        return {"op": op, "M": M, "N": N, "K": K, "in": rng.choice(["e4m3", "e5m2"]), "dtype": dtype,
                "bias": rng.random() < 0.5}
    group = rng.choice([32, 64, 128])
    K = _log(rng, 256, 14336, group)
    M = _log(rng, 1, min(4096, 2048 * 6144 * 4096 // (N * K)))
    return {"op": op, "M": M, "N": N, "K": K, "group": group, "zeros": rng.random() < 0.5,
            "dtype": dtype, "bias": rng.random() < 0.5}


def _inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device="cuda") * std

    if case["op"].startswith("norm"):
        rows, cols = case["rows"], case["cols"]
        # a residual stream: a few channels much larger than the others
        chan = 1 + 9 * (torch.rand(cols, generator=g, device="cuda") < 0.01).float()
        s = {"x": (normal(rows, cols) * chan).to(dt), "w": (1 + normal(cols, std=0.2)).to(dt)}
        if case["residual"]:
            s["r"] = (normal(rows, cols, std=2.0) * chan).to(dt)
        if case["op"] == "norm_train":
            s["dy"] = normal(rows, cols, std=0.1).to(dt)
            if case["residual"]:
                s["dh"] = normal(rows, cols, std=0.1).to(dt)
        return s
    M, N, K = case["M"], case["N"], case["K"]
    s = {"b": normal(N) if case["bias"] else None}
    if case["op"] == "linear_f8":
        f8, top = DTYPES[case["in"]], FMAX[case["in"]]
        # rows quantised to the type's full range, as rms_norm_quant leaves them
        for name, rows, std in (("x", M, 1.0), ("w", N, K ** -0.5)):
            v = normal(rows, K, std=std)
            scale = v.abs().amax(1) / top
            s[name], s["s" + name] = (v / scale[:, None]).to(f8), scale
        return s
    s["x"] = normal(M, K).to(dt)
    s["q"] = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    groups = K // case["group"]
    s["s"] = (torch.rand(N, groups, generator=g, device="cuda") + 0.5).mul(0.2 * K ** -0.5).to(dt)
    s["z"] = (torch.randint(6, 11, (N, groups), generator=g, device="cuda", dtype=torch.uint8)
              if case["zeros"] else None)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if own and case["op"] == "linear_w4":
        # the weight as a serving program keeps it, laid out once when it is loaded
        from invariant_matmul_amd import torch_ops
        s["packed"] = torch_ops.pack_w4(s["q"], s["s"], s["z"])
    return s


def run(state):
    op = {"norm": _norm, "norm_train": _norm_train, "norm_quant": _norm_quant,
          "linear_f8": _linear_f8, "linear_w4": _linear_w4}[state["case"]["op"]]
    return op(state, state["case"])


def _norm(s, case):
    if own:
        from invariant_matmul_amd import torch_ops
        return torch_ops.rms_norm(s["x"], s["w"], EPS, residual=s.get("r"))
    h, out = _stream(s)
    y = (h * _rstd(h) * s["w"].float()).to(out)
    return (y, h.to(out)) if "r" in s else y


def _norm_train(s, case):
    if own:
        from invariant_matmul_amd import torch_ops
        y, h, rstd = torch_ops.rms_norm_forward(s["x"], s["w"], EPS, residual=s.get("r"))
        dx, dw = torch_ops.rms_norm_backward(s["dy"], h, s["w"], rstd, s.get("dh"))
        return (y, dx, dw, h) if "r" in s else (y, dx, dw)
    h, out = _stream(s)
    w, dy, rstd = s["w"].float(), s["dy"].float(), _rstd(h)
    n = h * rstd
    wdy = w * dy
    dx = rstd * (wdy - n * (wdy * n).mean(1, keepdim=True))
    if "dh" in s:
        dx = dx + s["dh"].float()
    y, dx, dw = (n * w).to(out), dx.to(out), (dy * n).sum(0).to(out)
    return (y, dx, dw, h.to(out)) if "r" in s else (y, dx, dw)


def _norm_quant(s, case):
    if own:
        from invariant_matmul_amd import torch_ops
        return torch_ops.rms_norm_quant(s["x"], s["w"], EPS, residual=s.get("r"), dtype=DTYPES[case["out"]])
    h, out = _stream(s)
    t = h * _rstd(h) * s["w"].float()
    scale = (t.abs().amax(1) / FMAX[case["out"]]).clamp(min=MIN_SCALE)
    q = (t / scale[:, None]).to(DTYPES[case["out"]])
    return (q, scale, h.to(out)) if "r" in s else (q, scale)


def _linear_f8(s, case):
    out = DTYPES[case["dtype"]]
    if own:
        from invariant_matmul_amd import torch_ops
        return torch_ops.linear_f8(s["x"], s["sx"], s["w"], s["sw"], bias=s["b"], out_dtype=out)
    y = (s["x"].float() @ s["w"].float().t()) * s["sx"][:, None] * s["sw"]
    return (y if s["b"] is None else y + s["b"]).to(out)


def _linear_w4(s, case):
    out = DTYPES[case["dtype"]]
    if own:
        from invariant_matmul_amd import torch_ops
        return torch_ops.linear_w4(s["x"], s["packed"], bias=s["b"])
    # byte j of a row holds element 2 j in its low and 2 j + 1 in its high half
    q = torch.stack((s["q"] & 15, s["q"] >> 4), 2).reshape(case["N"], -1, case["group"]).float()
    z = 8.0 if s["z"] is None else s["z"].float()[:, :, None]
    w = ((q - z) * s["s"].float()[:, :, None]).reshape(case["N"], case["K"])
    y = s["x"].float() @ w.t()
    return (y if s["b"] is None else y + s["b"]).to(out)


def _stream(s):
    """The residual stream in 32 bits, as it is stored, and its type."""
    x = s["x"]
    if "r" not in s:
        return x.float(), x.dtype
    return (x.float() + s["r"].float()).to(x.dtype).float(), x.dtype


def _rstd(h):
    return torch.rsqrt((h * h).mean(1, keepdim=True) + EPS)


def work(case):
    if case["op"].startswith("norm"):
        n, rows, cols = case["rows"] * case["cols"], case["rows"], case["cols"]
        streams = 2 if case["residual"] else 1          # x (and r) in
        bytes_ = 2 * n * streams + 2 * cols
        bytes_ += 2 * n if case["residual"] else 0      # the stream out
        bytes_ += n + 4 * rows if case["op"] == "norm_quant" else 2 * n
        flops = 6 * n
        if case["op"] == "norm_train":
            # dy, the stream's gradient and the stream again in, dx and dw out
            bytes_ += 2 * n * (4 if case["residual"] else 3) + 4 * cols
            flops += 12 * n
        return {"bytes": bytes_, "flops": flops}
    M, N, K = case["M"], case["N"], case["K"]
    bytes_ = 2 * M * N + (4 * N if case["bias"] else 0)
    if case["op"] == "linear_f8":
        bytes_ += M * K + N * K + 4 * (M + N)
    else:
        bytes_ += 2 * M * K + N * K // 2 + N * (K // case["group"]) * (3 if case["zeros"] else 2)
    return {"bytes": bytes_, "flops": 2 * M * N * K}


def exact(case, seed):
    s = {k: v for k, v in _inputs(case, seed).items() if v is not None}
    if case["op"].startswith("norm"):
        h = s["x"].double()
        if "r" in s:  # the stream is stored in its own type
            h = (h + s["r"].double()).to(s["x"].dtype).double()
        w = s["w"].double()
        ms = torch.linalg.vector_norm(h, dim=1, keepdim=True) ** 2 / case["cols"] + EPS
        y = h / ms.sqrt() * w
        if case["op"] == "norm":
            return (y, h) if "r" in s else y
        if case["op"] == "norm_quant":
            scale = torch.clamp(y.abs().max(1).values / FMAX[case["out"]], min=MIN_SCALE)
            q = y / scale.unsqueeze(1)
            return (q, scale, h) if "r" in s else (q, scale)
        g = s["dy"].double() * w
        dot = torch.linalg.vecdot(g, h).unsqueeze(1)
        dx = g / ms.sqrt() - h * dot / (case["cols"] * ms ** 1.5)
        if "dh" in s:
            dx += s["dh"].double()
        dw = (s["dy"].double() * (h / ms.sqrt())).sum(0)
        return (y, dx, dw, h) if "r" in s else (y, dx, dw)
    x = s["x"].double()
    if case["op"] == "linear_f8":
        w = s["w"].double() * s["sw"].double().unsqueeze(1)
        x = x * s["sx"].double().unsqueeze(1)
    else:
        w = torch.empty(case["N"], case["K"], dtype=torch.float64, device="cuda")
        w[:, 0::2] = (s["q"] % 16).double()
        w[:, 1::2] = (s["q"] // 16).double()
        zero = s["z"].double() if "z" in s else torch.full(s["s"].shape, 8.0, dtype=torch.float64, device="cuda")
        w -= zero.repeat_interleave(case["group"], 1)
        w *= s["s"].double().repeat_interleave(case["group"], 1)
    y = x @ w.t()
    return y + s["b"].double() if "b" in s else y
