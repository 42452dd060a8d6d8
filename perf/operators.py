"""The layer operators around the gated delta rule, as cases to be measured.

Operators (the framework's entry points; see ``include/gdn.h``):

``rmsnorm_residual``   h = x + residual,  y = h / sqrt(mean(h^2) + eps) * w;  y in the compute dtype
                       or in 8 bits (e4m3) with one scale a row
``linear``             act(x W + bias) + residual, x and W in bf16, fp32 or 8 bits with scales
``linear_gated``       act(x Wg + bg) * (x Wu + bu) + residual, Wg and Wu stored as one weight

Where ``own`` is false, ``run`` computes them in their plain form; where it is true it makes the
framework's calls.  Sizes: H = 2048 hidden channels, value_dim = 4096 = 32 heads x 128, conv_dim =
8192, 64 sequences a decode step and 4 x 4096 tokens a prefill are this repository's own workloads;
the others are generic.
"""
import math

import torch

own = False

EPS = 1e-6
F8_MAX = 448.0      # largest finite e4m3 value
AMAX_MIN = 1e-30    # least row maximum that a scale is made from
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "f8": torch.float8_e4m3fn}
BYTES = {"bf16": 2, "f32": 4, "f8": 1}


def listed():
    norm = lambda name, rows, D, dtype, out, residual: {  # noqa: E731
        "name": name, "op": "norm", "rows": rows, "D": D, "dtype": dtype, "out": out, "residual": residual}
    mat = lambda name, op, M, K, N, dtype, out, layout, act, bias, residual: {  # noqa: E731
        "name": name, "op": op, "M": M, "K": K, "N": N, "dtype": dtype, "out": out, "layout": layout, "act": act,
        "bias": bias, "residual": residual}
    return [
        # one sequence's decode step: the norm in front of an 8-bit projection (latency)
        norm("norm_token_f8", 1, 2048, "bf16", "f8", True),
        # the decode step of 64 sequences: the norm in front of the decode block
        norm("norm_batch", 64, 2048, "bf16", "bf16", True),
        # fp32 compute, a row that no vector width divides, the first layer's norm (no residual yet)
        norm("norm_ragged_f32", 1237, 2051, "f32", "f32", False),
        # a prefill's 4 x 4096 tokens in front of an 8-bit projection
        norm("norm_prefill_f8", 16384, 2048, "bf16", "f8", True),
        # the same tokens in a wide model
        norm("norm_wide", 16384, 8192, "bf16", "bf16", True),
        # one token's output projection (value_dim -> H) added to the residual stream (latency, weight-bound)
        mat("linear_token", "linear", 1, 4096, 2048, "bf16", "bf16", "kn", "none", False, True),
        # the same for the decode step's 64 sequences
        mat("linear_batch", "linear", 64, 4096, 2048, "bf16", "bf16", "kn", "none", False, True),
        # the decode step's gated feed-forward projection in 8 bits
        mat("gated_batch_f8", "gated", 64, 2048, 8192, "f8", "bf16", "nk", "silu", False, False),
        # ragged tokens of several prompts and an odd output width, with bias and GELU
        mat("linear_ragged", "linear", 1003, 2056, 5001, "bf16", "bf16", "nk", "gelu", True, False),
        # fp32 compute, odd sizes (a small head on top of a model)
        mat("linear_f32", "linear", 333, 770, 1030, "f32", "f32", "kn", "relu", True, False),
        # a prefill's output projection added to the residual stream
        mat("linear_prefill", "linear", 16384, 4096, 2048, "bf16", "bf16", "kn", "none", False, True),
        # a prefill's gated feed-forward projection in 8 bits
        mat("gated_prefill_f8", "gated", 16384, 2048, 8192, "f8", "bf16", "nk", "silu", False, False),
    ]


def _size(rng, lo, hi, step):
    """A size spread over the logarithm of [lo, hi], a multiple of `step` (3072 is left out)."""
    while True:
        n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step
        n = min(max(n, lo), hi)
        if n != 3072:
            return n


def draw(rng):
    if rng.random() < 0.4:
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        while True:
            D = _size(rng, 64, 16384, rng.choice([64, 8, 8, 1]))
            rows = _size(rng, 1, 32768, 1)
            if rows * D * BYTES[dtype] <= 16384 * 8192 * 2:
                break
        return {"op": "norm", "rows": rows, "D": D, "dtype": dtype, "out": rng.choice([dtype, "f8"]),
                "residual": rng.random() < 0.75}
    op = rng.choice(["linear", "linear", "gated"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f8", "f8", "f32"])
    while True:
        M = _size(rng, 1, 16384, 1)
        if dtype == "f32":  # the small fp32 layers: sizes of any parity
            K, N = _size(rng, 64, 2048, rng.choice([8, 1])), _size(rng, 64, 2048, rng.choice([8, 1]))
        else:  # rows of whole 16-byte pieces mostly, as weights have them
            K = _size(rng, 64, 16384, rng.choice([64, 64, 16, 16, 16, 1]))
            N = _size(rng, 64, 16384, rng.choice([64, 64, 8, 8, 8, 1]))
        if M * K * N * (2 if op == "gated" else 1) <= 2 ** 38:
            break
    return {"op": op, "M": M, "K": K, "N": N, "dtype": dtype,
            "out": "f32" if dtype == "f32" or rng.random() < 0.15 else "bf16",
            "layout": "nk" if dtype == "f8" else rng.choice(["kn", "nk"]),
            "act": rng.choice(["silu", "gelu"] if op == "gated" else ["none", "none", "silu", "gelu", "relu"]),
            "bias": rng.random() < 0.4, "residual": rng.random() < 0.5}


def _to_8_bits(x):
    """Rows of x in e4m3 and the scales that they are multiplied by."""
    s = x.abs().amax(dim=1).clamp_min(AMAX_MIN) / F8_MAX
    return (x / s[:, None]).to(torch.float8_e4m3fn), s


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    normal = lambda *shape: torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)  # noqa: E731
    s = dict(case)
    if case["op"] == "norm":
        # a residual stream: channels of unequal size, a few of them large
        D, dt = case["D"], TYPES[case["dtype"]]
        width = torch.exp(0.7 * normal(D))
        s["x"] = (0.5 * normal(case["rows"], D)).to(dt)
        s["res"] = (width * normal(case["rows"], D)).to(dt) if case["residual"] else None
        s["w"] = 1.0 + 0.1 * normal(D)
        return s
    M, K, N = case["M"], case["K"], case["N"]
    n = 2 * N if case["op"] == "gated" else N
    x, w = normal(M, K), normal(n, K) / math.sqrt(K)
    s["xs"] = s["ws"] = None
    if case["dtype"] == "f8":
        (s["x"], s["xs"]), (s["w"], s["ws"]) = _to_8_bits(x), _to_8_bits(w)
    else:
        s["x"], s["w"] = x.to(TYPES[case["dtype"]]), w.to(TYPES[case["dtype"]])
    if case["layout"] == "kn":
        s["w"] = s["w"].t().contiguous()
    s["b"] = 0.1 * normal(n) if case["bias"] else None
    s["res"] = normal(M, N).to(TYPES[case["out"]]) if case["residual"] else None
    return s


def _act(name, x):
    if name == "silu":
        return x / (1 + torch.exp(-x))
    if name == "gelu":
        return 0.5 * x * (1 + torch.erf(x * math.sqrt(0.5)))
    if name == "relu":
        return x.clamp_min(0)
    return x


def _norm(s, as_type):
    """The norm's outputs before their rounding: (y, y's row scales or None, h)."""
    h = s["x"].to(as_type)
    if s["res"] is not None:
        h = h + s["res"].to(as_type)
    y = h * torch.rsqrt((h * h).mean(dim=1, keepdim=True) + EPS) * s["w"].to(as_type)
    if s["out"] != "f8":
        return y, None, h
    scale = y.abs().amax(dim=1).clamp_min(AMAX_MIN) / F8_MAX
    return y / scale[:, None], scale, h


def _matrix(s, as_type):
    """The product and its epilogue before the output's rounding."""
    w = s["w"].to(as_type)
    y = s["x"].to(as_type) @ (w if s["layout"] == "kn" else w.t())
    if s["xs"] is not None:
        y = y * s["xs"].to(as_type)[:, None] * s["ws"].to(as_type)[None, :]
    if s["b"] is not None:
        y = y + s["b"].to(as_type)
    if s["op"] == "gated":
        y = _act(s["act"], y[:, :s["N"]]) * y[:, s["N"]:]
    else:
        y = _act(s["act"], y)
    return y if s["res"] is None else y + s["res"].to(as_type)


def run(s):
    if own:
        import gated_delta_rule_20_gb300 as gdn
        if s["op"] == "norm":
            out, scale, h = gdn.rmsnorm_residual(s["x"], s["w"], s["res"], eps=EPS, out_dtype=TYPES[s["out"]])
            return {k: v for k, v in (("y", out), ("scale", scale), ("h", h)) if v is not None}
        call = gdn.linear_gated if s["op"] == "gated" else gdn.linear
        return call(s["x"], s["w"], s["b"], s["res"], activation=s["act"], weight_layout=s["layout"],
                    x_scale=s["xs"], weight_scale=s["ws"], out_dtype=TYPES[s["out"]])
    if s["op"] != "norm":
        return _matrix(s, torch.float32).to(TYPES[s["out"]])
    y, scale, h = _norm(s, torch.float32)
    r = {"y": y.to(TYPES[s["out"]])}
    if scale is not None:
        r["scale"] = scale
    if s["res"] is not None:
        r["h"] = h.to(TYPES[s["dtype"]])
    return r


def work(case):
    if case["op"] == "norm":
        n, b = case["rows"] * case["D"], BYTES[case["dtype"]]
        moved = n * (b + BYTES[case["out"]] + (2 * b if case["residual"] else 0)) + 4 * case["D"]
        return {"bytes": moved + (4 * case["rows"] if case["out"] == "f8" else 0), "flops": 5 * n}
    M, K, N, b, o = case["M"], case["K"], case["N"], BYTES[case["dtype"]], BYTES[case["out"]]
    n = 2 * N if case["op"] == "gated" else N
    moved = b * (M * K + n * K) + o * M * N * (2 if case["residual"] else 1) + (4 * n if case["bias"] else 0)
    return {"bytes": moved + (4 * (M + n) if case["dtype"] == "f8" else 0), "flops": 2 * M * n * K}


def exact(case, seed):
    s = prepare(case, seed)
    d = torch.float64
    if case["op"] == "norm":
        h = s["x"].to(d) if s["res"] is None else s["x"].to(d) + s["res"].to(d)
        y = h / torch.sqrt(h.square().sum(1, keepdim=True) / case["D"] + EPS) * s["w"].to(d)
        r = {"y": y}
        if case["out"] == "f8":
            r["scale"] = torch.clamp(y.abs().max(dim=1).values, min=AMAX_MIN) / F8_MAX
            r["y"] = y / r["scale"].unsqueeze(1)
        if s["res"] is not None:
            r["h"] = h
        return r
    # row by row of 2048 tokens, so that the 64-bit copies stay small
    x, w, N, parts = s["x"], s["w"].to(d), case["N"], []
    w = w if case["layout"] == "nk" else w.t()
    w = w if s["ws"] is None else w * s["ws"].to(d).unsqueeze(1)
    for at in range(0, case["M"], 2048):
        t = x[at:at + 2048].to(d)
        t = t if s["xs"] is None else t * s["xs"][at:at + 2048].to(d).unsqueeze(1)
        y = torch.einsum("mk,nk->mn", t, w)
        y = y if s["b"] is None else y + s["b"].to(d).unsqueeze(0)
        g, u = (y[:, :N], y[:, N:]) if case["op"] == "gated" else (y, None)
        if case["act"] == "silu":
            g = g * torch.sigmoid(g)
        elif case["act"] == "gelu":
            g = g * (0.5 - 0.5 * torch.erf(-g / math.sqrt(2.0)))
        elif case["act"] == "relu":
            g = torch.where(g > 0, g, torch.zeros_like(g))
        y = g if u is None else g * u
        parts.append(y if s["res"] is None else y + s["res"][at:at + 2048].to(d))
    return torch.cat(parts)
