"""Linear attention with a decay for each head, and rotary positions, as cases to be measured.

Operators (the framework's entry points; see ``include/gdn.h``):

``linear_attn_prefill``  S_t = e^{g_t} S_{t-1} + k_t v_t^T,  o_t = scale S_t^T q_t over whole prompts, the
                         decay a token's (g_log [B, Hv, S]) or a head's (g_log [Hv])
``linear_attn_step``     the same for one token of every sequence
``rotary``               rotary positions of q and k: half or interleaved pairs, a part of the head, given
                         frequencies (scaled for long contexts or not)

Where ``own`` is false, ``run`` computes them in their plain form; where it is true it makes the
framework's calls.  Heads (16 or 8 key heads, 32 value heads, 128 channels), 64 sequences a decode step,
4 x 4096, 1 x 32768 and 16 x 2048 tokens a prefill are this repository's own workloads; the others are
generic.
"""
import math

import torch

own = False

CHUNK = 128  # tokens that the plain form of the prefill takes together
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}


def listed():
    pre = lambda name, B, Hk, Hv, S, Dk, Dv, dtype, decay, start, ragged: {  # noqa: E731
        "name": name, "op": "prefill", "B": B, "Hk": Hk, "Hv": Hv, "S": S, "Dk": Dk, "Dv": Dv, "dtype": dtype,
        "decay": decay, "start": start, "ragged": ragged}
    step = lambda name, B, Hk, Hv, Dk, Dv, dtype, decay: {  # noqa: E731
        "name": name, "op": "step", "B": B, "Hk": Hk, "Hv": Hv, "S": 1, "Dk": Dk, "Dv": Dv, "dtype": dtype, "decay": decay,
        "start": True, "ragged": False}
    rot = lambda name, B, Hq, Hk, S, D, R, dtype, layout, packed, scaled, at: {  # noqa: E731
        "name": name, "op": "rotary", "B": B, "Hq": Hq, "Hk": Hk, "S": S, "D": D, "R": R, "dtype": dtype, "layout": layout,
        "packed": packed, "scaled": scaled, "at": at}
    return [
        # one short prompt of a small fp32 model (latency)
        pre("prefill_small_f32", 1, 2, 2, 128, 64, 64, "f32", "token", False, False),
        # a batch of prompts, each head with a decay of its own, from a cached state
        pre("prefill_batch", 4, 16, 32, 4096, 128, 128, "bf16", "head", True, False),
        # one long prompt from nothing: few heads for the whole card
        pre("prefill_long", 1, 16, 32, 32768, 128, 128, "bf16", "token", False, False),
        # many prompts, few key heads, decays down to e^-2 a token
        pre("prefill_wide", 16, 8, 32, 2048, 128, 128, "bf16", "strong", True, False),
        # a padded batch of prompts of unequal length, heads of 96 and 64 channels
        pre("prefill_ragged", 3, 4, 12, 1237, 96, 64, "bf16", "head", True, True),
        # one sequence's decode step (latency)
        step("step_one", 1, 16, 32, 128, 128, "bf16", "head"),
        # the decode step of 64 sequences
        step("step_batch", 64, 16, 32, 128, 128, "bf16", "token"),
        # an fp32 model with odd heads
        step("step_odd_f32", 37, 3, 9, 96, 75, "f32", "token"),
        # one sequence's decode step: q and k out of the packed q | k | v row (latency)
        rot("rotary_token", 1, 16, 16, 1, 128, 128, "bf16", "half", True, False, "far"),
        # a prefill's q and k out of the packed projection into head-major rows
        rot("rotary_prefill", 4, 16, 16, 4096, 128, 128, "bf16", "half", True, False, "start"),
        # one long prompt, a quarter of each head, frequencies scaled for a long context
        rot("rotary_long", 1, 32, 8, 32768, 128, 32, "bf16", "interleaved", False, True, "start"),
        # fp32, odd sizes, the sequences at positions of their own
        rot("rotary_odd_f32", 7, 5, 3, 333, 90, 46, "f32", "interleaved", False, False, "far"),
    ]


def _size(rng, lo, hi, step=1):
    """A size spread over the logarithm of [lo, hi], a multiple of `step`."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step
    return min(max(n, lo), hi)


def _heads(rng, most):
    Hk = _size(rng, 1, most)
    return Hk, Hk * rng.choice([1, 1, 2, 2, 3, 4])


def draw(rng):
    op = rng.choice(["prefill", "prefill", "step", "rotary"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op == "rotary":
        while True:
            B, S, D = _size(rng, 1, 64), _size(rng, 1, 32768), rng.choice([64, 80, 96, 128, 128, 192, 256, _size(rng, 16, 256, 2)])
            Hq = _size(rng, 1, 64)
            Hk = rng.choice([Hq, max(1, Hq // 4), 0, _size(rng, 1, 64)])
            if B * S * (Hq + Hk) * D * BYTES[dtype] <= 2 ** 28:
                break
        R = D if rng.random() < 0.5 else _size(rng, 2, D, 2)
        return {"op": op, "B": B, "Hq": Hq, "Hk": Hk, "S": S, "D": D, "R": R, "dtype": dtype,
                "layout": rng.choice(["half", "interleaved"]), "packed": rng.random() < 0.5, "scaled": rng.random() < 0.4,
                "at": rng.choice(["start", "far"])}
    decay = rng.choice(["token", "head", "strong"])
    while True:
        B, (Hk, Hv) = _size(rng, 1, 64), _heads(rng, 32)
        if dtype == "bf16":
            Dk, Dv = (rng.choice([128, 128, 128, 64, 96, 80, _size(rng, 8, 128)]) for _ in range(2))
        else:
            Dk, Dv = (rng.choice([128, 64, _size(rng, 8, 128)]) for _ in range(2))
        S = 1 if op == "step" else _size(rng, 2, 32768)
        # at most the work of 4 x 32 heads x 4096 tokens in bf16, and of an eighth of that in fp32
        if B * Hv * S <= (2 ** 19 if dtype == "bf16" else 2 ** 16):
            break
    return {"op": op, "B": B, "Hk": Hk, "Hv": Hv, "S": S, "Dk": Dk, "Dv": Dv, "dtype": dtype, "decay": decay,
            "start": op == "step" or rng.random() < 0.6, "ragged": op == "prefill" and rng.random() < 0.3}


def _frequencies(case):
    """The angles that a position adds, and what the rotated channels are multiplied by."""
    n = case["R"] // 2
    f = 10000.0 ** (-torch.arange(n, dtype=torch.float64) / n)
    if not case["scaled"]:
        return f, 1.0
    # positions past 4096 at a factor of 8: slow pairs are slowed by it, fast ones are left, a ramp between
    turns = 4096 * f / (2 * math.pi)
    keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0, 1)
    return f * (keep + (1 - keep) / 8.0), 0.1 * math.log(8.0) + 1.0


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    normal = lambda *shape: torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)  # noqa: E731
    uniform = lambda *shape: torch.rand(shape, generator=gen, device="cuda", dtype=torch.float32)  # noqa: E731
    s, dt = dict(case), TYPES[case["dtype"]]
    B, S = case["B"], case["S"]
    if case["op"] == "rotary":
        Hq, Hk, D = case["Hq"], case["Hk"], case["D"]
        if case["packed"]:  # views into the projection's rows: q | k | v
            rows = normal(B, S, (Hq + 2 * Hk) * D).to(dt)
            s["q"] = rows[..., :Hq * D].view(B, S, Hq, D).transpose(1, 2)
            s["k"] = rows[..., Hq * D:(Hq + Hk) * D].view(B, S, Hk, D).transpose(1, 2) if Hk else None
        else:
            s["q"], s["k"] = normal(B, Hq, S, D).to(dt), normal(B, Hk, S, D).to(dt) if Hk else None
        f, s["amplitude"] = _frequencies(case)
        s["inv_freq"] = f.cuda()
        at = torch.zeros(B, 1, device="cuda") if case["at"] == "start" else uniform(B, 1) * 2.0 ** 20
        s["positions"] = at.to(torch.int64) + torch.arange(S, device="cuda")
        return s
    Hk, Hv, Dk, Dv = case["Hk"], case["Hv"], case["Dk"], case["Dv"]
    s["q"], s["k"] = normal(B, Hk, S, Dk).to(dt), normal(B, Hk, S, Dk).to(dt)
    s["v"] = normal(B, Hv, S, Dv).to(dt)
    if case["decay"] == "token":    # this repository's gates of a prefill
        s["g"] = -(0.005 + 0.495 * uniform(B, Hv, S))
    elif case["decay"] == "strong":
        s["g"] = -(0.001 + 1.999 * uniform(B, Hv, S))
    else:                           # a head's own: 1 / 2 to 1 / 512 of the state is lost a token
        s["g"] = -(2.0 ** (-1 - 8 * uniform(Hv)))
    s["state"] = 0.5 * normal(B, Hv, Dk, Dv) if case["start"] else None
    s["lengths"] = None
    if case["ragged"]:              # one sequence has every row, one may have none
        s["lengths"] = (uniform(B) * (S + 1)).to(torch.int32).clamp_max(S)
        s["lengths"][0] = S
    s["scale"] = Dk ** -0.5
    return s


def _prefill(s):
    """Chunk by chunk, all at once: a chunk's own part is a masked product, and the states in front of the
    chunks are the products of the chunks' own states with the decays between them."""
    B, Hk, S, Dk = s["q"].shape
    Hv, Dv = s["v"].shape[1], s["v"].shape[3]
    r, N = Hv // Hk, -(-S // CHUNK)
    n = S if s["lengths"] is None else s["lengths"].view(B, 1, 1)
    there = (torch.arange(N * CHUNK, device="cuda") < n).expand(B, 1, N * CHUNK)
    g = s["g"].double()
    g = g.view(1, Hv, 1).expand(B, Hv, S) if g.dim() == 1 else g
    cut = lambda x: torch.nn.functional.pad(x, (0, 0, 0, N * CHUNK - S)) * there[..., None]  # noqa: E731
    q = cut(s["q"].float()).view(B, Hk, 1, N, CHUNK, Dk)
    k = cut(s["k"].float()).view(B, Hk, 1, N, CHUNK, Dk)
    v = cut(s["v"].float()).view(B, Hk, r, N, CHUNK, Dv)
    g = cut(g[..., None]).view(B, Hk, r, N, CHUNK)
    c = g.cumsum(-1)                                    # (64 bits: the differences are next to each other)
    total = c[..., -1]
    low = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device="cuda").tril()
    between = torch.exp((c[..., :, None] - c[..., None, :]).masked_fill(~low, -math.inf).float())
    inner = torch.matmul(torch.matmul(q, k.transpose(-1, -2)) * between, v)
    own_state = torch.matmul((k * torch.exp(total[..., None] - c).float()[..., None]).transpose(-1, -2), v)
    # the start state and the chunks' states, each decayed to the front of chunk 0 .. N (N: the end)
    start = torch.zeros(B, Hk, r, 1, Dk, Dv, device="cuda") if s["state"] is None else s["state"].view(B, Hk, r, 1, Dk, Dv)
    parts = torch.cat([start, own_state], 3)
    at = torch.nn.functional.pad(total, (1, 0)).cumsum(-1)
    low = torch.ones(N + 1, N + 1, dtype=torch.bool, device="cuda").tril()
    decay = torch.exp((at[..., :, None] - at[..., None, :]).masked_fill(~low, -math.inf).float())
    states = torch.matmul(decay, parts.flatten(-2)).view(parts.shape)
    out = s["scale"] * (inner + torch.exp(c).float()[..., None] * torch.matmul(q, states[..., :-1, :, :]))
    out = out.reshape(B, Hv, N * CHUNK, Dv) * there[..., None]
    return out[:, :, :S].to(s["q"].dtype), states[..., -1, :, :].reshape(B, Hv, Dk, Dv)


def _step(s):
    r = s["Hv"] // s["Hk"]
    q, k = s["q"].float().repeat_interleave(r, 1), s["k"].float().repeat_interleave(r, 1)
    state = torch.exp(s["g"]).view(-1, s["Hv"], 1, 1) * s["state"] + k.transpose(-1, -2) * s["v"].float()
    return (s["scale"] * torch.matmul(q, state)).to(s["q"].dtype), state


def _rotary(s, x):
    """x [B, H, S, D] with its first R channels turned."""
    R = s["R"]
    angle = s["positions"].double()[:, None, :, None] * s["inv_freq"]
    cos, sin = ((s["amplitude"] * f(angle)).float() for f in (torch.cos, torch.sin))
    t = x[..., :R].float()
    if s["layout"] == "half":
        a, b = t[..., :R // 2], t[..., R // 2:]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = t[..., 0::2], t[..., 1::2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([y.to(x.dtype), x[..., R:]], -1)


def run(s):
    if own:
        import gated_delta_rule_20_gb300 as gdn
        if s["op"] == "prefill":
            fresh = None if s["state"] is None else torch.empty_like(s["state"])
            return gdn.linear_attn_prefill(s["q"], s["k"], s["v"], s["g"], s["scale"], s["state"], lengths=s["lengths"],
                                           state_out=fresh)
        if s["op"] == "step":
            return gdn.linear_attn_step(s["q"], s["k"], s["v"], s["g"], s["scale"], s["state"],
                                        state_out=torch.empty_like(s["state"]))
        y = gdn.rotary(s["q"], s["k"], s["inv_freq"], s["positions"], layout=s["layout"], amplitude=s["amplitude"])
        return y if s["k"] is not None else y[:1]
    if s["op"] == "prefill":
        return _prefill(s)
    if s["op"] == "step":
        return _step(s)
    return (_rotary(s, s["q"]),) if s["k"] is None else (_rotary(s, s["q"]), _rotary(s, s["k"]))


def work(case):
    B, S, b = case["B"], case["S"], BYTES[case["dtype"]]
    if case["op"] == "rotary":
        heads = case["Hq"] + case["Hk"]
        return {"bytes": 2 * b * B * S * heads * case["D"] + 8 * B * S + 4 * case["R"],
                "flops": 3 * B * S * heads * case["R"]}
    Hk, Hv, Dk, Dv = case["Hk"], case["Hv"], case["Dk"], case["Dv"]
    rows = B * S if not case["ragged"] else S + (B - 1) * S // 2  # (half of a padded sequence's rows, on average)
    tokens = b * rows * (2 * Hk * Dk + 2 * Hv * Dv)
    gates = 4 * (Hv if case["decay"] == "head" else rows * Hv)
    states = 4 * B * Hv * Dk * Dv * (2 if case["start"] else 1)
    return {"bytes": tokens + gates + states, "flops": 4 * rows * Hv * Dk * Dv}


def exact(case, seed):
    """The definitions in 64 bits: the recurrence token by token, and the turn of each pair as a complex number."""
    s = prepare(case, seed)
    d = torch.float64
    if case["op"] == "rotary":
        turn = torch.polar(torch.full((), s["amplitude"], dtype=d, device="cuda"),
                           torch.einsum("bs,f->bsf", s["positions"].to(d), s["inv_freq"])).unsqueeze(1)
        ys = []
        for x in (s["q"], s["k"]):
            if x is None:
                continue
            y, R = x.to(d).contiguous(), case["R"]
            if case["layout"] == "half":
                z = torch.complex(y[..., :R // 2], y[..., R // 2:R]) * turn
                y[..., :R // 2], y[..., R // 2:R] = z.real, z.imag
            else:
                z = torch.complex(y[..., 0:R:2], y[..., 1:R:2]) * turn
                y[..., 0:R:2], y[..., 1:R:2] = z.real, z.imag
            ys.append(y)
        return tuple(ys)
    B, Hk, Hv, S, Dk, Dv = (case[n] for n in ("B", "Hk", "Hv", "S", "Dk", "Dv"))
    if B * Hv * S * Dk * Dv > 2 ** 36:
        return None
    state = torch.zeros(B, Hk, Hv // Hk, Dk, Dv, dtype=d, device="cuda")
    if s["state"] is not None:
        state += s["state"].view(state.shape)
    g = s["g"].to(d).view(-1, Hk, Hv // Hk, s["g"].shape[-1] if s["g"].dim() == 3 else 1, 1, 1)
    outs = torch.zeros(B, Hk, Hv // Hk, S, Dv, dtype=d, device="cuda")
    v = s["v"].view(B, Hk, Hv // Hk, S, Dv)
    lengths = None if s["lengths"] is None else s["lengths"].tolist()
    for t in range(S):
        new = state * g[:, :, :, t if g.shape[3] > 1 else 0].exp()
        new += s["k"][:, :, t].to(d)[:, :, None, :, None] * v[:, :, :, t].to(d)[:, :, :, None, :]
        o = torch.einsum("ghk,ghrkv->ghrv", s["q"][:, :, t].to(d), new) * s["scale"]
        if lengths is None:
            state, outs[:, :, :, t] = new, o
            continue
        live = torch.tensor([t < n for n in lengths], device="cuda")
        state = torch.where(live[:, None, None, None, None], new, state)
        outs[:, :, :, t] = torch.where(live[:, None, None, None], o, torch.zeros_like(o))
    return outs.view(B, Hv, S, Dv), state.view(B, Hv, Dk, Dv)
