"""linear_attn_prefill and linear_attn_step against the recurrence in fp64 (oracle/linear_attn.py)."""
import numpy as np
import pytest
import torch

import gated_delta_rule_20_gb300 as gdn
from oracle import linear_attn as ref

pytestmark = pytest.mark.gpu
U = 2.0 ** -24       # half a step of fp32
HALF_BF16 = 2.0 ** -8
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def inputs(B, Hk, Hv, S, Dk, Dv, dtype, decay="token", start=True, seed=0):
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    dt = TYPES[dtype]
    x = dict(q=n(B, Hk, S, Dk).to(dt), k=n(B, Hk, S, Dk).to(dt), v=n(B, Hv, S, Dv).to(dt))
    u = torch.rand(B, Hv, S, generator=gen)
    x["g"] = {"token": -0.5 * u, "strong": -8.0 * u * u, "none": 0 * u, "weak": -0.001 * u,
              "head": -(2.0 ** (-1 - 8 * torch.rand(Hv, generator=gen)))}[decay].contiguous()
    x["state"] = 0.5 * n(B, Hv, Dk, Dv) if start else None
    return x


def bounds(r, size, dtype, tc):
    """Errors allowed to the outputs and the state, element by element.

    fp32 recurrence: a token's decay (e^g: 2 steps of the function, half one of its argument for |g| < 8: 8 U at most),
    product and sum round with 11 U of the magnitudes together; o adds Dk products in some order, and scale.
    Tensor cores: outputs take the scores and the state rounded to bf16 once each (a term passes one of the two); the state's
    sums of a chunk are cut at every 16 of 3 x 128 terms (24 times 2 U); the decays within a chunk are products of a few
    exponentials of sums (16 U and 2^-17 for the scores' differences of log-decays up to 64); the sums of the outputs
    are cut 2 x 8 times."""
    out, _ = r
    out_mag, mag, out_acc, acc = size
    Dk = mag.shape[2]
    if tc:
        o = out_mag * (HALF_BF16 + 2.0 ** -15) + 11 * U * out_acc
        s = 80 * U * mag + 11 * U * acc
    else:
        o = (Dk + 2) * U * out_mag + 11 * U * out_acc
        s = 11 * U * acc
    if dtype == "bf16":
        o = o + HALF_BF16 * (np.abs(out) + o)
    return o + 1e-37, s + 1e-37


def compare(got, r, size, dtype, tc, what):
    for x, want, most, name in zip(got, r, bounds(r, size, dtype, tc), ("out", "state")):
        x = x.double().cpu().numpy()
        assert np.isfinite(x).all(), "%s: %s has %d non-finite values" % (what, name, (~np.isfinite(x)).sum())
        worst = np.max(np.abs(x - want) / most)
        assert worst <= 1, "%s: %s is %.3g times its bound off" % (what, name, worst)
        norm = np.linalg.norm(want)
        rel = np.linalg.norm(x - want) / norm if norm else 0.0
        assert rel <= (4e-3 if name == "out" and dtype == "bf16" else 1e-6), "%s: %s off by %.3g" % (what, name, rel)


def run(x, scale, lengths=None, in_place=False, out=None, **kw):
    d = {n: t.cuda() if t is not None else None for n, t in x.items()}
    if lengths is not None:
        kw["lengths"] = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    state = d["state"]
    new = state if in_place or state is None else torch.full_like(state, float("nan"))
    y = gdn.linear_attn_prefill(d["q"], d["k"], d["v"], d["g"], scale, state, out, state_out=new, **kw)
    torch.cuda.synchronize()
    assert gdn.device_status(0) == 0
    return y


def prefill_case(B, Hk, Hv, S, Dk, Dv, dtype, decay, start, lengths=None, **kw):
    x = inputs(B, Hk, Hv, S, Dk, Dv, dtype, decay, start, seed=S + Dk)
    scale = Dk ** -0.5
    out, st, size = ref.recurrence(x["q"], x["k"], x["v"], x["g"], scale, x["state"], lengths)
    tc = dtype == "bf16" and Dk % 8 == 0 and Dv % 8 == 0 and not kw.get("force_ffma")
    compare(run(x, scale, lengths, **kw), (out, st), size, dtype, tc,
            "B %d heads %d/%d S %d D %d x %d %s %s" % (B, Hk, Hv, S, Dk, Dv, dtype, decay))


SHAPES = [
    (1, 1, 1, 1, 128, 128), (2, 1, 2, 2, 128, 128), (1, 2, 2, 127, 128, 128), (1, 1, 3, 128, 128, 128),
    (2, 2, 4, 129, 128, 128), (1, 1, 2, 300, 64, 64), (1, 2, 2, 257, 96, 64), (1, 1, 1, 385, 64, 128),
    (3, 1, 1, 70, 8, 8), (1, 1, 2, 200, 104, 120), (1, 1, 1, 1030, 128, 128), (2, 3, 3, 33, 128, 16)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_prefill(shape, dtype):
    prefill_case(*shape, dtype, "token", True)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(2, 1, 1, 65, 1, 1), (1, 1, 2, 130, 75, 33), (1, 2, 2, 48, 127, 125), (1, 1, 1, 40, 7, 128)],
                         ids=lambda s: "x".join(map(str, s)))
def test_prefill_odd_heads(shape, dtype):
    prefill_case(*shape, dtype, "token", True)


@pytest.mark.parametrize("decay", ["strong", "none", "weak", "head"])
@pytest.mark.parametrize("start", [True, False])
@pytest.mark.parametrize("kw", [dict(dtype="f32"), dict(dtype="bf16"), dict(dtype="bf16", force_ffma=True)],
                         ids=["f32", "bf16", "bf16_ffma"])
def test_prefill_decays(decay, start, kw):
    prefill_case(2, 1, 2, 290, 128, 128, kw["dtype"], decay, start, force_ffma=kw.get("force_ffma", False))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("S", [1, 128, 300])
def test_prefill_lengths(dtype, S):
    lengths = [S, 0, max(S - 1, 0), min(129, S), -5, S + 7, S // 2]
    prefill_case(len(lengths), 1, 2, S, 128, 64, dtype, "token", True, lengths=lengths)
    prefill_case(len(lengths), 1, 2, S, 64, 128, dtype, "head", False, lengths=lengths)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_behind_a_length_have_no_influence(dtype):
    """NaN and infinities behind the last token reach nothing, and the outputs' rows there stay as they were."""
    B, S, lengths = 4, 200, [130, 0, 64, 200]
    x = inputs(B, 1, 2, S, 128, 128, dtype)
    a = run(x, 0.1, lengths)
    for b, n in enumerate(lengths):
        x["q"][b, :, n:] = float("nan")
        x["k"][b, :, n:] = float("inf")
        x["v"][b, :, n:] = float("nan")
        x["g"][b, :, n:] = float("nan")
    out = torch.full((B, 2, S, 128), 7.0, dtype=TYPES[dtype], device="cuda")
    b_ = run(x, 0.1, lengths, out=out)
    assert b_[0] is out and torch.equal(a[1], b_[1])
    for b, n in enumerate(lengths):
        assert torch.equal(a[0][b, :, :n], out[b, :, :n]) and bool((out[b, :, n:] == 7.0).all())
        assert bool((a[0][b, :, n:] == 0).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_minus_infinity_starts_anew(dtype):
    """g_log of -infinity (and the type's lowest value) at a token: the outputs and the state are those of a sequence that
    starts there, to the 1e-28 of the older state that the documentation allows."""
    S = 260
    x = inputs(1, 1, 2, S, 128, 128, dtype)
    for t, lowest in ((0, -float("inf")), (100, torch.finfo(torch.float32).min), (101, -float("inf")), (200, -1e30)):
        x["g"][:, :, t] = lowest
    out, st, size = ref.recurrence(x["q"], x["k"], x["v"], x["g"], 0.1, x["state"])
    compare(run(x, 0.1), (out, st), size, dtype, dtype == "bf16", "resets")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_state_in_place_and_no_tokens(dtype):
    x = inputs(2, 1, 2, 150, 128, 128, dtype)
    a, b = run(x, 0.2), run(x, 0.2, in_place=True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    e = {n: (t[:, :, :0] if n in "qkvg" else t) for n, t in x.items()}
    out, st = run(e, 0.2)
    assert out.shape == (2, 2, 0, 128) and torch.equal(st.cpu(), x["state"])
    e["state"] = None
    assert bool((run(e, 0.2)[1] == 0).all())
    # a whole batch of empty sequences
    out, st = run(x, 0.2, [0, 0])
    assert torch.equal(st.cpu(), x["state"]) and bool((out == 0).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_prompt_in_two_halves_and_token_by_token(dtype):
    """A prompt, the same in two calls through the state, and its last tokens by steps."""
    S, at = 280, 171
    x = inputs(2, 2, 4, S, 128, 128, dtype)
    d = {n: t.cuda() for n, t in x.items()}
    part = lambda lo, hi: (d[n][:, :, lo:hi].contiguous() for n in "qkvg")  # noqa: E731
    scale = 128 ** -0.5
    st = d["state"].clone()
    outs = [gdn.linear_attn_prefill(*part(0, at), scale, st)[0], gdn.linear_attn_prefill(*part(at, S - 3), scale, st)[0]]
    for t in range(S - 3, S):
        outs.append(gdn.linear_attn_step(*part(t, t + 1), scale, st)[0])
    out, s, size = ref.recurrence(x["q"], x["k"], x["v"], x["g"], scale, x["state"])
    compare((torch.cat(outs, 2), st), (out, s), size, dtype, dtype == "bf16", "parts")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 1, 1, 128, 128), (1, 16, 32, 128, 128), (64, 4, 8, 128, 128), (3, 2, 6, 64, 128),
                                   (5, 1, 3, 75, 33), (2, 2, 2, 1, 1), (7, 3, 3, 128, 96), (300, 1, 1, 16, 8), (2, 1, 1, 96, 75),
                                   # many heads: rows of whole 16 bytes, pieces that run from one row into the next, single numbers
                                   (80, 8, 8, 24, 96), (80, 4, 8, 128, 64), (41, 3, 9, 96, 75), (40, 2, 8, 128, 127), (77, 4, 4, 2, 6),
                                   (152, 1, 2, 8, 5), (39, 8, 8, 127, 4), (80, 8, 8, 44, 33), (80, 8, 8, 45, 33), (50, 4, 8, 7, 100),
                                   (70, 9, 9, 128, 3), (80, 8, 8, 98, 90), (77, 8, 8, 1, 128), (40, 8, 8, 127, 127)],
                         ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("decay", ["token", "head"])
def test_step(shape, dtype, decay):
    B, Hk, Hv, Dk, Dv = shape
    x = inputs(B, Hk, Hv, 1, Dk, Dv, dtype, decay)
    out, st, size = ref.recurrence(x["q"], x["k"], x["v"], x["g"], 0.3, x["state"])
    d = {n: t.cuda() for n, t in x.items()}
    new = torch.full_like(d["state"], float("nan"))
    y = gdn.linear_attn_step(d["q"], d["k"], d["v"], d["g"], 0.3, d["state"], state_out=new)
    assert y[1] is new and torch.equal(d["state"].cpu(), x["state"])
    compare(y, (out, st), size, dtype, False, "step %s" % (shape,))
    z = gdn.linear_attn_step(d["q"], d["k"], d["v"], d["g"], 0.3, d["state"])
    assert z[1] is d["state"] and torch.equal(z[1], new) and torch.equal(z[0], y[0])


def test_step_from_nothing_and_reset():
    x = inputs(2, 1, 2, 1, 128, 128, "f32")
    d = {n: t.cuda() for n, t in x.items()}
    a = gdn.linear_attn_step(d["q"], d["k"], d["v"], d["g"], 1.0, None)
    b = gdn.linear_attn_step(d["q"], d["k"], d["v"], torch.full_like(d["g"], -float("inf")), 1.0, d["state"].clone())
    kv = x["k"].transpose(-1, -2) * x["v"]
    assert torch.equal(a[1].cpu(), kv) and torch.equal(b[1].cpu(), kv) and torch.equal(a[0], b[0])


def test_operands_off_16_bytes():
    """Views that start at odd elements: no tensor-core tiles, no vectors, the same results."""
    x = inputs(1, 1, 2, 140, 128, 128, "bf16")
    scale = 0.1
    out, st, size = ref.recurrence(x["q"], x["k"], x["v"], x["g"], scale, x["state"])
    d = {n: torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")[1:].view(t.shape).copy_(t) for n, t in x.items()}
    assert all(t.data_ptr() % 16 for t in d.values())
    new = torch.empty(d["state"].numel() + 1, device="cuda")[1:].view(d["state"].shape)
    y = gdn.linear_attn_prefill(d["q"], d["k"], d["v"], d["g"], scale, d["state"], state_out=new)
    compare(y, (out, st), size, "bf16", False, "unaligned")
    one = {n: t[:, :, :1].contiguous() if n != "state" else t for n, t in x.items()}
    out, st, size = ref.recurrence(one["q"], one["k"], one["v"], one["g"], scale, one["state"])
    e = {n: torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")[1:].view(t.shape).copy_(t) for n, t in one.items()}
    y = gdn.linear_attn_step(e["q"], e["k"], e["v"], e["g"], scale, e["state"], state_out=new)
    compare(y, (out, st), size, "bf16", False, "unaligned step")


@pytest.mark.parametrize("dtype, B, Hv, S, Dv, split", [
    ("bf16", 7, 2, 300, 128, False), ("bf16", 6, 3, 1000, 64, True), ("bf16", 80, 4, 300, 8, False), ("f32", 6, 2, 300, 64, True),
    ("bf16", 5, 1, 77, 75, True)])
def test_zero_padding(dtype, B, Hv, S, Dv, split):
    """Rows of out behind the lengths set to zero, whatever the inputs and out held there; all others as without."""
    lengths = ([S, 0, 130, 128, 257, S - 1, -3] * 12)[:B]
    x = inputs(B, 1, Hv, S, 64, Dv, dtype, "head")
    d = {n: t.cuda() for n, t in x.items()}
    at = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    for b, n in enumerate(lengths):
        for name in ("q", "k", "v"):
            d[name][b, :, max(n, 0):] = float("nan")
    code = gdn.GDN_BF16 if dtype == "bf16" else gdn.GDN_F32
    assert (gdn.linear_attn_segments(B, 1, Hv, S, 64, Dv, code) > 1) == split
    outs = []
    for flags in (0, gdn.GDN_ZERO_PADDING):
        out, st = torch.full_like(d["v"], 7.0), torch.empty_like(d["state"])
        dims = gdn.make_dims(B, 1, Hv, S, 64, Dv, code, flags | gdn.GDN_HEAD_DECAY)
        assert gdn.lib().gdn_linear_attn_prefill(
            *(d[n].data_ptr() for n in ("q", "k", "v", "g")), at.data_ptr(), 0.1, d["state"].data_ptr(), st.data_ptr(),
            out.data_ptr(), dims, None, 0, torch.cuda.current_stream().cuda_stream) == 0
        torch.cuda.synchronize()
        outs.append((out, st))
    assert gdn.device_status(0) == 0 and torch.equal(outs[0][1], outs[1][1])
    for b, n in enumerate(max(n, 0) for n in lengths):
        assert torch.equal(outs[0][0][b, :, :n], outs[1][0][b, :, :n])
        assert bool((outs[0][0][b, :, n:] == 7.0).all()) and bool((outs[1][0][b, :, n:] == 0).all())


def test_refusals_of_the_binding():
    x = {n: t.cuda() for n, t in inputs(2, 1, 2, 8, 64, 64, "bf16").items()}
    call = lambda **kw: gdn.linear_attn_prefill(*(kw.pop(n, x[n]) for n in ("q", "k", "v", "g")), 1.0,  # noqa: E731
                                                kw.pop("state", x["state"]), **kw)
    for bad in (dict(k=x["k"][:, :, :4]), dict(v=x["v"].transpose(1, 2)), dict(g=x["g"][:1]), dict(state=x["state"][:1]),
                dict(q=x["q"].cpu()), dict(q=x["q"][0]), dict(lengths=torch.zeros(3, dtype=torch.int32, device="cuda")),
                dict(workspace=torch.zeros(8, device="cuda"))):
        with pytest.raises(ValueError):
            call(**bad)
    for bad in (dict(q=x["q"].half()), dict(k=x["k"].float()), dict(g=x["g"].double()), dict(state=x["state"].half()),
                dict(lengths=torch.zeros(2, dtype=torch.int64, device="cuda"))):
        with pytest.raises(TypeError):
            call(**bad)
    with pytest.raises(gdn.GdnError):
        call(out=x["v"])  # over an input
