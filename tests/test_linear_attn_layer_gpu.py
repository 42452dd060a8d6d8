"""A linear attention layer as it is used: rotary positions of q and k out of the packed projection's rows, linear attention
over the prompt, RMSNormGated, output projection onto the residual stream, then single tokens; against fp64."""
import numpy as np
import pytest
import torch

import gated_delta_rule_20_gb300 as gdn
from oracle import gated_decode as gated
from oracle import linear_attn as ref

pytestmark = pytest.mark.gpu

B, S, H, Hk, Hv, D = 2, 150, 256, 2, 4, 64


def layer(p, x, hidden, state, first):
    """hidden [B, n, H] -> the new residual stream; ``state`` is updated in place."""
    n = hidden.shape[1]
    y, _, _ = gdn.rmsnorm_residual(hidden, p["norm"])
    rows = gdn.linear(y, p["W_in"])                                     # q | k | v | z of every token
    cut = lambda lo, hi, heads: rows[..., lo:hi].view(B, n, heads, D).transpose(1, 2)  # noqa: E731
    kq, kv = Hk * D, Hv * D
    q, k = gdn.rotary(cut(0, kq, Hk), cut(kq, 2 * kq, Hk), p["inv_freq"], first_position=first)
    v, z = (cut(lo, lo + kv, Hv).contiguous() for lo in (2 * kq, 2 * kq + kv))
    call = gdn.linear_attn_step if n == 1 else gdn.linear_attn_prefill
    o, _ = call(q, k, v, p["g"], D ** -0.5, state)
    o = gdn.rmsnorm_gated(o, z, p["norm_out"])
    return gdn.linear(o.transpose(1, 2).reshape(B, n, kv), p["W_out"], None, hidden)


def layer64(p, hidden, state, first):
    f = lambda t: t.double().cpu().numpy()  # noqa: E731
    x = f(hidden)
    n = x.shape[1]
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-6) * f(p["norm"])
    rows = y @ f(p["W_in"])
    cut = lambda lo, hi, heads: rows[..., lo:hi].reshape(B, n, heads, D).transpose(0, 2, 1, 3)  # noqa: E731
    kq, kv = Hk * D, Hv * D
    pos = first + np.arange(n)
    q, k = (ref.rotary(cut(lo, lo + kq, Hk), p["inv_freq"].cpu().numpy(), pos) for lo in (0, kq))
    v, z = (cut(lo, lo + kv, Hv) for lo in (2 * kq, 2 * kq + kv))
    o, st, _ = ref.recurrence(q, k, v, f(p["g"]), D ** -0.5, state)
    o = o / np.sqrt((o * o).mean(-1, keepdims=True) + 1e-6) * f(p["norm_out"]) * z / (1 + np.exp(-z))
    return x + o.transpose(0, 2, 1, 3).reshape(B, n, kv) @ f(p["W_out"]), st


def test_prompt_then_tokens():
    gen = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    width = 2 * Hk * D + 2 * Hv * D
    bf = torch.bfloat16
    p = dict(norm=1 + 0.1 * r(H), norm_out=1 + 0.1 * r(D), W_in=(r(H, width) / H ** 0.5).to(bf),
             W_out=(r(Hv * D, H) / (Hv * D) ** 0.5).to(bf), g=-(2.0 ** (-2 - 6 * torch.rand(Hv, generator=gen))))
    p = {n: t.cuda() for n, t in p.items()}
    p["inv_freq"] = gdn.rotary_frequencies(D, device="cuda")[0]
    tokens = r(B, S + 3, H).to(bf).cuda()
    state = torch.zeros(B, Hv, D, D, device="cuda")
    got = layer(p, None, tokens[:, :S].contiguous(), state, 0)
    want, st = layer64(p, tokens[:, :S], None, 0)
    norm = lambda a, b: np.linalg.norm(a - b) / np.linalg.norm(b)  # noqa: E731
    # five roundings to bf16 on the way (2^-9 of the norm each, on average less) on half of the stream's energy or less
    assert norm(got.double().cpu().numpy(), want) < 6e-3
    assert norm(state.double().cpu().numpy(), st) < 1e-2
    # single tokens, from a captured graph: the same graph for every position but the first
    hidden = torch.empty(B, 1, H, dtype=bf, device="cuda")
    for t in range(S, S + 3):
        hidden.copy_(tokens[:, t:t + 1])
        got = layer(p, None, hidden, state, t)
        want, st = layer64(p, tokens[:, t:t + 1], st, t)
        assert norm(got.double().cpu().numpy(), want) < 6e-3
    assert norm(state.double().cpu().numpy(), st) < 1e-2
    assert gdn.device_status(0) == 0 and gated is not None
