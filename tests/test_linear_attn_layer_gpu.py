"""A linear attention layer as it is used (examples/linear_attn_layer.py): rotary positions of q and k out of the packed
projection's rows, linear attention over the prompt, RMSNormGated, output projection onto the residual stream, then
single tokens from a captured graph; against fp64."""
import os
import sys

import numpy as np
import pytest
import torch

import gated_delta_rule_20_gb300 as gdn
from oracle import linear_attn as ref

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import linear_attn_layer as example  # noqa: E402

pytestmark = pytest.mark.gpu

B, S, H, Hk, Hv, D = 2, 150, 256, 2, 4, 64


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
    o, st, _ = ref.recurrence(q, k, v, f(p["g_log"]), D ** -0.5, state)
    o = o / np.sqrt((o * o).mean(-1, keepdims=True) + 1e-6) * f(p["norm_out"]) * z / (1 + np.exp(-z))
    return x + o.transpose(0, 2, 1, 3).reshape(B, n, kv) @ f(p["W_out"]), st


def off(a, b):
    return float(np.linalg.norm(a.double().cpu().numpy() - b) / np.linalg.norm(b))


def test_prompt_then_tokens():
    p = example.make_layer(H, Hk, Hv, D, seed=3)
    gen = torch.Generator().manual_seed(4)
    tokens = torch.randn(B, S + 3, H, generator=gen).to(torch.bfloat16).cuda()
    state = torch.zeros(B, Hv, D, D, device="cuda")
    got = example.forward(p, tokens[:, :S].contiguous(), state)
    want, st = layer64(p, tokens[:, :S], None, 0)
    # five roundings to bf16 on the way (2^-9 of the norm each, on average less) on half of the stream's energy or less
    assert off(got, want) < 6e-3 and off(state, st) < 1e-2
    # single tokens: one captured graph, replayed at every position
    hidden = torch.empty(B, 1, H, dtype=torch.bfloat16, device="cuda")
    position = torch.full((1,), S, dtype=torch.int64, device="cuda")
    keep = state.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        hidden.copy_(tokens[:, S:S + 1])
        example.forward(p, hidden, state, position)
    torch.cuda.current_stream().wait_stream(side)
    state.copy_(keep)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = example.forward(p, hidden, state, position)
    for t in range(S, S + 3):
        hidden.copy_(tokens[:, t:t + 1])
        position.fill_(t)
        graph.replay()
        want, st = layer64(p, tokens[:, t:t + 1], st, t)
        assert off(got, want) < 6e-3
    assert off(state, st) < 1e-2
    assert gdn.device_status(0) == 0


def test_example_runs(capsys):
    example.main(["--batch", "2", "--hidden", "256", "--prompt", "300", "--steps", "4"])
    assert "us a step of 2 sequences" in capsys.readouterr().out
