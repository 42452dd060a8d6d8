"""A linear attention layer with rotary positions: norm, packed projection, rotary positions of q and k out of its rows, linear
attention with a decay for each head, RMSNormGated, output projection onto the residual stream.

    python examples/linear_attn_layer.py [--batch 4] [--hidden 2048] [--prompt 4096] [--steps 32]

runs a prompt and then single tokens, those from a captured CUDA graph, on synthetic weights, and prints the times.
(tests/test_linear_attn_layer_gpu.py compares the layer with fp64.)
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gated_delta_rule_20_gb300 as gdn  # noqa: E402


def make_layer(hidden, Hk, Hv, D, seed=0, device="cuda"):
    """Weights of a layer of Hk key and Hv value heads of D channels."""
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    bf = torch.bfloat16
    p = dict(norm=1 + 0.1 * r(hidden), norm_out=1 + 0.1 * r(D), W_in=(r(hidden, 2 * (Hk + Hv) * D) / hidden ** 0.5).to(bf),
             W_out=(r(Hv * D, hidden) / (Hv * D) ** 0.5).to(bf), g_log=-(2.0 ** (-2 - 6 * torch.rand(Hv, generator=gen))))
    p = {n: t.to(device) for n, t in p.items()}
    p["inv_freq"], p["amplitude"] = gdn.rotary_frequencies(D, device=device)
    return dict(p, Hk=Hk, Hv=Hv, D=D)


def forward(p, hidden, state, positions=None):
    """hidden [B, n, H] bf16 -> the new residual stream; ``state`` [B, Hv, D, D] is updated in place.  ``positions``: [B, n] or
    [n] (None: 0 .. n - 1)."""
    B, n = hidden.shape[:2]
    D, kq, kv = p["D"], p["Hk"] * p["D"], p["Hv"] * p["D"]
    y, _, _ = gdn.rmsnorm_residual(hidden, p["norm"])
    rows = gdn.linear(y, p["W_in"])                                              # q | k | v | z of every token
    heads = lambda lo, hi: rows[..., lo:hi].view(B, n, (hi - lo) // D, D).transpose(1, 2)  # noqa: E731
    q, k = gdn.rotary(heads(0, kq), heads(kq, 2 * kq), p["inv_freq"], positions, amplitude=p["amplitude"])
    v, z = heads(2 * kq, 2 * kq + kv).contiguous(), heads(2 * kq + kv, 2 * kq + 2 * kv).contiguous()
    attend = gdn.linear_attn_step if n == 1 else gdn.linear_attn_prefill
    o, _ = attend(q, k, v, p["g_log"], D ** -0.5, state)
    o = gdn.rmsnorm_gated(o, z, p["norm_out"])
    return gdn.linear(o.transpose(1, 2).reshape(B, n, kv), p["W_out"], None, hidden)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--batch", type=int, default=4)
    ap.add_argument("--hidden", type=int, default=2048)
    ap.add_argument("--prompt", type=int, default=4096)
    ap.add_argument("--steps", type=int, default=32)
    a = ap.parse_args(argv)
    p = make_layer(a.hidden, 16, 32, 128)
    tokens = torch.randn(a.batch, a.prompt, a.hidden, device="cuda").to(torch.bfloat16)
    state = torch.zeros(a.batch, p["Hv"], p["D"], p["D"], device="cuda")
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    forward(p, tokens, state.clone())
    begin.record()
    forward(p, tokens, state)
    end.record()
    torch.cuda.synchronize()
    print("%.1f us a prompt of %d x %d tokens" % (begin.elapsed_time(end) * 1e3, a.batch, a.prompt))

    hidden = tokens[:, -1:].contiguous()
    position = torch.full((1,), a.prompt, dtype=torch.int64, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        forward(p, hidden, state.clone(), position)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hidden.copy_(forward(p, hidden, state, position) * 0.5)  # (halved, so that the stream of many steps stays in range)
        position.add_(1)
    for _ in range(3):
        graph.replay()
    begin.record()
    for _ in range(a.steps):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    if gdn.device_status(0) != 0:
        raise RuntimeError("a kernel reported a wait timeout")
    print("%.1f us a step of %d sequences" % (begin.elapsed_time(end) * 1e3 / a.steps, a.batch))


if __name__ == "__main__":
    main()
