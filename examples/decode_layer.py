"""One token through a whole layer around the gated delta rule: norm, decode block, output
projection, norm behind the residual in 8 bits, gated feed-forward in 8 bits, down projection onto the
residual stream.

    python examples/decode_layer.py [--batch 64] [--hidden 2048] [--ffn 8192] [--steps 32]

runs decode steps from a captured CUDA graph on synthetic weights and prints the time of a step.
(tests/test_decode_layer_gpu.py compares the step with fp64.)
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gated_delta_rule_20_gb300 as gdn  # noqa: E402
import workloads  # noqa: E402


def make_layer(w, ffn, seed=0, device="cuda"):
    """Weights and states of a layer for the decode-block workload ``w`` and a feed-forward of ``ffn`` channels."""
    x = workloads.make_block_inputs(w, device=device)
    gen = torch.Generator().manual_seed(seed)
    rand = lambda n, k: torch.randn(n, k, generator=gen) / k ** 0.5  # noqa: E731
    gate_up = rand(2 * ffn, w.H)
    scale = gate_up.abs().amax(dim=1) / 448.0
    x.update(W_out=rand(w.Hv * w.Dv, w.H).to(torch.bfloat16), W_down=rand(ffn, w.H).to(torch.bfloat16),
             W_gate_up=(gate_up / scale[:, None]).to(torch.float8_e4m3fn), gate_up_scale=scale,
             norm1=1 + 0.1 * torch.randn(w.H, generator=gen), norm2=1 + 0.1 * torch.randn(w.H, generator=gen))
    return {k: v.to(device) if isinstance(v, torch.Tensor) else v for k, v in x.items()}


def decode(p, w, hidden):
    """One token of every sequence: the residual stream ``hidden`` [B, H] bf16 in and out; the conv window and
    the recurrent state of ``p`` are updated in place."""
    y, _, _ = gdn.rmsnorm_residual(hidden, p["norm1"])
    core, _, _ = gdn.decode_block(y.unsqueeze(1), p["W_qkv"], p["W_z"], p["W_a"], p["W_b"], p["conv_weight"],
                                  p["conv_state"], p["A_log"], p["dt_bias"], p["norm_weight"], p["state"], w.Hk, w.Hv, w.Dk,
                                  w.Dv)
    mixed = gdn.linear(core.view(w.B, w.Hv * w.Dv), p["W_out"])
    # the residual's addition, the norm and the rounding to 8 bits in one pass; the new stream beside it
    y8, scale, hidden = gdn.rmsnorm_residual(mixed, p["norm2"], hidden, out_dtype=torch.float8_e4m3fn)
    up = gdn.linear_gated(y8, p["W_gate_up"], weight_layout="nk", x_scale=scale, weight_scale=p["gate_up_scale"])
    return gdn.linear(up, p["W_down"], None, hidden)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--batch", type=int, default=64)
    ap.add_argument("--hidden", type=int, default=2048)
    ap.add_argument("--ffn", type=int, default=8192)
    ap.add_argument("--steps", type=int, default=32)
    a = ap.parse_args(argv)
    w = workloads.DECODE_BLOCK.with_(B=a.batch, H=a.hidden)
    p = make_layer(w, a.ffn)
    hidden = p["hidden"].view(w.B, w.H).clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        decode(p, w, hidden)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hidden.copy_(decode(p, w, hidden) * 0.5)  # (halved, so that the stream of many steps stays in range)
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    for _ in range(3):
        graph.replay()
    begin.record()
    for _ in range(a.steps):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    if gdn.device_status(0) != 0:
        raise RuntimeError("a kernel reported a wait timeout")
    print("%.1f us a step of %d sequences (H = %d, feed-forward %d)" % (begin.elapsed_time(end) * 1e3 / a.steps, w.B, w.H,
                                                                     a.ffn))


if __name__ == "__main__":
    main()
