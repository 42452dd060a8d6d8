"""The example layer (examples/decode_layer.py): norm, decode block, output projection, norm in 8 bits,
gated feed-forward and down projection together, against the same step in fp64.

The bar: the e4m3 rounding of the second norm is off by at most 2^-4 of a value and 2^-4 / sqrt(3) in the
mean of squares (3.6e-2); it reaches the output through the feed-forward only, as a relative error of
that branch: both of its factors are products of the same rounded row, 2 x 3.6e-2 of it at the most.
The output is the stream plus that branch, and the bf16 roundings and the block's own bar (1e-2) add to it:
relative L2 <= 1e-2 + 7.2e-2 |branch| / |output|."""
import os
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import workloads  # noqa: E402
from oracle import decode_block as block  # noqa: E402
from oracle import layer  # noqa: E402

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def reference(p, w, hidden):
    """The same step in fp64 (no rounding between the operators)."""
    y, _ = layer.rmsnorm_residual(hidden, p["norm1"])
    core, _, _ = block.decode_block(y[:, None, :], p["W_qkv"], p["W_z"], p["W_a"], p["W_b"], p["conv_weight"], p["conv_state"],
                                    p["A_log"], p["dt_bias"], p["norm_weight"], p["state"], w.Hk, w.Hv, w.Dk, w.Dv)
    mixed = layer.linear(core.reshape(w.B, -1), p["W_out"])
    y, h = layer.rmsnorm_residual(mixed, p["norm2"], hidden)
    up = layer.linear(y, p["W_gate_up"].float(), act="silu", x_scale=torch.ones(w.B), weight_scale=p["gate_up_scale"],
                      layout="nk", gated=True)
    return layer.linear(up, p["W_down"], residual=h)


@pytest.mark.parametrize("B,H,ffn", [(1, 256, 512), (5, 512, 1000), (64, 2048, 1024)])
def test_decode_layer_against_fp64(B, H, ffn):
    import decode_layer as ex
    w = workloads.DECODE_BLOCK.with_(B=B, H=H, Hk=2, Hv=8, Dk=64, Dv=64, seed=B)
    p = ex.make_layer(w, ffn, seed=B)
    hidden = p["hidden"].view(B, H).clone()
    ref = reference(p, w, hidden)
    # the feed-forward's part of the output: what the down projection adds to the stream
    zero = dict(p, W_down=torch.zeros_like(p["W_down"]))
    branch = ref - reference(zero, w, hidden)
    got = ex.decode(p, w, hidden).double().cpu().numpy()
    off = np.linalg.norm(got - ref) / np.linalg.norm(ref)
    assert np.isfinite(got).all()
    assert off <= 1e-2 + 7.2e-2 * np.linalg.norm(branch) / np.linalg.norm(ref), off
