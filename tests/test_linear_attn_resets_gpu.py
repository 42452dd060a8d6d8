"""Decays of linear_attn_prefill on the tensor cores where tokens that start anew (g_log of -infinity, counted as -100) make
large sums beside small ones: the small ones keep their accuracy."""
import math

import numpy as np
import pytest
import torch

import gated_delta_rule_20_gb300 as gdn

pytestmark = pytest.mark.gpu


def test_weak_decays_in_front_of_many_resets():
    """Tokens in front of resets in the same 32: o_i = e^{c_i} S_r exactly, but for the output's rounding, as q picks one row of a
    state of bf16 values and k is zero.  Allowed: half a step of the output's binade; and 2^-19 of it for c_i (sums of 16 log-decays
    of 0.001 and a product: below 2^-23), the exponential (2^-22), and the products by it and by scale (2^-24 each)."""
    H, S, Dk, Dv = 64, 32, 16, 128
    gen = torch.Generator().manual_seed(3)
    g = -0.001 * torch.rand(1, H, S, generator=gen)
    g[:, :, 16:] = -math.inf
    row = torch.randint(0, Dk, (1, H, S), generator=gen)
    q = torch.nn.functional.one_hot(row, Dk).bfloat16()
    k, v = torch.zeros(1, H, S, Dk).bfloat16(), torch.randn(1, H, S, Dv, generator=gen).bfloat16()
    state = torch.randn(1, H, Dk, Dv, generator=gen).bfloat16().float()
    out, _ = gdn.linear_attn_prefill(*(x.cuda() for x in (q, k, v, g)), 1.0, state.cuda())
    assert gdn.device_status(0) == 0
    c = g[:, :, :16].double().cumsum(-1)
    want = (torch.gather(state, 2, row[..., None].expand(1, H, S, Dv))[:, :, :16].double() * c.exp()[..., None]).numpy()
    got = out[:, :, :16].double().cpu().numpy()
    half = 2.0 ** (np.floor(np.log2(np.abs(want))) - 8)
    off = np.abs(got - want) - half - 2.0 ** -19 * np.abs(want)
    assert off.max() <= 0, "%d of %d off by up to 2^%.1f more" % ((off > 0).sum(), off.size, np.log2((off / np.abs(want)).max()))


def test_weak_decays_behind_a_block_of_resets():
    """Scores of a query and a key in different 32s behind a whole 32 of resets.  Score and output are rounded to bf16 once
    each, by 2^-8 of them at the most; over 2^19 unlike products such errors add up to nothing.  Allowed to the mean: what Hoeffding's
    inequality gives for a chance of 1e-9, (b - a) sqrt(ln(2e9) / 2N) with b - a = 2^-6, 7.1e-5, and 2^-15 for the roundings'
    own bias (2^-16) and the exponentials'."""
    B, H, S, D, j = 64, 256, 128, 8, 70
    gen = torch.Generator(device="cuda").manual_seed(5)
    bf = lambda *s: (1 + torch.rand(*s, generator=gen, device="cuda")).bfloat16()  # noqa: E731
    g = torch.full((B, H, S), -math.inf, device="cuda")
    for lo, x in ((32, 0.072), (64, 0.0311), (96, 0.01)):
        g[:, :, lo:lo + 32] = -x
    q, k, v = (torch.zeros(B, H, S, D, dtype=torch.bfloat16, device="cuda") for _ in range(3))
    q[..., 0], k[:, :, j, 0], v[:, :, j] = bf(B, H, S), bf(B, H), 1.0
    out, _ = gdn.linear_attn_prefill(q, k, v, g, 1.0)
    assert gdn.device_status(0) == 0
    c = g[:, :, j + 1:].double().cumsum(-1)[:, :, 95 - j:]
    want = q[:, :, 96:, 0].double() * k[:, :, j, None, 0].double() * c.exp()
    off = out[:, :, 96:, 0].double() / want - 1
    assert bool((off.abs() <= 2.0 ** -7 + 2.0 ** -14).all())
    n = off.numel()
    assert n == 1 << 19
    most = 2.0 ** -6 * math.sqrt(math.log(2e9) / (2 * n)) + 2.0 ** -15
    assert abs(float(off.mean())) <= most, "a mean of %.3g, at most %.3g allowed" % (float(off.mean()), most)
