"""linear_attn_prefill just below the magnitudes from which its sums pass their type's range (see gdn.h)."""

import pytest
import torch

import gated_delta_rule_20_gb300 as gdn

pytestmark = pytest.mark.gpu


def one_key(c, size, share, dtype, at=64):
    """Tokens whose log-decays add up to c at token `at`, which alone has a key; q . k = size ** share there and behind it, and
    v the rest of size: o = size from that token on (nothing decays any more)."""
    H, S, D = 2, 200, 16
    q, k, v = (torch.zeros(1, H, S, D, dtype=torch.float64) for _ in range(3))
    q[..., 3] = k[:, :, at, 3] = size ** (share / 2)
    v[:, :, at] = size ** (1 - share)
    q, k, v = (x.to(dtype) for x in (q, k, v))
    g = torch.zeros(1, H, S)
    g[:, :, :at] = c / at
    want = q[:, :, at:, 3].double() * k[:, :, at, None, 3].double() * v[:, :, at, None, 0].double()
    return [x.cuda() for x in (q, k, v, g)], want


@pytest.mark.parametrize("share", [0.0, 0.5, 1.0])
@pytest.mark.parametrize("c, size", [(-64, 5.1e10), (-200, 5.1e10), (-20, 6.6e29), (0, 3.2e38)])
def test_below_the_range_of_the_tensor_cores(c, size, share):
    """3.4e38 e^max(c, -64) is 5.45e10, 7.0e29 and 3.4e38; roundings of the operands (2^-8 each) leave sizes below these.  Scores and
    outputs are rounded to bf16 once each, 2^-7 + 2^-16 of the output together, and e^64 is off by less than 2^-16."""
    x, want = one_key(c, size, share, torch.bfloat16)
    out, _ = gdn.linear_attn_prefill(*x, 1.0)
    assert gdn.device_status(0) == 0
    got = out[:, :, 64:128].double().cpu()   # (the key's chunk)
    assert bool(torch.isfinite(got).all())
    off = (got / want[:, :, :64, None] - 1).abs().max()
    assert off <= 2.0 ** -7 + 2.0 ** -15, "off by %.3g" % off


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("c, size", [(-64, 1e12), (-200, 1e30), (-20, 1e34), (-7.9 * 79 / 15, 9e34), (0, 9e34)])
def test_below_the_range_of_the_fma_units(c, size, dtype):
    """Far past the tensor cores' range; the key is its block's last token, behind decays of e^-7.9 there at the most, as what
    passes e^-8 is taken token by token.  Three products and two exponentials of 2 steps each: 11 * 2^-24; bf16: the output's
    2^-8 as well."""
    x, want = one_key(c, size, 0.5, dtype, at=79)
    out, _ = gdn.linear_attn_prefill(*x, 1.0, force_ffma=True, single_pass=True)
    got = out[:, :, 79:].double().cpu()
    off = (got / want[..., None] - 1).abs().max()
    assert off <= 11 * 2.0 ** -24 + (2.0 ** -8 if dtype is torch.bfloat16 else 0), "off by %.3g" % off
