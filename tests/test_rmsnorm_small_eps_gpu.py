"""``gdn_rmsnorm_residual`` in 8 bits where the norm's factor over the row's scale passes fp32's range: a small eps,
and rows of zeros or of very small numbers, whose scale is the least one."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import layer  # noqa: E402

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def gdn():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gated_delta_rule_20_gb300 as g
    g.lib()
    return g


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("eps", [1e-12, 1e-20, 1e-30])
@pytest.mark.parametrize("D", [128, 2048, 2049, 8192, 16392])
def test_rows_of_zeros(gdn, D, eps, dtype):
    """Zeros and the least scale, next to a row like any other (formula: 0 / sqrt(eps) = 0)."""
    x = torch.zeros(3, D, dtype=dtype, device="cuda")
    x[1] = torch.randn(D, generator=torch.Generator().manual_seed(D)).to(dtype).cuda()
    q, s, _ = gdn.rmsnorm_residual(x, torch.ones(D, device="cuda"), out_dtype=torch.float8_e4m3fn, eps=eps)
    q, s = q.float().cpu(), s.cpu()
    assert (q[0] == 0).all() and (q[2] == 0).all()
    assert s[0] == s[2] == torch.tensor(1e-30) / 448
    y, _ = layer.rmsnorm_residual(x.cpu(), np.ones(D), None, eps)
    ref = layer.row_scale(y)
    assert abs(float(s[1]) - ref[1]) <= (D / 64 + 30) * U * ref[1]
    assert (np.abs(q[1].double().numpy() - y[1] / ref[1]) <= 2.0 ** -4 * np.abs(y[1] / ref[1]) + 2.0 ** -9).all()


@pytest.mark.parametrize("D", [128, 2049, 4096, 16392])
def test_rows_of_very_small_numbers(gdn, D):
    """|y| of 1e-33 to 1e-31, under the least maximum that a scale is made from, with 1 / sqrt(eps) = 1e6."""
    h = 10.0 ** torch.linspace(-37, -36, D) * (1e-1 ** torch.arange(2.0))[:, None] * torch.tensor([1.0, -1.0])[:, None]
    w = torch.full((D,), 0.5)
    h[1] *= 1.0  # the second row: subnormal numbers
    q, s, _ = gdn.rmsnorm_residual(h.cuda(), w.cuda(), out_dtype=torch.float8_e4m3fn, eps=1e-12)
    y, _ = layer.rmsnorm_residual(h, w, None, 1e-12)
    scale = layer.row_scale(y)
    assert (scale == 1e-30 / 448).all() and (np.abs(s.cpu().double().numpy() / scale - 1) <= 2.0 ** -20).all()
    v = y / scale[:, None]
    # half a step of e4m3; the products h w and h w / sqrt(eps) of subnormal numbers: 2^-149 x 1e6 / scale = 6e-7
    assert (np.abs(q.float().cpu().double().numpy() - v) <= np.maximum(2.0 ** -4 * np.abs(v), 2.0 ** -10) * (1 + 1e-4) + 1e-6).all()
