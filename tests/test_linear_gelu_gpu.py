"""GELU of fp32 outputs at fp32's relative error, tails included, through every kernel of ``gdn_linear``.

The bar, with u = 2^-24: gelu(v) = v Phi(v).  For v < 0 an error of r in z = v / sqrt 2 moves Phi by (2 z^2 + 1) r = (v^2 + 1) r
of itself at most; three roundings on the way there and 12 more for the fit, the exponential, the quotient and the
products: (3 (v^2 + 1) + 12) u of the value.  The operands are chosen so that every sum is exact."""
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
    yield g
    assert g.device_status(0) == 0


def _gelu(v):
    """v Phi(v) in 64 bits, Phi from erfc, which does not cancel."""
    import math
    return v * np.vectorize(lambda t: 0.5 * math.erfc(-t / math.sqrt(2)), otypes=[np.float64])(v)


def _check(got, v, factor=1.0):
    v = v.double().numpy()
    ref = _gelu(v)
    assert np.allclose(ref, layer.activation("gelu", v), rtol=0, atol=1e-14)
    got = got.detach().cpu().double().numpy()
    bad = np.abs(got - factor * ref) > (3 * (v * v + 1) + 12) * U * np.abs(factor * ref)
    assert not bad.any(), "worst at v = %r" % v[bad][:5]


def test_over_its_range(gdn):
    v = torch.cat([torch.linspace(-12, 12, 60001), torch.logspace(-20, 1, 4000), -torch.logspace(-20, 1, 4000)])
    v = v[v != 0]
    got = gdn.linear(v.cuda()[:, None].contiguous(), torch.ones(1, 1, device="cuda"), activation="gelu")
    _check(got.flatten(), v)


# few rows, one tile and many of both FFMA kernels; the three tensor-core kernels; fp32 by parts on two of them
@pytest.mark.parametrize("M,N,K,dtype,layout,ffma", [
    (1, 64, 64, "f32", "nk", False), (9, 200, 130, "bf16", "kn", True), (100, 130, 64, "f32", "kn", False),
    (3000, 2000, 16, "f32", "nk", False), (3, 256, 512, "bf16", "nk", False), (64, 300, 2048, "bf16", "kn", False),
    (4096, 1001, 64, "bf16", "nk", False), (384, 2048, 4096, "bf16", "kn", False), (1500, 640, 256, "f8", "nk", False),
    (64, 2048, 2048, "f32", "nk", False), (1024, 1024, 512, "f32", "kn", False)])
@pytest.mark.parametrize("gated", [False, True])
def test_every_kernel(gdn, M, N, K, dtype, layout, ffma, gated):
    dt = {"f32": torch.float32, "bf16": torch.bfloat16, "f8": torch.float8_e4m3fn}[dtype]
    v = -12 * torch.rand(M, generator=torch.Generator().manual_seed(M)) ** 1.5
    v = (v if dtype != "f8" else v.clamp(max=-0.02)).to(dt)
    v[M // 2] = 2.5
    x = torch.zeros(M, K)
    x[:, 3], x[:, 5] = v.float(), 1.0
    w = torch.zeros(2 * N if gated else N, K)
    w[:N, 3] = 1.0
    w[N:, 5] = -0.5
    w = (w if layout == "nk" else w.t()).contiguous().to(dt).cuda()
    kw = dict(x_scale=torch.ones(M, device="cuda"), weight_scale=torch.ones(2 * N if gated else N, device="cuda")) if dtype == "f8" else {}
    call = gdn.linear_gated if gated else gdn.linear
    got = call(x.to(dt).cuda(), w, activation="gelu", weight_layout=layout, out_dtype=torch.float32, force_ffma=ffma, **kw)
    torch.cuda.synchronize()
    assert got.shape == (M, N) and (got == got[:, :1]).all()
    _check(got[:, 0], v.float(), -0.5 if gated else 1.0)


def test_silu_over_its_range(gdn):
    """The header's bound of silu: (5 + 1.2 |v|) 2^-23 of the value for v > -87 (the fast exponential's error grows with
    its argument)."""
    v = torch.cat([torch.linspace(-86.9, 88, 60001), torch.logspace(-20, 1, 4000), -torch.logspace(-20, 1, 4000)])
    v = v[v != 0]
    got = gdn.linear(v.cuda()[:, None].contiguous(), torch.ones(1, 1, device="cuda"), activation="silu")
    got, v = got.flatten().cpu().double().numpy(), v.double().numpy()
    ref = v / (1 + np.exp(-v))
    assert (np.abs(got - ref) <= (5 + 1.2 * np.abs(v)) * 2.0 ** -23 * np.abs(ref)).all()
