"""fp32 outputs of bf16 and e4m3 products (``gdn_linear``) keep the accuracy of fp32 sums whatever K is.

The tensor cores truncate a partial sum once in 16 terms, by 0.36 x 2^-23 of it on average.  K is worked off in blocks of
at most 512 (e4m3: 1024), whose sums are added with rounding, so with L = 512 or 1024, u = 2^-24 and B = K / L blocks:

* operands of both signs: the losses of a block are 0.36 x 2^-23 of the sum of its K / 16 partial sums, whose norm is
  sqrt(L^3 / 3) / 16 of a term's, that is 1.55e-9 L of the block's own norm; the B additions are off by u sqrt(B / 6), and 2 u
  for the rest.  Bar of the error's norm: ``1.6e-9 L + (sqrt(B / 6) + 2) u``;
* operands of one sign: 1.34e-9 L of the sum; the additions by u / 3 sqrt(B) on average, 10 u at the most of all.  Bar of
  the largest relative error: ``1.5e-9 L + 10 u``."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f8": torch.float8_e4m3fn}


@pytest.fixture(scope="module")
def gdn():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gated_delta_rule_20_gb300 as g
    g.lib()
    yield g
    assert g.device_status(0) == 0


def _scaled(t, dtype):
    if dtype == "bf16":
        return t.bfloat16(), None
    s = t.abs().amax(1) / 448
    return (t / s[:, None]).to(DT["f8"]), s


def _operands(M, n, K, dtype, kind):
    gen = torch.Generator("cuda").manual_seed(K + M)
    normal = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    x, w = normal(M, K), normal(n, K)
    if kind == "one sign":
        x, w = x.abs().clamp(0.5, 2), w.abs().clamp(0.5, 2)
    if kind == "channels":  # channels of very unequal size, whose products differ in their lowest bits
        x, w = x * torch.exp(1.5 * normal(1, K)), w * torch.exp(normal(1, K))
    return _scaled(x, dtype) + _scaled(w, dtype)


def _f64(t, s):
    return t.double() if s is None else t.float().double() * s.double()[:, None]


def _run(gdn, M, N, K, dtype, layout, kind, gated=False):
    x, xs, w, ws = _operands(M, 2 * N if gated else N, K, dtype, kind)
    wd = w if layout == "nk" else w.t().contiguous()
    call = gdn.linear_gated if gated else gdn.linear
    out = call(x, wd, weight_layout=layout, x_scale=xs, weight_scale=ws, activation="none", out_dtype=torch.float32)
    torch.cuda.synchronize()
    ref = _f64(x, xs) @ _f64(w, ws).t()
    L = 1024 if dtype == "f8" else 512
    return out.double(), ref, L


# long and short K on every kernel; K of one block, of a whole number of blocks, of ragged ones and with a ragged last slab
SHAPES = [(2048, 1024, 512, "bf16", "nk"), (2048, 1024, 576, "bf16", "nk"), (2048, 1024, 2048, "bf16", "kn"), (1000, 1016, 4104, "bf16", "nk"),
          (2048, 1024, 8192, "bf16", "nk"), (4100, 700, 16384, "bf16", "nk"), (768, 2048, 8192, "bf16", "kn"), (256, 512, 16384, "bf16", "nk"),
          (1, 2048, 32768, "bf16", "nk"), (64, 300, 5000, "bf16", "kn"), (33, 4096, 8200, "bf16", "nk"), (17, 40000, 2048, "bf16", "nk"),
          (130, 20000, 1500, "bf16", "kn"), (513, 1001, 9001, "bf16", "nk"), (96, 96, 70000, "bf16", "nk"),
          (2048, 1024, 8192, "f8", "nk"), (2048, 1024, 32768, "f8", "nk"), (768, 2048, 16384, "f8", "nk"), (64, 512, 65536, "f8", "nk"),
          (9, 3000, 16400, "f8", "nk"), (777, 1003, 4097, "f8", "nk")]


@pytest.mark.parametrize("M,N,K,dtype,layout", SHAPES)
@pytest.mark.parametrize("kind", ["both signs", "channels"])
def test_operands_of_both_signs(gdn, M, N, K, dtype, layout, kind):
    out, ref, L = _run(gdn, M, N, K, dtype, layout, kind)
    error = ((out - ref).norm() / ref.norm()).item()
    assert error <= 1.6e-9 * min(L, K) + ((K / L / 6) ** 0.5 + 2) * U, "%.3g" % error


@pytest.mark.parametrize("M,N,K,dtype,layout", SHAPES)
def test_operands_of_one_sign(gdn, M, N, K, dtype, layout):
    out, ref, L = _run(gdn, M, N, K, dtype, layout, "one sign")
    error = (out / ref - 1).abs().max().item()
    assert error <= 1.5e-9 * min(L, K) + 10 * U, "%.3g" % error


@pytest.mark.parametrize("M,N,K,dtype,layout", [(2048, 512, 8192, "bf16", "nk"), (300, 1000, 4104, "bf16", "kn"), (40, 264, 16384, "bf16", "nk"),
                                                (1500, 520, 16384, "f8", "nk"), (5, 130, 40000, "f8", "nk")])
def test_gated(gdn, M, N, K, dtype, layout):
    """Both factors of a gated product are such sums (bar: twice theirs, of the product's norm)."""
    out, ref, L = _run(gdn, M, N, K, dtype, layout, "both signs", gated=True)
    ref = ref[:, :N] * ref[:, N:]
    error = ((out - ref).norm() / ref.norm()).item()
    assert error <= 2 * (1.6e-9 * L + ((K / L / 6) ** 0.5 + 2) * U), "%.3g" % error


@pytest.mark.parametrize("M,N,K", [(2048, 1024, 8192), (300, 1000, 4104), (40, 300, 16384), (700, 40000, 1024), (5000, 3000, 1600)])
@pytest.mark.parametrize("gated", [False, True])
def test_epilogue_and_repeats(gdn, M, N, K, gated):
    """Many tiles a CTA pair, with bias, activation and residual behind several blocks of K, bit for bit the same each
    time, and next to the same call with bf16 outputs."""
    gen = torch.Generator("cuda").manual_seed(M)
    n = 2 * N if gated else N
    x = torch.randn(M, K, generator=gen, device="cuda").bfloat16()
    w = (torch.randn(n, K, generator=gen, device="cuda") / K ** 0.5).bfloat16()
    b, r = torch.randn(n, generator=gen, device="cuda"), torch.randn(M, N, generator=gen, device="cuda").bfloat16()
    call = gdn.linear_gated if gated else gdn.linear
    f = lambda dt: call(x, w, b, r.to(dt), activation="silu", weight_layout="nk", out_dtype=dt)  # noqa: E731
    out, low = f(torch.float32), f(torch.bfloat16)
    a = x.double() @ w.double().t() + b.double()
    act = a[:, :N] / (1 + torch.exp(-a[:, :N]))
    ref = (act * a[:, N:] if gated else act) + r.double()
    assert ((out.double() - ref).norm() / ref.norm()).item() < 2e-6
    assert ((low.double() - ref).norm() / ref.norm()).item() < 2.0 ** -8
    for _ in range(4):
        assert torch.equal(f(torch.float32), out)
