"""fp32 products by bf16 parts at the longest K that they run for (3072 to 4096): the sums of x1 w1 lie in accumulators of at
most 1024 of K.  The bar is that of sums of one sign in ``test_linear_parts_gpu`` for that share: the largest relative error
is at most ``1.5e-9 x 1024 + 4 u``, u = 2^-24 (twice that for the two factors of a gated product)."""
import pytest

torch = pytest.importorskip("torch")

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


@pytest.mark.parametrize("M,N,K", [(1024, 1024, 4096), (2048, 2048, 4096), (700, 1500, 4001), (1500, 1030, 3500), (64, 2048, 4096),
                                   (33, 5000, 3136), (200, 4100, 4090)])
@pytest.mark.parametrize("layout", ["kn", "nk"])
@pytest.mark.parametrize("gated", [False, True])
def test_sums_of_one_sign(gdn, M, N, K, layout, gated):
    gen = torch.Generator("cuda").manual_seed(K)
    x = torch.rand(M, K, generator=gen, device="cuda") + 0.5
    w = torch.rand(2 * N if gated else N, K, generator=gen, device="cuda") + 0.5
    wd = w if layout == "nk" else w.t().contiguous()
    call = gdn.linear_gated if gated else gdn.linear
    out = call(x, wd, activation="none", weight_layout=layout).double()
    ref = x.double() @ w.double().t()
    ref = ref[:, :N] * ref[:, N:] if gated else ref
    assert not torch.equal(out, call(x, wd, activation="none", weight_layout=layout, force_ffma=True).double())
    worst = (out / ref - 1).abs().max().item()
    assert worst <= (2 if gated else 1) * (1.5e-9 * 1024 + 4 * U), "%.3g" % worst
