"""fp32 products on the tensor cores by bf16 parts (``gdn_linear``): that the parts are what ran, over which range
of operands, and how far they are from the products in 64 bits.

Two bars, with u = 2^-24:

* Operands of both signs.  A partial sum of k products is about sqrt(k) of a term, and each of at most K additions is
  off by u / sqrt 3 of it (a rounding; the tensor cores' truncations come once in 16 terms), so the norm of the error is
  at most u sqrt(K / 6) of the norm of the products; 8 u more for the parts that are left out and the joins:
  ``(sqrt(K / 6) + 8) u``.  Without the third parts the error is about 2^-18 of every term, 4e-6 of the norm, which
  ``test_the_bar_sees_a_missing_part`` shows for every shape here.
* Operands of one sign.  A truncation every 16 terms loses on average 0.36 x 2^-23 of the partial sum, that is
  0.36 x 2^-23 / 32 = 1.34e-9 of the sum for every term of an accumulator's share of K; the bar takes 1.5e-9 and 4 u for
  the joins: ``1.5e-9 share + 4 u``, share = 704 of K up to K = 2112, a third of K beyond."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

U = 2.0 ** -24
gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def gdn():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gated_delta_rule_20_gb300 as g
    g.lib()
    yield g
    assert g.device_status(0) == 0


def _operands(M, N, K, seed):
    gen = torch.Generator().manual_seed(seed)
    return torch.randn(M, K, generator=gen), torch.randn(N, K, generator=gen) / K ** 0.5


def _linear(gdn, x, w, layout="nk", **kw):
    """x [M, K], w [N, K] on the host; the product in ``layout`` on the GPU, and what it is in 64 bits."""
    wd = (w if layout == "nk" else w.t().contiguous()).cuda()
    out = gdn.linear(x.cuda(), wd, weight_layout=layout, **kw)
    torch.cuda.synchronize()
    return out.cpu()


def _exact(x, w):
    return x.double().numpy() @ w.double().numpy().T


def _norm_error(out, ref):
    return np.linalg.norm(out.double().numpy() - ref) / np.linalg.norm(ref)


def _norm_bar(K):
    return ((K / 6) ** 0.5 + 8) * U


SHAPES = [(333, 1030, 770), (1000, 1001, 1003), (600, 515, 1000), (64, 4096, 1024), (32, 2048, 4096), (3000, 700, 130),
          (1024, 1024, 2048)]


def _parts(t):
    a = t.bfloat16().float()
    b = (t - a).bfloat16().float()
    return a.double().numpy(), b.double().numpy(), (t - a - b).bfloat16().double().numpy()


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_the_bar_sees_a_missing_part(M, N, K):
    """In 64 bits: three parts stay far inside the bar, two do not, and neither does a product with the third part of
    one operand left out."""
    x, w = _operands(min(M, 64), min(N, 64), K, seed=K)
    ref, (x1, x2, x3), (w1, w2, w3) = _exact(x, w), _parts(x), _parts(w)
    two = x1 @ w1.T + x1 @ w2.T + x2 @ w1.T
    six = two + x2 @ w2.T + x1 @ w3.T + x3 @ w1.T
    error = lambda p: np.linalg.norm(p - ref) / np.linalg.norm(ref)  # noqa: E731
    assert error(six) < 0.1 * _norm_bar(K)
    assert error(two) > _norm_bar(K) and error(six - x3 @ w1.T) > _norm_bar(K) and error(six - x1 @ w3.T) > _norm_bar(K)


@gpu
@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("layout", ["kn", "nk"])
def test_error_of_products_of_both_signs(gdn, M, N, K, layout):
    assert 2 * M * N * K >= 3e8
    x, w = _operands(M, N, K, seed=K)
    out = _linear(gdn, x, w, layout)
    assert not torch.equal(out, _linear(gdn, x, w, layout, force_ffma=True))  # the parts are what ran
    assert _norm_error(out, _exact(x, w)) <= _norm_bar(K)


@gpu
@pytest.mark.parametrize("M,N,K", [(256, 1024, 704), (256, 512, 2048), (72, 1024, 2048), (1024, 1024, 2048), (128, 512, 4096), (512, 1024, 4096)])
def test_error_of_sums_of_one_sign(gdn, M, N, K):
    gen = torch.Generator().manual_seed(K)
    x, w = torch.rand(M, K, generator=gen) + 0.5, torch.rand(N, K, generator=gen) + 0.5
    out, ref = _linear(gdn, x, w), _exact(x, w)
    assert not torch.equal(out, _linear(gdn, x, w, force_ffma=True))
    share = min(K, max(704, K / 3))
    worst = np.abs(out.double().numpy() / ref - 1).max()
    assert worst <= 1.5e-9 * share + 4 * U, "%.3g" % worst


@gpu
@pytest.mark.parametrize("M,N,K,layout", [(333, 1030, 770, "kn"), (64, 2048, 2048, "nk")])
@pytest.mark.parametrize("ax,aw", [(60, 0), (0, 60), (50, 50), (-60, 0), (0, -60), (60, -90), (-40, 10)])
def test_powers_of_two_keep_the_bits(gdn, M, N, K, layout, ax, aw):
    """Operands scaled by powers of two, inside the range that runs by parts: the same bits, scaled (the FFMA kernel
    would give others)."""
    x, w = _operands(M, N, K, seed=5)
    base = _linear(gdn, x, w, layout)
    assert not torch.equal(base, _linear(gdn, x, w, layout, force_ffma=True))
    out = _linear(gdn, x * 2.0 ** ax, w * 2.0 ** aw, layout)
    assert torch.equal(out, base * 2.0 ** (ax + aw))


@gpu
@pytest.mark.parametrize("M,N,K,layout", [(64, 1024, 4096, "nk"), (200, 512, 2048, "kn"), (1024, 1024, 4096, "nk"), (700, 2048, 2048, "kn")])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_sums_past_the_range_of_operands_under_2_to_63(gdn, M, N, K, layout, sign):
    """Both operands just under 2^63, where the second parts are negative: infinities of the sum's sign, not NaN."""
    v = 2.0 ** 62 * (1 + 126.6 / 128)
    out = _linear(gdn, torch.full((M, K), v), torch.full((N, K), sign * v), layout)
    assert (out == sign * float("inf")).all()


@gpu
def test_largest_sums_in_range(gdn):
    """Sums up to a quarter of the largest fp32 number are finite and as near as any."""
    M, N, K = 64, 1024, 4096
    x, w = torch.full((M, K), 1.9 * 2.0 ** 56), torch.full((N, K), 1.9 * 2.0 ** 56)
    x[::2] *= -1
    out, ref = _linear(gdn, x, w), _exact(x, w)
    assert (np.abs(out.double().numpy() / ref - 1) <= 1.5e-9 * K / 3 + 4 * U).all()


@gpu
@pytest.mark.parametrize("M,N,K,layout", [(333, 1030, 770, "kn"), (64, 2048, 2048, "nk")])
@pytest.mark.parametrize("ax,aw", [(-118, 0), (0, -115), (-118, 60), (60, -118), (-52, -56)])
def test_operands_that_are_tiny_whole(gdn, M, N, K, layout, ax, aw):
    """Operands whose parts would pass below the least bf16 number keep the accuracy of fp32 sums."""
    x, w = _operands(M, N, K, seed=7)
    x, w = x * 2.0 ** ax, w * 2.0 ** aw
    assert _norm_error(_linear(gdn, x, w, layout), _exact(x, w)) <= _norm_bar(K)


@gpu
@pytest.mark.parametrize("which", ["x", "weight"])
def test_tiny_rows_among_others(gdn, which):
    """Rows of x (or columns of the weight) of 2^-100 to 2^-140 beside ordinary ones: what an element has below 2^-133 may
    be lost, at most 2^-133 of every element, and no more.  (The other operand is 2^40, so that the sums are ordinary
    numbers.)"""
    M, N, K = 128, 1024, 1500
    x, w = _operands(M, N, K, seed=11)
    w = w * K ** 0.5
    scale = torch.zeros(M if which == "x" else N)
    scale[:30] = torch.tensor([-100.0, -110, -115, -120, -125, -130] * 5)
    scale[30] = -140
    tiny = (x if which == "x" else w) * 2.0 ** scale[:, None]
    x, w = (tiny, w * 2.0 ** 40) if which == "x" else (x * 2.0 ** 40, tiny)
    out, ref = _linear(gdn, x, w).double().numpy(), _exact(x, w)
    assert not torch.equal(_linear(gdn, x, w), _linear(gdn, x, w, force_ffma=True))
    s = np.abs(x.double().numpy()) @ np.abs(w.double().numpy()).T
    lost = np.abs(w.double().numpy()).sum(1)[None, :] if which == "x" else np.abs(x.double().numpy()).sum(1)[:, None]
    assert (np.abs(out - ref) <= (8 * K ** 0.5 + 8) * U * s + 2.0 ** -133 * lost).all()


@gpu
@pytest.mark.parametrize("which", ["x", "weight", "both"])
def test_operands_of_zeros(gdn, which):
    x, w = _operands(64, 2048, 2048, seed=3)
    if which != "weight":
        x.zero_()
    if which != "x":
        w.zero_()
    assert (_linear(gdn, x, w) == 0).all()


@gpu
@pytest.mark.parametrize("gated", [False, True])
def test_the_largest_numbers_go_to_the_ffma_kernel(gdn, gated):
    """One row of the largest fp32 numbers: the whole product is the FFMA kernel's, bit for bit."""
    x, w = _operands(128, 1024, 1500, seed=2)
    x[2] = 3.4028235e38 * x[2].sign()
    x, w = x.cuda(), (w * 2.0 ** -20).cuda()
    call = gdn.linear_gated if gated else gdn.linear
    a, b = (call(x, w, activation="none", weight_layout="nk", force_ffma=f) for f in (False, True))
    assert torch.equal(a.view(torch.int32), b.view(torch.int32))
