"""GPU parity of ``gdn_rmsnorm_residual`` with the fp64 oracle ``oracle.layer``.

Bars, each derived from what the kernel rounds (u = 2^-24, fp32's unit roundoff):

* the fp32 row: the sum of squares adds at most D / 32 + 40 terms in a row (relative error
  (D / 32 + 40) u, halved by the root), and rsqrt (2 ulp), the two products and the addition of the
  residual add under 8 u: rel = (D / 64 + 28) u + the output's own rounding;
* bf16 outputs: 2^-8 more; the smallest normal numbers add an absolute 1e-38;
* e4m3: v = y / scale is off by at most half a step, max(2^-4 |v|, 2^-10), and by 2 rel |v|.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import layer  # noqa: E402

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def gdn():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gated_delta_rule_20_gb300 as g
    g.lib()
    return g


def _draw(rows, D, dtype, seed, residual=True):
    gen = torch.Generator().manual_seed(seed)
    width = torch.exp(torch.randn(D, generator=gen))
    x = (torch.randn(rows, D, generator=gen)).to(DT[dtype]).cuda()
    r = (width * torch.randn(rows, D, generator=gen)).to(DT[dtype]).cuda() if residual else None
    return x, (1 + 0.2 * torch.randn(D, generator=gen)).cuda(), r


def _f64(t):
    return t.detach().cpu().double().numpy()


def _check(x, w, r, out, scale, h, eps=1e-6):
    D = x.shape[-1]
    rel = (D / 64 + 28) * U
    y, hr = layer.rmsnorm_residual(x, w, r, eps)
    near = lambda got, ref, e, what: np.testing.assert_array_less(  # noqa: E731
        np.abs(_f64(got) - ref), e * np.abs(ref) + 1e-38, err_msg=what)
    step = 2.0 ** -8 if x.dtype == torch.bfloat16 else U
    if h is not None:
        near(h, hr, step + 2 * U, "residual_out")
    if scale is None:
        near(out, y, step * (1 + rel) + rel, "out")
        return
    s = layer.row_scale(y)
    near(scale, s, rel + 2 * U, "scale")
    v = y / s[..., None]
    d = np.abs(_f64(out.float()) - v)
    assert (d <= np.maximum(2.0 ** -4 * np.abs(v), 2.0 ** -10) * (1 + 1e-9) + 2 * rel * np.abs(v)).all(), "out (e4m3)"


# rows of one to many pieces of 16 bytes and of none (odd D), every group size, one row to more
# than the grid holds at once
SHAPES = [(1, 1), (3, 2), (2, 7), (5, 8), (1, 64), (9, 72), (33, 256), (4, 264), (7, 512), (3, 1000), (2, 1024), (6, 1032),
          (1, 2048), (2, 2051), (5, 4096), (3, 4104), (2, 8192), (2, 8200), (3, 16384), (2, 16392), (1, 32768), (2, 32767),
          (0, 128), (5000, 136), (3001, 2048)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("rows,D", SHAPES)
def test_shapes(gdn, rows, D, dtype, f8):
    x, w, r = _draw(rows, D, dtype, seed=rows * 7 + D)
    for res in (r, None):
        out, scale, h = gdn.rmsnorm_residual(x, w, res, out_dtype=torch.float8_e4m3fn if f8 else None)
        torch.cuda.synchronize()
        assert (scale is not None) == f8 and (h is not None) == (res is not None)
        assert out.shape == x.shape and out.dtype == (torch.float8_e4m3fn if f8 else DT[dtype])
        if rows:
            _check(x, w, res, out, scale, h)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [128, 200, 4096, 16384])
@pytest.mark.parametrize("f8", [False, True])
def test_unaligned_pointers(gdn, D, dtype, f8):
    """Every operand one element past a 16-byte boundary; guard bands around the outputs."""
    x, w, r = _draw(5, D, dtype, seed=D)

    def shifted(t):
        b = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
        b[1:].view(t.shape).copy_(t)
        return b[1:].view(t.shape)
    odt = torch.float8_e4m3fn if f8 else DT[dtype]
    ob = torch.zeros(x.numel() + 2, device="cuda").to(odt)
    hb = torch.full((x.numel() + 2,), 7.0, dtype=x.dtype, device="cuda")
    out, h = ob[1:-1].view(x.shape), hb[1:-1].view(x.shape)
    _, scale, _ = gdn.rmsnorm_residual(shifted(x), shifted(w), shifted(r), out=out, residual_out=h)
    torch.cuda.synchronize()
    _check(x, w, r, out, scale, h)
    assert hb[0] == 7 and hb[-1] == 7 and ob[0].float() == 0 and ob[-1].float() == 0


def test_in_place_and_leading_dims(gdn):
    x, w, r = _draw(24, 640, "bf16", seed=3)
    ref = gdn.rmsnorm_residual(x, w, r)
    x3, r3 = x.view(2, 3, 4, 640).clone(), r.view(2, 3, 4, 640).clone()
    out, _, h = gdn.rmsnorm_residual(x3, w, r3, out=x3, residual_out=r3)
    assert out is x3 and h is r3
    assert torch.equal(out.view(24, 640), ref[0]) and torch.equal(h.view(24, 640), ref[2])
    _, scale, _ = gdn.rmsnorm_residual(x.view(4, 6, 640), w, out_dtype=torch.float8_e4m3fn)
    assert scale.shape == (4, 6)


@pytest.mark.parametrize("rows,D,dtype", [(900, 641, "bf16"), (4000, 1027, "bf16"), (700, 4099, "f32"), (5, 16381, "bf16"),
                                          (3000, 3, "f32"), (2000, 13, "bf16")])
def test_rows_off_16_bytes_in_place(gdn, rows, D, dtype):
    """Rows that start anywhere in a 16-byte piece: neighbouring rows share pieces, which a row in place must
    not disturb; more rows than run at once; guard bands behind the arrays."""
    x, w, r = _draw(rows, D, dtype, seed=D)
    ref = gdn.rmsnorm_residual(x, w, r)
    _check(x, w, r, ref[0], None, ref[2])
    xb = torch.full((rows * D + 9,), 5.0, dtype=x.dtype, device="cuda")
    rb = torch.full((rows * D + 9,), 5.0, dtype=x.dtype, device="cuda")
    xi, ri = xb[:rows * D].view(rows, D), rb[:rows * D].view(rows, D)
    xi.copy_(x)
    ri.copy_(r)
    gdn.rmsnorm_residual(xi, w, ri, out=xi, residual_out=ri)
    assert torch.equal(xi, ref[0]) and torch.equal(ri, ref[2])
    assert (xb[rows * D:] == 5).all() and (rb[rows * D:] == 5).all()


@pytest.mark.parametrize("D", [4096, 4100, 4099])
def test_offsets_past_32_bits(gdn, D):
    """More than 2^31 elements (8-bit output: more than 2^32 bytes of input); a sample of rows is checked."""
    rows = 2 ** 31 // D + 70
    gen = torch.Generator("cuda").manual_seed(D)
    x = torch.randn(rows, D, generator=gen, device="cuda", dtype=torch.bfloat16)
    w = torch.rand(D, generator=gen, device="cuda") + 0.5
    q, s, _ = gdn.rmsnorm_residual(x, w, out_dtype=torch.float8_e4m3fn)
    for r in (0, rows // 2, rows - 60, rows - 1):
        _check(x[r:r + 1], w, None, q[r:r + 1], s[r:r + 1], None)


@pytest.mark.parametrize("D", [256, 2048, 2049])
def test_rows_of_zeros_infinities_and_nan(gdn, D):
    """Zero rows give zeros (and the least scale); a NaN or an infinity stays in its own row."""
    x = torch.randn(4, D, device="cuda", generator=torch.Generator("cuda").manual_seed(1)).to(torch.bfloat16)
    w = torch.ones(D, device="cuda")
    x[0] = 0
    x[1, D // 2] = float("nan")
    x[2, 5] = float("inf")
    out, _, _ = gdn.rmsnorm_residual(x, w)
    q, s, _ = gdn.rmsnorm_residual(x, w, out_dtype=torch.float8_e4m3fn)
    o = out.float()
    assert (o[0] == 0).all() and o[1].isnan().all() and o[3].isfinite().all()
    assert o[2, 5].isnan() and (o[2, :5] == 0).all() and (o[2, 6:] == 0).all()   # finite / infinity, and inf / inf
    q = q.float()
    assert (q[0] == 0).all() and q[1].isnan().all() and q[2].isnan().all() and q[3].isfinite().all()
    assert s[0] == torch.tensor(1e-30) / 448 and s[1].isnan() and s[2].isnan() and s[3].isfinite()
    wn = w.clone()
    wn[7] = float("nan")
    q, s, _ = gdn.rmsnorm_residual(x, wn, out_dtype=torch.float8_e4m3fn)
    assert s.isnan().all() and q.float().isnan().all()


def test_eps_and_small_values(gdn):
    x, w, _ = _draw(6, 512, "f32", seed=9, residual=False)
    for eps, factor in ((0.0, 1.0), (1e-3, 1e-2), (1.0, 1e-12)):
        out, _, _ = gdn.rmsnorm_residual(x * factor, w, eps=eps)
        _check(x * factor, w, None, out, None, None, eps=eps)
        q, s, _ = gdn.rmsnorm_residual(x * factor, w, eps=eps, out_dtype=torch.float8_e4m3fn)
        _check(x * factor, w, None, q, s, None, eps=eps)


def test_repeats_bit_for_bit_and_on_another_stream(gdn):
    x, w, r = _draw(700, 4096, "bf16", seed=5)
    a = gdn.rmsnorm_residual(x, w, r, out_dtype=torch.float8_e4m3fn)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b = gdn.rmsnorm_residual(x, w, r, out_dtype=torch.float8_e4m3fn, stream=s)
    s.synchronize()
    assert torch.equal(a[0].view(torch.uint8), b[0].view(torch.uint8)) and torch.equal(a[1], b[1]) and torch.equal(a[2], b[2])


def test_refusals(gdn):
    x, w, r = _draw(4, 64, "bf16", seed=1)
    with pytest.raises(ValueError):
        gdn.rmsnorm_residual(x.t(), w)                       # not contiguous
    with pytest.raises(ValueError):
        gdn.rmsnorm_residual(x, w[:32].contiguous())
    with pytest.raises(ValueError):
        gdn.rmsnorm_residual(x, w, r[:2].contiguous())
    with pytest.raises(ValueError):
        gdn.rmsnorm_residual(x, w.cpu())
    with pytest.raises(TypeError):
        gdn.rmsnorm_residual(x, w.to(torch.bfloat16))
    with pytest.raises(TypeError):
        gdn.rmsnorm_residual(x, w, r.float())
    with pytest.raises(TypeError):
        gdn.rmsnorm_residual(x.half(), w)
    with pytest.raises(TypeError):
        gdn.rmsnorm_residual(x, w, out_dtype=torch.float32)
    with pytest.raises(ValueError):
        gdn.rmsnorm_residual(x, w, out_scale=torch.empty(4, device="cuda"))
    with pytest.raises(gdn.GdnError) as e:
        gdn.rmsnorm_residual(x, w, out=r, residual_out=r)
    assert e.value.code == gdn.GDN_ERR_UNSUPPORTED
    with pytest.raises(gdn.GdnError) as e:
        gdn.rmsnorm_residual(torch.zeros(1, 32769, device="cuda"), torch.ones(32769, device="cuda"))
    assert e.value.code == gdn.GDN_ERR_DIMS
