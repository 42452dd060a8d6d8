"""GPU parity of ``gdn_linear`` (``linear``, ``linear_gated``) with the fp64 oracle ``oracle.layer``.

The bar of a sum of K products with fp32 accumulation, whatever its order: every one of at most K
additions rounds (or truncates) a partial sum of magnitude at most S = sum |x w| to 2^-23 of it.  The
errors of one sum add up like a random walk, so a few sqrt(K) of them are what can be seen; the bar
takes 8 sqrt(K) + 8 steps of 2^-24 S (the scales' and the bias's roundings are within the 8).  It goes
through the epilogue by the activations' slopes (at most 1.13) and the product rule, plus 16 u of the
value for the fast exponential and division (u = 2^-24), and the output's rounding: 2^-8 of the value
in bf16."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import layer  # noqa: E402

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32, "f8": torch.float8_e4m3fn}


@pytest.fixture(scope="module")
def gdn():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gated_delta_rule_20_gb300 as g
    g.lib()
    yield g
    assert g.device_status(0) == 0


def _draw(M, N, K, dtype, layout, gated, bias, residual, out, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    n = 2 * N if gated else N
    normal = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    x, w, xs, ws = normal(M, K), normal(n, K) / K ** 0.5, None, None
    if dtype == "f8":
        xs, ws = x.abs().amax(1) / 448, w.abs().amax(1) / 448
        x, w = x / xs[:, None], w / ws[:, None]
    x, w = x.to(DT[dtype]), w.to(DT[dtype])
    if layout == "kn":
        w = w.t().contiguous()
    return dict(x=x, weight=w, x_scale=xs, weight_scale=ws, bias=normal(n) if bias else None,
                residual=normal(M, N).to(DT[out]) if residual else None)


def _check(out, t, act, layout, gated):
    args = {k: None if t[k] is None else t[k].float().cpu() for k in t}
    a, s = layer.affine(args["x"], args["weight"], args["bias"], args["x_scale"], args["weight_scale"], layout)
    K = t["x"].shape[1]
    e = (8 * K ** 0.5 + 8) * U * s
    if gated:
        n = a.shape[1] // 2
        g, u, eg, eu = layer.activation(act, a[:, :n]), a[:, n:], 1.13 * e[:, :n], e[:, n:]
        eg = eg + 16 * U * np.abs(g)
        ref, e = g * u, eg * np.abs(u) + np.abs(g) * eu + eg * eu
    else:
        ref = layer.activation(act, a)
        e = 1.13 * e + 16 * U * np.abs(ref)
    if args["residual"] is not None:
        ref = ref + args["residual"].double().numpy()
    e = e + 2 * U * np.abs(ref)
    if out.dtype == torch.bfloat16:
        e = e + 2.0 ** -8 * (np.abs(ref) + e)
    got = out.detach().cpu().double().numpy()
    assert np.isfinite(got).all()
    bad = np.abs(got - ref) > e + 1e-30
    assert not bad.any(), "%d of %d elements beyond the bar, worst %.3g at %s" % (
        bad.sum(), bad.size, (np.abs(got - ref) / (e + 1e-30)).max(), np.argwhere(bad)[:3].tolist())


@pytest.mark.parametrize("dtype", ["bf16", "f8"])
@pytest.mark.parametrize("M", [1, 64, 700])
def test_graph_capture(gdn, M, dtype):
    """A norm and a product behind it, captured and replayed (programmatic launches in a graph)."""
    D, N = 1024, 768
    gen = torch.Generator("cuda").manual_seed(M)
    x, r = (torch.randn(M, D, generator=gen, device="cuda").to(torch.bfloat16) for _ in range(2))
    nw = torch.ones(D, device="cuda")
    w = torch.randn(N, D, generator=gen, device="cuda") / D ** 0.5
    ws = w.abs().amax(1) / 448 if dtype == "f8" else None
    w = (w / ws[:, None]).to(DT["f8"]) if dtype == "f8" else w.to(DT["bf16"])

    def layer():
        y, s, h = gdn.rmsnorm_residual(x, nw, r, out_dtype=DT[dtype])
        return gdn.linear(y, w, weight_layout="nk", x_scale=s, weight_scale=ws), h
    ref = layer()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = layer()
    for _ in range(3):
        out[0].zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], ref[0]) and torch.equal(out[1], ref[1])


@pytest.mark.parametrize("M,N,K,dtype", [(2048, 2048, 256, "bf16"), (700, 1536, 512, "bf16"), (64, 2048, 2048, "bf16"), (300, 1024, 1024, "f32"),
                                         (3, 2048, 2048, "f32"), (1500, 2048, 128, "f8")])
def test_outputs_reach_the_next_kernel(gdn, M, N, K, dtype):
    """A product, a norm of it and a product of the norm, launched at once behind one another into reused buffers,
    against the same calls with a synchronisation after each: the same bits, forty times over."""
    out = "f32" if dtype == "f32" else "bf16"
    t = [_draw(M, N, K, dtype, "nk", False, False, False, out, seed=i) for i in range(4)]
    nw, w2 = torch.ones(N, device="cuda"), t[0]["weight"].new_zeros((256, N)).float().normal_().to(DT[out])
    y, z = torch.empty(M, N, dtype=DT[out], device="cuda"), torch.empty(M, 256, dtype=DT[out], device="cuda")

    def chain(i, wait):
        gdn.linear(t[i]["x"], t[i]["weight"], weight_layout="nk", x_scale=t[i]["x_scale"], weight_scale=t[i]["weight_scale"], out=y)
        if wait:
            torch.cuda.synchronize()
        n = gdn.rmsnorm_residual(y, nw)[0]
        if wait:
            torch.cuda.synchronize()
        gdn.linear(n, w2, weight_layout="nk", out=z)
        return z.clone()
    ref = [chain(i, True) for i in range(4)]
    got = [chain(i % 4, False) for i in range(40)]
    assert all(torch.equal(got[i], ref[i % 4]) for i in range(40))


def _run(gdn, M, N, K, dtype="bf16", layout="nk", gated=False, act="none", bias=False, residual=False, out=None, **kw):
    out = out or ("f32" if dtype == "f32" else "bf16")
    t = _draw(M, N, K, dtype, layout, gated, bias, residual, out, seed=M * 31 + N * 7 + K)
    call = gdn.linear_gated if gated else gdn.linear
    # NaN in the output before the call: what is not written shows, and so does a write past the end
    buf = torch.full((M * N + 64,), float("nan"), dtype=DT[out], device="cuda")
    got = call(t["x"], t["weight"], t["bias"], t["residual"], activation=act, weight_layout=layout,
               x_scale=t["x_scale"], weight_scale=t["weight_scale"], out=buf[:M * N].view(M, N), **kw)
    torch.cuda.synchronize()
    assert buf[M * N:].isnan().all()
    _check(got, t, act, layout, gated)
    return got, t


# a token to many; sizes under, at and over a tile's; widths that no 16 bytes divide
MNK = [(1, 1, 1), (1, 1, 16), (1, 128, 64), (1, 2048, 4096), (2, 130, 72), (3, 64, 48), (5, 7, 33), (16, 256, 128), (17, 200, 144),
       (33, 96, 1040), (64, 128, 64), (65, 129, 80), (100, 1000, 272), (127, 136, 200), (128, 512, 512), (129, 640, 336), (200, 72, 16),
       (256, 256, 2048), (257, 384, 192), (300, 1111, 96), (513, 264, 1056), (700, 2056, 520)]


@pytest.mark.parametrize("M,N,K", MNK)
@pytest.mark.parametrize("layout", ["kn", "nk"])
@pytest.mark.parametrize("gated", [False, True])
def test_bf16_shapes(gdn, M, N, K, layout, gated):
    _run(gdn, M, N, K, "bf16", layout, gated, act="silu" if gated else "none")


@pytest.mark.parametrize("M,N,K", MNK)
@pytest.mark.parametrize("gated", [False, True])
def test_f8_shapes(gdn, M, N, K, gated):
    _run(gdn, M, N, K, "f8", "nk", gated, act="silu" if gated else "none", bias=True)


@pytest.mark.parametrize("M,N,K", MNK)
@pytest.mark.parametrize("layout", ["kn", "nk"])
def test_f32_shapes(gdn, M, N, K, layout):
    _run(gdn, M, N, K, "f32", layout, gated=M % 2 == 0, act="gelu", bias=True)


@pytest.mark.parametrize("M,N,K", [(3, 136, 192), (70, 300, 520), (400, 520, 264)])
@pytest.mark.parametrize("dtype", ["bf16", "f8", "f32"])
@pytest.mark.parametrize("act", ["none", "silu", "gelu", "relu"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("bias,residual,out", [(False, False, "f32"), (True, True, "f32"), (False, True, None), (True, False, None)])
def test_epilogues(gdn, M, N, K, dtype, act, gated, bias, residual, out):
    _run(gdn, M, N, K, dtype, "nk", gated, act, bias, residual, out)


@pytest.mark.parametrize("M,N,K,dtype,layout,gated", [
    (4096, 2048, 2048, "bf16", "kn", False), (3001, 1501, 1040, "bf16", "nk", False), (2050, 1030, 2048, "f8", "nk", True),
    (1500, 4104, 648, "bf16", "kn", True), (5000, 300, 256, "f8", "nk", False),
    # token tiles of every width from 64 to 256
    (1003, 5000, 512, "bf16", "nk", False), (1024, 5120, 256, "bf16", "kn", False), (1531, 2600, 384, "f8", "nk", True),
    (930, 4096, 256, "f8", "nk", False), (1300, 3400, 256, "bf16", "nk", True), (2222, 2048, 320, "bf16", "kn", False),
    (640, 6000, 264, "bf16", "nk", False), (1100, 4999, 256, "bf16", "nk", False), (377, 9001, 256, "f8", "nk", True), (1, 16384, 8192, "bf16", "nk", False)])
def test_larger(gdn, M, N, K, dtype, layout, gated):
    _run(gdn, M, N, K, dtype, layout, gated, "silu" if gated else "none", residual=True)


@pytest.mark.parametrize("M,N,K,dtype,layout,gated", [
    (1000, 1001, 1003, "bf16", "kn", False), (1000, 1001, 1003, "bf16", "nk", False), (515, 700, 1404, "bf16", "kn", True),
    (515, 701, 1408, "bf16", "kn", True), (2000, 3001, 130, "bf16", "nk", True), (1037, 1111, 1001, "f8", "nk", False),
    (700, 803, 1030, "f8", "nk", True), (9, 16001, 4001, "bf16", "kn", False), (4100, 129, 2050, "bf16", "kn", False)])
def test_large_products_of_rows_off_16_bytes(gdn, M, N, K, dtype, layout, gated):
    """Odd row pitches (and a gated [K, 2 N] weight whose halves do not start on 16 bytes) in products
    of 1e9 operations and more, whose operands are copied to aligned rows; also from unaligned addresses
    and under graph capture."""
    assert 2 * M * N * (2 if gated else 1) * K >= 1e9
    got, t = _run(gdn, M, N, K, dtype, layout, gated, "silu" if gated else "none", bias=True, residual=True)
    for which in ("x", "weight"):
        b = torch.empty(t[which].numel() + 1, dtype=t[which].dtype, device="cuda")
        b[1:].view(t[which].shape).copy_(t[which])
        t[which] = b[1:].view(t[which].shape)
    call = gdn.linear_gated if gated else gdn.linear
    f = lambda: call(t["x"], t["weight"], t["bias"], t["residual"], activation="silu" if gated else "none",  # noqa: E731
                     weight_layout=layout, x_scale=t["x_scale"], weight_scale=t["weight_scale"])
    assert torch.equal(f(), got)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = f()
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, got)


@pytest.mark.parametrize("M,N,K,layout,gated", [
    (333, 1030, 770, "kn", False), (333, 1030, 770, "nk", False), (1000, 1001, 1003, "kn", False), (600, 515, 1000, "kn", True),
    (600, 513, 999, "nk", True), (64, 4096, 1024, "nk", False), (32, 2048, 4096, "kn", False), (3000, 700, 130, "kn", False),
    (1024, 1024, 1024, "kn", False)])
def test_fp32_products_by_parts(gdn, M, N, K, layout, gated):
    """fp32 products large enough for the tensor cores (parts of 8 bits), at the bar of fp32 sums: the products
    of parts left out are under 2 x 2^-24 of every term.  Also with operands of the widest range: the largest
    fp32 numbers, subnormal ones, and neighbours of powers of two."""
    assert 2 * M * N * (2 if gated else 1) * K >= 3e8
    got, t = _run(gdn, M, N, K, "f32", layout, gated, "gelu", bias=True, residual=True)
    gen = torch.Generator("cuda").manual_seed(K)
    x = torch.randn(M, K, generator=gen, device="cuda") * 2.0 ** torch.randint(-40, 40, (M, 1), generator=gen, device="cuda")
    x[1], x[2] = x[1].sign() * 2.0 ** -140, 3.4028235e38 * x[2].sign()
    x[3] = torch.where(x[3] > 0, 1 + 2.0 ** -23, 1 - 2.0 ** -24)
    w = t["weight"].clone()
    w[0] *= 2.0 ** -20
    w[-1] *= 2.0 ** -60
    wide = dict(t, x=x, weight=w * 2.0 ** -20, bias=None, residual=None)
    call = gdn.linear_gated if gated else gdn.linear
    out = call(x, wide["weight"], activation="none", weight_layout=layout)
    if gated:  # the product of two huge sums may pass fp32's range
        keep = torch.ones(M, dtype=torch.bool, device="cuda")
        keep[2] = False
        out, wide["x"] = out[keep], x[keep]
    _check(out, wide, "none", layout, gated)


@pytest.mark.parametrize("M,N,K,dtype", [(1000, 1001, 1003, "bf16"), (500, 700, 900, "f32"), (40, 64, 64, "bf16")])
def test_scratch_of_the_library_and_of_the_caller(gdn, M, N, K, dtype):
    """gdn_linear (stream-ordered scratch of its own) and gdn_linear_ws give the same bits; a workspace is not
    written past its size."""
    import ctypes
    from gated_delta_rule_20_gb300 import _binding as b
    t = _draw(M, N, K, dtype, "kn", False, False, False, "f32", seed=6)
    L, code = gdn.lib(), gdn.GDN_BF16 if dtype == "bf16" else gdn.GDN_F32
    d = gdn.GdnLinearDims(M, N, K, code, gdn.GDN_F32, 0, 0)
    outs = [torch.full((M, N), float("nan"), device="cuda") for _ in range(3)]
    x, w, s = t["x"].data_ptr(), t["weight"].data_ptr(), torch.cuda.current_stream().cuda_stream
    b._check(L.gdn_linear(x, None, w, None, None, None, outs[0].data_ptr(), ctypes.byref(d), s))
    need = L.gdn_linear_workspace_bytes(x, w, ctypes.byref(d))
    ws = torch.full((need + 64,), 0x5A, dtype=torch.uint8, device="cuda")
    b._check(L.gdn_linear_ws(x, None, w, None, None, None, outs[1].data_ptr(), ctypes.byref(d), ws.data_ptr(), need, s))
    outs[2] = gdn.linear(t["x"], t["weight"], out=outs[2])
    torch.cuda.synchronize()
    assert (need > 0) == (K > 64) and (ws[need:] == 0x5A).all()
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("where", ["x", "weight"])
def test_fp32_products_with_infinities_and_nan(gdn, where, bad, gated):
    """An operand that has one is left to the FFMA kernel: the same bits as when it is asked for, and the
    residual in place is added once."""
    t = _draw(400, 500, 900, "f32", "nk", gated, False, True, "f32", seed=3)
    t[where][77, 11] = bad
    call = gdn.linear_gated if gated else gdn.linear
    ref = call(t["x"], t["weight"], None, t["residual"], activation="silu", weight_layout="nk", force_ffma=True)
    r = t["residual"].clone()
    got = call(t["x"], t["weight"], None, r, activation="silu", weight_layout="nk", out=r)
    assert torch.equal(got.view(torch.int32), ref.view(torch.int32)) and not torch.isfinite(ref).all()


@pytest.mark.parametrize("M,N,K,dtype,layout,gated,out", [
    (384, 2048, 4096, "bf16", "kn", False, "bf16"), (391, 2041, 4104, "bf16", "nk", False, "bf16"), (768, 2048, 8192, "bf16", "kn", False, "f32"),
    (250, 1100, 6000, "bf16", "nk", False, "bf16"), (513, 1024, 8192, "bf16", "nk", True, "bf16"), (300, 1016, 4120, "bf16", "kn", True, "f32"),
    (500, 2048, 8192, "f8", "nk", False, "bf16"), (380, 1001, 8208, "f8", "nk", True, "bf16"), (1100, 500, 16000, "bf16", "nk", False, "f32")])
@pytest.mark.parametrize("full", [False, True])
def test_few_tiles_and_a_long_K(gdn, M, N, K, dtype, layout, gated, out, full):
    """The sizes of the pairs that split K: whole and ragged tiles, uneven shares of K, odd rows; with everything in
    the epilogue and without."""
    _run(gdn, M, N, K, dtype, layout, gated, "gelu" if full else "none", bias=full, residual=full, out=out)


@pytest.mark.parametrize("dtype,layout", [("f32", "kn"), ("f32", "nk"), ("bf16", "kn"), ("bf16", "nk"), ("f8", "nk")])
@pytest.mark.parametrize("M,N,K", [
    (1, 1, 1), (1, 31, 37), (1, 64, 128), (1, 600, 130), (1, 33, 9000), (1, 2000, 1025), (1, 16, 12345), (2, 130, 257), (3, 48, 512),
    (4, 96, 2048), (4, 129, 8193), (5, 72, 1000), (8, 256, 4112), (8, 515, 1537), (9, 40, 300), (12, 136, 640), (12, 7, 3001)])
@pytest.mark.parametrize("gated", [False, True])
def test_few_rows_on_the_fma_units(gdn, M, N, K, dtype, layout, gated):
    """Few rows without tensor cores: K inside, at and over the pieces, the chunks and the ranks' shares."""
    _run(gdn, M, N, K, dtype, layout, gated, "silu" if gated else "none", bias=True, residual=M % 2 == 0, force_ffma=True)


@pytest.mark.parametrize("dtype,layout", [("f32", "kn"), ("f32", "nk"), ("bf16", "kn"), ("bf16", "nk"), ("f8", "nk")])
def test_few_rows_keep_nan_apart(gdn, dtype, layout):
    """A NaN in x stays in its row and one in the weight in its column, at sizes with rows and columns to spare."""
    M, N, K = 5, 70, 777
    t = _draw(M, N, K, dtype, layout, False, False, False, "f32", seed=9)
    nan = torch.tensor(float("nan"), device="cuda").to(DT[dtype])
    t["x"][3, 5] = nan
    t["weight"][(11, 60) if layout == "kn" else (60, 11)] = nan
    out = gdn.linear(t["x"], t["weight"], weight_layout=layout, x_scale=t["x_scale"], weight_scale=t["weight_scale"], force_ffma=True)
    far = torch.zeros(M, N, dtype=torch.bool, device="cuda")
    far[3], far[:, 60] = True, True
    assert torch.equal(out.isnan(), far)


@pytest.mark.parametrize("M,N,K,layout,gated", [
    (65, 2080, 1200, "kn", False), (65, 2080, 4096, "nk", False), (97, 1032, 2000, "kn", True), (257, 515, 1409, "nk", True),
    (2000, 1300, 64, "kn", False), (900, 2100, 3001, "kn", False), (700, 3001, 1999, "kn", True), (2000, 1999, 705, "nk", False)])
def test_fp32_parts_of_every_plan(gdn, M, N, K, layout, gated):
    """K of one slab to 4096 (one to three accumulators of the largest products), few and many tokens, odd rows;
    operands up to 2^63, and rows whose elements lie 2^40 apart."""
    assert 2 * M * N * (2 if gated else 1) * K >= 3e8
    t = _draw(M, N, K, "f32", layout, gated, False, False, "f32", seed=K)
    gen = torch.Generator("cuda").manual_seed(M)
    x = t["x"] * 2.0 ** torch.randint(-20, 20, (M, K), generator=gen, device="cuda")
    x[1] = 9.2e18 * x[1].sign()
    x[2] = torch.where(x[2] > 0, 1 + 2.0 ** -23, 1 - 2.0 ** -24)
    t = dict(t, x=x)
    out = (gdn.linear_gated if gated else gdn.linear)(x, t["weight"], activation="none", weight_layout=layout)
    torch.cuda.synchronize()
    if gated:  # (the product of two sums of 1e18 passes fp32's range)
        keep = torch.ones(M, dtype=torch.bool, device="cuda")
        keep[1] = False
        out, t["x"] = out[keep], x[keep]
    _check(out, t, "none", layout, gated)


def test_fp32_products_past_the_range(gdn):
    """Products that pass fp32's range are infinities of the sum's sign, not NaN."""
    gen = torch.Generator("cuda").manual_seed(5)
    x = torch.rand(300, 700, generator=gen, device="cuda") + 0.5
    w = torch.rand(800, 700, generator=gen, device="cuda") + 0.5
    x[7] *= 1e30
    w[9] *= -1e30
    out = gdn.linear(x, w, weight_layout="nk")
    far = torch.zeros_like(out, dtype=torch.bool)
    far[7, 9] = True
    assert out[7, 9] == float("-inf") and torch.isfinite(out[~far]).all()


@pytest.mark.parametrize("M,N,K", [(5, 128, 128), (300, 264, 192)])
@pytest.mark.parametrize("dtype", ["bf16", "f8"])
def test_tensor_cores_agree_with_ffma(gdn, M, N, K, dtype):
    _run(gdn, M, N, K, dtype, "nk", True, "gelu", True, True, force_ffma=True)


@pytest.mark.parametrize("which", ["x", "weight"])
@pytest.mark.parametrize("dtype", ["bf16", "f8"])
def test_unaligned_operands(gdn, which, dtype):
    """An operand one element past a 16-byte boundary."""
    t = _draw(40, 96, 128, dtype, "nk", False, False, False, "bf16", seed=2)
    b = torch.empty(t[which].numel() + 1, dtype=t[which].dtype, device="cuda")
    b[1:].view(t[which].shape).copy_(t[which])
    t[which] = b[1:].view(t[which].shape)
    got = gdn.linear(t["x"], t["weight"], weight_layout="nk", x_scale=t["x_scale"], weight_scale=t["weight_scale"])
    torch.cuda.synchronize()
    _check(got, t, "none", "nk", False)


@pytest.mark.parametrize("M", [1, 100, 1000])
@pytest.mark.parametrize("dtype", ["bf16", "f8"])
def test_nan_and_infinity_stay_in_their_rows_and_columns(gdn, M, dtype):
    """A NaN in a token's row makes that row NaN and no other; one in a weight column that column;
    an infinity (a NaN in e4m3) too.  Nothing of a padded tile leaks into what is written."""
    N, K = 72, 80
    t = _draw(M, N, K, dtype, "nk", False, False, False, "bf16", seed=4)
    i, j = M // 2, 41
    t["x"].view(torch.uint8 if dtype == "f8" else torch.int16)[i, K - 1] = 0x7F if dtype == "f8" else 0x7FC0
    t["weight"].view(torch.uint8 if dtype == "f8" else torch.int16)[j, 0] = 0x7F if dtype == "f8" else 0x7F80
    got = gdn.linear(t["x"], t["weight"], weight_layout="nk", x_scale=t["x_scale"], weight_scale=t["weight_scale"]).float()
    assert got[i].isnan().all()
    rest = torch.ones(M, N, dtype=torch.bool, device="cuda")
    rest[i] = False
    rest[:, j] = False
    assert got[rest].isfinite().all()
    col = torch.cat([got[:i, j], got[i + 1:, j]])
    assert not col.isfinite().any()


def test_activations_over_their_range(gdn):
    """gelu within its approximation's 0.75e-7 |v| and 8 roundings of v, silu within 16 roundings of the value."""
    v = torch.cat([torch.linspace(-14, 14, 40001), torch.logspace(-30, 1, 4000), -torch.logspace(-30, 1, 4000)])
    w = torch.ones(1, 1, device="cuda")
    for act, bar in (("gelu", lambda r: (0.75e-7 + 8 * U) * v.abs().numpy()), ("silu", lambda r: 16 * U * np.abs(r))):
        ref = layer.activation(act, v.double().numpy())
        got = gdn.linear(v.cuda()[:, None].contiguous(), w, activation=act).flatten().cpu().double().numpy()
        assert (np.abs(got - ref) <= bar(ref) + 1e-37).all(), act


def test_activations_at_their_ends(gdn):
    """Sums of +-200 and of +-infinity through every activation, against the formulas' limits."""
    x = torch.tensor([[200.0], [-200.0], [float("inf")], [float("-inf")]], device="cuda")
    w = torch.ones(1, 1, device="cuda")
    r = {a: gdn.linear(x, w, activation=a).flatten().tolist() for a in ("none", "silu", "gelu", "relu")}
    inf = float("inf")
    assert r["none"] == [200.0, -200.0, inf, -inf] and r["relu"] == [200.0, 0.0, inf, 0.0]
    assert r["silu"][0] == 200.0 and abs(r["silu"][1]) < 1e-30 and r["silu"][2] == inf
    assert r["gelu"][0] == 200.0 and abs(r["gelu"][1]) < 1e-30 and r["gelu"][2] == inf


def test_in_place_residual_leading_dims_and_streams(gdn):
    t = _draw(6 * 35, 512, 256, "bf16", "kn", False, True, True, "bf16", seed=8)
    ref = gdn.linear(t["x"], t["weight"], t["bias"], t["residual"], activation="silu")
    x, r = t["x"].view(6, 35, 256), t["residual"].view(6, 35, 512).clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = gdn.linear(x, t["weight"], t["bias"], r, activation="silu", out=r, stream=s)
    s.synchronize()
    assert out is r and torch.equal(r.view(-1, 512), ref)
    assert gdn.linear(x[0, 0].contiguous(), t["weight"]).shape == (512,)
    assert gdn.linear(torch.empty(0, 256, dtype=torch.bfloat16, device="cuda"), t["weight"]).shape == (0, 512)


@pytest.mark.parametrize("M,N,K,dtype,layout,gated", [
    (40000, 65536, 64, "bf16", "nk", False), (40001, 65537, 32, "f8", "nk", False), (70000, 32768, 64, "bf16", "kn", True),
    (4, 1 << 17, 16400, "bf16", "kn", False), (3, 1 << 17, 16400, "f8", "nk", False), (140000, 16, 16384, "bf16", "nk", False),
    (3, 1 << 16, 40000, "f32", "kn", False), (4100000, 64, 16, "bf16", "nk", False), (4194240, 3, 5, "f32", "kn", False)])
def test_offsets_past_32_bits(gdn, M, N, K, dtype, layout, gated):
    """Outputs, weights and rows of more than 2^31 elements, and the most rows that a call takes; a sample of
    rows and columns at both ends is checked."""
    gen = torch.Generator("cuda").manual_seed(N)
    n = 2 * N if gated else N
    x = torch.randn(M, K, generator=gen, device="cuda", dtype=torch.bfloat16).to(DT[dtype])
    w = torch.randn(*((K, n) if layout == "kn" else (n, K)), generator=gen, device="cuda", dtype=torch.bfloat16)
    w = w.to(DT[dtype])
    xs, ws = (torch.rand(M, device="cuda"), torch.rand(n, device="cuda")) if dtype == "f8" else (None, None)
    call = gdn.linear_gated if gated else gdn.linear
    out = call(x, w, activation="none", weight_layout=layout, x_scale=xs, weight_scale=ws)
    rows = torch.tensor(sorted({0, M // 2, max(0, M - 130), M - 1}), device="cuda")
    cols = torch.tensor(sorted({0, N // 2, max(0, N - 131), N - 1}), device="cuda")
    at = torch.cat([cols, cols + N]) if gated else cols
    pick = (lambda v: v[:, at]) if layout == "kn" else (lambda v: v.view(torch.uint8)[at].view(DT["f8"]) if dtype == "f8" else v[at])
    xr = x.view(torch.uint8)[rows].view(DT["f8"]) if dtype == "f8" else x[rows]
    t = dict(x=xr, weight=pick(w), bias=None, residual=None, x_scale=None if xs is None else xs[rows],
             weight_scale=None if ws is None else ws[at])
    _check(out[rows][:, cols], t, "none", layout, gated)


@pytest.mark.parametrize("M,N,K,dtype", [(1, 2048, 4096, "bf16"), (64, 2048, 2048, "f8"), (1111, 1024, 512, "bf16")])
def test_repeats_bit_for_bit(gdn, M, N, K, dtype):
    t = _draw(M, N, K, dtype, "nk", False, False, False, "f32", seed=1)
    f = lambda: gdn.linear(t["x"], t["weight"], weight_layout="nk", x_scale=t["x_scale"],  # noqa: E731
                           weight_scale=t["weight_scale"], out_dtype=torch.float32)
    a = f()
    for _ in range(5):
        assert torch.equal(a, f())


def test_refusals(gdn):
    bf = torch.bfloat16
    x, w = torch.zeros(4, 64, dtype=bf, device="cuda"), torch.zeros(64, 32, dtype=bf, device="cuda")
    for bad in (dict(weight_layout="mn"), dict(activation="tanh"), dict(x_scale=torch.ones(4, device="cuda")),
                dict(bias=torch.zeros(31, device="cuda")), dict(residual=torch.zeros(4, 31, dtype=bf, device="cuda")),
                dict(out=torch.zeros(4, 31, dtype=bf, device="cuda")), dict(weight=w.t()), dict(weight=w[:32].contiguous()),
                dict(weight=w.cpu())):
        with pytest.raises(ValueError):
            gdn.linear(**dict(dict(x=x, weight=w), **bad))
    for bad in (dict(weight=w.float()), dict(bias=torch.zeros(32, dtype=bf, device="cuda")),
                dict(residual=torch.zeros(4, 32, device="cuda")), dict(x=x.half(), weight=w.half())):
        with pytest.raises(TypeError):
            gdn.linear(**dict(dict(x=x, weight=w), **bad))
    with pytest.raises(ValueError):
        gdn.linear_gated(x, torch.zeros(64, 31, dtype=bf, device="cuda"))
    x8, w8 = x.to(torch.float8_e4m3fn), torch.zeros(32, 64, device="cuda").to(torch.float8_e4m3fn)
    with pytest.raises(ValueError):
        gdn.linear(x8, w8, weight_layout="nk")                       # scales are missing
    with pytest.raises(gdn.GdnError) as e:
        gdn.linear(x8, w8.t().contiguous(), weight_layout="kn", x_scale=torch.ones(4, device="cuda"),
                   weight_scale=torch.ones(32, device="cuda"))
    assert e.value.code == gdn.GDN_ERR_UNSUPPORTED
    with pytest.raises(gdn.GdnError) as e:
        gdn.linear(x.float(), w.float(), out_dtype=bf)
    assert e.value.code == gdn.GDN_ERR_UNSUPPORTED
