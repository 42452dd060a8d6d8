"""Outputs of the layer operators that lie over their inputs: in place where the header allows it, and refused before
any launch where rows would be read after they are overwritten."""
import ctypes

import pytest
import torch

import gated_delta_rule_20_gb300 as gdn
from gated_delta_rule_20_gb300 import build as gbuild


@pytest.fixture(scope="module")
def L():
    gbuild.build()
    return gdn.lib()


X, W, R, O = 0x100000, 0x200000, 0x300000, 0x400000  # room for 64 x 64 elements of any type each


@pytest.mark.parametrize("dtype,e", [(gdn.GDN_BF16, 2), (gdn.GDN_F32, 4), (gdn.GDN_F8E4M3, 1)])
@pytest.mark.parametrize("gated", [False, True])
def test_linear(L, dtype, e, gated):
    M, N, K = 16, 32, 64
    f8 = dtype == gdn.GDN_F8E4M3
    odt, o = (gdn.GDN_F32, 4) if dtype == gdn.GDN_F32 else (gdn.GDN_BF16, 2)
    d = gdn.GdnLinearDims(M, N, K, dtype, odt, 0, gdn.GDN_LINEAR_WEIGHT_NK | (gdn.GDN_LINEAR_GATED if gated else 0))
    s = 0x500000 if f8 else None

    def call(out, res=None):
        return L.gdn_linear(X, s, W, s, None, res, out, ctypes.byref(d), None)
    wbytes = (2 * N if gated else N) * K * e
    for out in (X, X + M * K * e - 16, X - M * N * o + 16, W, W + wbytes - 16, W - M * N * o + 16):
        assert call(out) == gdn.GDN_ERR_UNSUPPORTED, hex(out)
    assert call(O, O + 16) == gdn.GDN_ERR_UNSUPPORTED and call(O, O - 16) == gdn.GDN_ERR_UNSUPPORTED
    if not torch.cuda.is_available():  # past the checks: no device
        for out, res in ((O, None), (O, O), (O, R), (X + M * K * e, None), (X - M * N * o, None), (W + wbytes, None)):
            assert call(out, res) == gdn.GDN_ERR_CUDA, hex(out)


@pytest.mark.parametrize("dtype,e", [(gdn.GDN_BF16, 2), (gdn.GDN_F32, 4)])
def test_norm(L, dtype, e):
    rows, D = 16, 64

    def call(out, h=None, f8=False):
        return L.gdn_rmsnorm_residual(X, R, W, h, out, 0x500000 if f8 else None, rows, D, dtype, gdn.GDN_F8E4M3 if f8 else dtype,
                                      1e-6, None)
    n = rows * D * e
    for out in (X + 16, X - 16, R + 16, R - 16):
        assert call(out) == gdn.GDN_ERR_UNSUPPORTED and call(O, h=out) == gdn.GDN_ERR_UNSUPPORTED
    for out in (X, R, X + n - 16, X - rows * D + 16, R + n - 16):
        assert call(out, f8=True) == gdn.GDN_ERR_UNSUPPORTED
    assert call(O, h=O) == gdn.GDN_ERR_UNSUPPORTED and call(O, h=O + n - 16) == gdn.GDN_ERR_UNSUPPORTED
    assert call(X, h=X) == gdn.GDN_ERR_UNSUPPORTED and call(O, h=O + rows * D - 16, f8=True) == gdn.GDN_ERR_UNSUPPORTED
    if not torch.cuda.is_available():  # past the checks: no device
        for out, h, f8 in ((X, R, False), (X, None, False), (R, X, False), (O, X, True), (O, R, True), (O, O + rows * D, True),
                           (X + n, None, False)):
            assert call(out, h, f8) == gdn.GDN_ERR_CUDA


@pytest.mark.gpu
def test_in_place(L):
    """What is allowed in place gives the same bits: the norm's out over x or the residual, its sum over either; a
    product's out over its residual."""
    gen = torch.Generator("cuda").manual_seed(4)
    for D, dt in ((640, torch.bfloat16), (641, torch.bfloat16), (1001, torch.float32), (40001 // 2, torch.bfloat16)):
        x, r = (torch.randn(300, D, generator=gen, device="cuda").to(dt) for _ in range(2))
        w = torch.rand(D, generator=gen, device="cuda")
        ref = gdn.rmsnorm_residual(x, w, r)
        for o, h in ((0, 1), (1, 0), (0, None), (1, None), (None, 0), (None, 1)):
            t = [x.clone(), r.clone()]
            out, _, hh = gdn.rmsnorm_residual(t[0], w, t[1], out=None if o is None else t[o],
                                              residual_out=None if h is None else t[h])
            assert torch.equal(out, ref[0]) and torch.equal(hh, ref[2])
    with pytest.raises(gdn.GdnError):
        b = torch.zeros(64, 64, dtype=torch.bfloat16, device="cuda")
        gdn.linear(b, torch.zeros(64, 64, dtype=torch.bfloat16, device="cuda"), out=b)
