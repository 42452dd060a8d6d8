"""Host-side checks of the layer operators' entry points and of their binding: every refusal
comes back as its code, or as an exception, before any launch, so no GPU is needed."""
import ctypes

import pytest
import torch

import gated_delta_rule_20_gb300 as gdn
from gated_delta_rule_20_gb300 import build as gbuild


@pytest.fixture(scope="module")
def L():
    gbuild.build()
    return gdn.lib()


P = 0x1000


def test_rmsnorm_residual_argument_checks(L):
    def call(x=P, res=P, w=P, h=0x2000, out=0x3000, scale=None, rows=4, D=128, dtype=gdn.GDN_BF16,
             out_dtype=gdn.GDN_BF16, eps=1e-6):
        return L.gdn_rmsnorm_residual(x, res, w, h, out, scale, rows, D, dtype, out_dtype, eps, None)
    assert call(rows=0) == gdn.GDN_OK and call(rows=0, x=None) == gdn.GDN_OK
    assert call(dtype=5) == gdn.GDN_ERR_UNSUPPORTED
    assert call(dtype=gdn.GDN_F8E4M3, out_dtype=gdn.GDN_F8E4M3) == gdn.GDN_ERR_UNSUPPORTED
    assert call(out_dtype=gdn.GDN_F32) == gdn.GDN_ERR_UNSUPPORTED            # neither x's dtype nor e4m3
    assert call(D=0) == gdn.GDN_ERR_DIMS and call(rows=-1) == gdn.GDN_ERR_DIMS
    assert call(D=32769) == gdn.GDN_ERR_DIMS and call(rows=1 << 31) == gdn.GDN_ERR_DIMS
    assert call(eps=-1.0) == gdn.GDN_ERR_DIMS and call(eps=float("nan")) == gdn.GDN_ERR_DIMS
    assert call(x=None) == gdn.GDN_ERR_NULL and call(w=None) == gdn.GDN_ERR_NULL and call(out=None) == gdn.GDN_ERR_NULL
    assert call(out_dtype=gdn.GDN_F8E4M3) == gdn.GDN_ERR_NULL                # e4m3 needs the scales
    assert call(h=0x3000) == gdn.GDN_ERR_UNSUPPORTED                         # two results in one buffer
    assert call(x=P + 1) == gdn.GDN_ERR_ALIGN and call(res=P + 1) == gdn.GDN_ERR_ALIGN
    assert call(h=P + 1) == gdn.GDN_ERR_ALIGN and call(out=P + 1) == gdn.GDN_ERR_ALIGN
    assert call(w=P + 2) == gdn.GDN_ERR_ALIGN
    assert call(out=P + 1, out_dtype=gdn.GDN_F8E4M3, scale=P + 2) == gdn.GDN_ERR_ALIGN
    assert call(x=P + 2, dtype=gdn.GDN_F32, out_dtype=gdn.GDN_F32) == gdn.GDN_ERR_ALIGN


def test_linear_argument_checks(L):
    def call(x=P, xs=None, w=P, ws=None, b=None, res=None, out=P, M=4, N=64, K=64, dtype=gdn.GDN_BF16,
             out_dtype=gdn.GDN_BF16, act=0, flags=0):
        d = gdn.GdnLinearDims(M, N, K, dtype, out_dtype, act, flags)
        return L.gdn_linear(x, xs, w, ws, b, res, out, ctypes.byref(d), None)
    f8 = dict(dtype=gdn.GDN_F8E4M3, flags=gdn.GDN_LINEAR_WEIGHT_NK, xs=P, ws=P)
    assert L.gdn_linear(P, None, P, None, None, None, P, None, None) == gdn.GDN_ERR_NULL
    assert call(M=0) == gdn.GDN_OK and call(M=0, x=None, out=None) == gdn.GDN_OK
    assert call(dtype=7) == gdn.GDN_ERR_UNSUPPORTED and call(out_dtype=gdn.GDN_F8E4M3) == gdn.GDN_ERR_UNSUPPORTED
    assert call(dtype=gdn.GDN_F32, out_dtype=gdn.GDN_BF16) == gdn.GDN_ERR_UNSUPPORTED
    assert call(act=4) == gdn.GDN_ERR_UNSUPPORTED and call(act=-1) == gdn.GDN_ERR_UNSUPPORTED
    assert call(flags=1 << 3) == gdn.GDN_ERR_UNSUPPORTED
    assert call(**dict(f8, flags=0)) == gdn.GDN_ERR_UNSUPPORTED              # e4m3 weights are [N, K]
    assert call(xs=P) == gdn.GDN_ERR_UNSUPPORTED and call(ws=P) == gdn.GDN_ERR_UNSUPPORTED
    assert call(M=-1) == gdn.GDN_ERR_DIMS and call(N=0) == gdn.GDN_ERR_DIMS and call(K=0) == gdn.GDN_ERR_DIMS
    assert call(M=4194241) == gdn.GDN_ERR_DIMS and call(K=1 << 31) == gdn.GDN_ERR_DIMS
    assert call(N=(1 << 30) + 1, flags=gdn.GDN_LINEAR_GATED) == gdn.GDN_ERR_DIMS
    assert call(x=None) == gdn.GDN_ERR_NULL and call(w=None) == gdn.GDN_ERR_NULL and call(out=None) == gdn.GDN_ERR_NULL
    assert call(**dict(f8, xs=None)) == gdn.GDN_ERR_NULL and call(**dict(f8, ws=None)) == gdn.GDN_ERR_NULL
    assert call(x=P + 1) == gdn.GDN_ERR_ALIGN and call(w=P + 1) == gdn.GDN_ERR_ALIGN
    assert call(out=P + 1) == gdn.GDN_ERR_ALIGN and call(res=P + 1) == gdn.GDN_ERR_ALIGN
    assert call(b=P + 2) == gdn.GDN_ERR_ALIGN
    assert call(out=P + 2, out_dtype=gdn.GDN_F32) == gdn.GDN_ERR_ALIGN
    assert call(**dict(f8, xs=P + 2)) == gdn.GDN_ERR_ALIGN and call(**dict(f8, ws=P + 2)) == gdn.GDN_ERR_ALIGN


def test_linear_workspace(L):
    """The scratch of a product: none for operands that the tensor cores take as they lie or that are small, and
    what the copies or parts need otherwise; a workspace that is too small or misaligned is refused."""
    def need(M, N, K, dtype=gdn.GDN_BF16, out=gdn.GDN_F32, flags=0, x=P, w=P):
        return L.gdn_linear_workspace_bytes(x, w, ctypes.byref(gdn.GdnLinearDims(M, N, K, dtype, out, 0, flags)))
    nk, gated, ffma = gdn.GDN_LINEAR_WEIGHT_NK, gdn.GDN_LINEAR_GATED, gdn.GDN_LINEAR_FORCE_FFMA
    assert need(4096, 4096, 4096) == 0 and need(4096, 4096, 4096, flags=nk) == 0
    assert need(10, 11, 13) == 0                                        # FFMA kernel
    assert need(1000, 1000, 1001) == 1000 * 1008 * 2                    # x only: the [K, N] weight's rows fit
    assert need(1000, 1000, 1001, flags=nk) == 2 * 1000 * 1008 * 2
    assert need(1000, 1001, 1000) == 1000 * 1008 * 2                    # the weight only
    assert need(1000, 1001, 1000, flags=nk) == 0
    assert need(1000, 1004, 1000, flags=gated) == 1000 * 2 * 1008 * 2   # its halves do not start on 16 bytes
    assert need(1000, 1000, 1000, x=P + 2) == 1000 * 1000 * 2
    assert need(1000, 1000, 1001, gdn.GDN_F8E4M3, flags=nk) == 2 * 1000 * 1008
    assert need(1000, 1000, 1001, flags=ffma) == 0
    assert need(1000, 1000, 1000, gdn.GDN_F32) >= 3 * 2 * 2 * 1000 * 1024   # three parts of both
    assert need(15, 4096, 4096, gdn.GDN_F32) == 0 < need(16, 4096, 4096, gdn.GDN_F32)
    assert need(1000, 1000, 8192, gdn.GDN_F32) == 0 and need(8, 10000, 4096, gdn.GDN_F32) == 0
    assert need(1000000, 1000, 4096, gdn.GDN_F32) == 0                  # past 4 GiB
    assert need(0, 1000, 1001) == 0 and need(1000, 0, 1001) == 0
    assert L.gdn_linear_workspace_bytes(P, P, None) == 0
    d = gdn.GdnLinearDims(1000, 1000, 1001, gdn.GDN_BF16, gdn.GDN_BF16, 0, 0)
    call = lambda ws, n: L.gdn_linear_ws(P, None, P, None, None, None, P, ctypes.byref(d), ws, n, None)  # noqa: E731
    assert call(P, 1000 * 1008 * 2 - 1) == gdn.GDN_ERR_WORKSPACE
    assert call(P + 8, 1 << 30) == gdn.GDN_ERR_ALIGN


def test_binding_refuses_host_tensors():
    x, w = torch.zeros(2, 8, dtype=torch.bfloat16), torch.ones(8)
    with pytest.raises(ValueError):
        gdn.rmsnorm_residual(x, w)
    with pytest.raises(ValueError):
        gdn.linear(x, torch.zeros(8, 8, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        gdn.linear_gated(x, torch.zeros(8, 8, dtype=torch.bfloat16))
