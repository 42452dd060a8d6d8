"""The kernel, token tile and splits of K that ``gdn_linear`` takes (``gdn_linear_plan``, on the host), and every such
variant on the GPU against the fp64 oracle."""
import ctypes

import pytest
import torch

import gated_delta_rule_20_gb300 as gdn
from gated_delta_rule_20_gb300 import build as gbuild

CODES = {"bf16": gdn.GDN_BF16, "f32": gdn.GDN_F32, "f8": gdn.GDN_F8E4M3}
SMS = 152  # of a GB300, for which the cases' plans are written down

# M, N, K, type, layout, gated, and the plan: every tile and split of the tensor-core kernels that sizes of
# 17 to 1500 rows, 256 to 4096 columns and K = 512 to 16384 lead to
CASES = [
    (320, 1000, 2048, "bf16", "nk", False, "joint", 64, 3), (130, 1000, 16384, "bf16", "kn", False, "joint", 64, 4),
    (130, 4096, 2048, "bf16", "nk", False, "joint", 96, 2), (130, 2048, 4096, "bf16", "kn", False, "joint", 96, 3),
    (513, 500, 8192, "bf16", "nk", False, "joint", 96, 4), (200, 4096, 2048, "bf16", "kn", False, "joint", 128, 2),
    (200, 2048, 4096, "bf16", "nk", False, "joint", 128, 3), (700, 500, 4096, "bf16", "nk", False, "joint", 128, 4),
    (513, 2048, 2048, "bf16", "nk", False, "joint", 160, 2), (320, 2048, 4096, "bf16", "kn", False, "joint", 160, 3),
    (130, 2048, 8192, "bf16", "nk", False, "joint", 160, 4), (700, 2048, 4096, "bf16", "kn", False, "joint", 192, 2),
    (900, 1000, 4096, "bf16", "nk", False, "joint", 192, 3), (1024, 500, 8192, "bf16", "nk", False, "joint", 192, 4),
    (200, 4096, 16384, "bf16", "nk", False, "joint", 224, 3),
    (450, 4096, 8192, "bf16", "kn", False, "joint", 256, 2), (130, 2048, 512, "bf16", "nk", False, "pairs", 64, 1),
    (320, 4096, 512, "bf16", "kn", False, "pairs", 96, 1), (450, 4096, 512, "bf16", "nk", False, "pairs", 128, 1),
    (513, 4096, 512, "bf16", "kn", False, "pairs", 160, 1), (700, 4096, 512, "bf16", "nk", False, "pairs", 192, 1),
    (900, 4096, 512, "bf16", "kn", False, "pairs", 256, 1), (17, 256, 512, "bf16", "nk", False, "small", 16, 4),
    (17, 256, 1024, "bf16", "kn", False, "small", 16, 8), (320, 500, 512, "bf16", "nk", False, "small", 32, 4),
    (40, 1000, 4096, "bf16", "kn", False, "small", 32, 8), (130, 2048, 1024, "bf16", "nk", False, "small", 64, 4),
    (130, 500, 8192, "bf16", "nk", False, "small", 64, 8), (320, 500, 2048, "bf16", "nk", True, "joint", 64, 3),
    (130, 500, 16384, "bf16", "nk", True, "joint", 64, 4), (130, 2048, 2048, "bf16", "nk", True, "joint", 96, 2),
    (130, 1000, 4096, "bf16", "kn", True, "joint", 96, 3), (513, 256, 8192, "bf16", "nk", True, "joint", 96, 4),
    (200, 2048, 2048, "bf16", "kn", True, "joint", 128, 2), (200, 1000, 4096, "bf16", "nk", True, "joint", 128, 3),
    (700, 256, 4096, "bf16", "kn", True, "joint", 128, 4), (513, 1000, 2048, "bf16", "nk", True, "joint", 160, 2),
    (320, 1000, 4096, "bf16", "kn", True, "joint", 160, 3), (130, 1000, 8192, "bf16", "nk", True, "joint", 160, 4),
    (700, 1000, 4096, "bf16", "kn", True, "joint", 192, 2), (900, 500, 4096, "bf16", "nk", True, "joint", 192, 3),
    (513, 500, 8192, "bf16", "nk", True, "joint", 192, 4), (200, 4096, 8192, "bf16", "nk", True, "joint", 224, 2),
    (200, 2048, 16384, "bf16", "kn", True, "joint", 224, 3), (900, 1000, 8192, "bf16", "nk", True, "joint", 256, 2),
    (40, 4096, 1024, "bf16", "kn", True, "pairs", 128, 1), (450, 4096, 512, "bf16", "nk", True, "pairs", 256, 1),
    (40, 4096, 512, "bf16", "kn", True, "small", 32, 2), (40, 1000, 1024, "bf16", "nk", True, "small", 32, 4),
    (40, 500, 4096, "bf16", "nk", True, "small", 32, 8), (100, 4096, 8192, "bf16", "nk", True, "small", 128, 4),
    (130, 4096, 512, "f32", "kn", False, "pairs", 64, 1), (320, 4096, 512, "f32", "nk", False, "pairs", 96, 1),
    (450, 4096, 512, "f32", "kn", False, "pairs", 128, 1), (513, 4096, 512, "f32", "nk", False, "pairs", 160, 1),
    (700, 4096, 512, "f32", "kn", False, "pairs", 192, 1), (900, 4096, 512, "f32", "nk", False, "pairs", 256, 1),
    (513, 500, 1024, "f32", "nk", False, "small", 32, 2), (40, 2048, 2048, "f32", "nk", False, "small", 32, 4),
    (513, 1000, 512, "f32", "kn", False, "small", 64, 2), (320, 500, 1024, "f32", "nk", False, "small", 64, 4),
    (40, 1000, 4096, "f32", "kn", False, "small", 64, 8), (1200, 256, 512, "f32", "nk", False, "small", 128, 4),
    (200, 4096, 512, "f32", "kn", True, "pairs", 128, 1), (450, 4096, 512, "f32", "nk", True, "pairs", 256, 1),
    (513, 256, 1024, "f32", "kn", True, "small", 32, 2), (40, 1000, 2048, "f32", "nk", True, "small", 32, 4),
    (320, 500, 512, "f32", "nk", True, "small", 128, 4), (320, 1000, 4096, "f8", "nk", False, "joint", 64, 3),
    (130, 4096, 4096, "f8", "nk", False, "joint", 96, 2), (130, 2048, 8192, "f8", "nk", False, "joint", 96, 3),
    (513, 500, 16384, "f8", "nk", False, "joint", 96, 4), (200, 4096, 4096, "f8", "nk", False, "joint", 128, 2),
    (200, 2048, 8192, "f8", "nk", False, "joint", 128, 3), (700, 500, 8192, "f8", "nk", False, "joint", 128, 4),
    (513, 2048, 4096, "f8", "nk", False, "joint", 160, 2), (320, 2048, 8192, "f8", "nk", False, "joint", 160, 3),
    (130, 2048, 16384, "f8", "nk", False, "joint", 160, 4), (700, 2048, 8192, "f8", "nk", False, "joint", 192, 2),
    (900, 1000, 8192, "f8", "nk", False, "joint", 192, 3), (1024, 500, 16384, "f8", "nk", False, "joint", 192, 4),
    (320, 500, 512, "f8", "nk", False, "pairs", 64, 1), (100, 2048, 512, "f8", "nk", False, "pairs", 96, 1),
    (900, 2048, 512, "f8", "nk", False, "pairs", 128, 1), (100, 4096, 512, "f8", "nk", False, "pairs", 160, 1),
    (700, 4096, 512, "f8", "nk", False, "pairs", 192, 1), (900, 4096, 1024, "f8", "nk", False, "pairs", 256, 1),
    (17, 256, 512, "f8", "nk", False, "small", 16, 2), (17, 256, 1024, "f8", "nk", False, "small", 16, 4),
    (17, 256, 2048, "f8", "nk", False, "small", 16, 8), (320, 500, 1024, "f8", "nk", False, "small", 32, 4),
    (40, 1000, 8192, "f8", "nk", False, "small", 32, 8), (130, 2048, 2048, "f8", "nk", False, "small", 64, 4),
    (130, 500, 16384, "f8", "nk", False, "small", 64, 8), (320, 500, 4096, "f8", "nk", True, "joint", 64, 3),
    (130, 2048, 4096, "f8", "nk", True, "joint", 96, 2), (130, 1000, 8192, "f8", "nk", True, "joint", 96, 3),
    (513, 256, 16384, "f8", "nk", True, "joint", 96, 4), (200, 2048, 4096, "f8", "nk", True, "joint", 128, 2),
    (200, 1000, 8192, "f8", "nk", True, "joint", 128, 3), (700, 256, 8192, "f8", "nk", True, "joint", 128, 4),
    (513, 1000, 4096, "f8", "nk", True, "joint", 160, 2), (320, 1000, 8192, "f8", "nk", True, "joint", 160, 3),
    (130, 1000, 16384, "f8", "nk", True, "joint", 160, 4), (700, 1000, 8192, "f8", "nk", True, "joint", 192, 2),
    (900, 500, 8192, "f8", "nk", True, "joint", 192, 3), (513, 500, 16384, "f8", "nk", True, "joint", 192, 4),
    (200, 4096, 16384, "f8", "nk", True, "joint", 224, 2), (900, 1000, 16384, "f8", "nk", True, "joint", 256, 2),
    (40, 4096, 2048, "f8", "nk", True, "pairs", 128, 1), (450, 4096, 1024, "f8", "nk", True, "pairs", 256, 1),
    (40, 4096, 512, "f8", "nk", True, "small", 32, 2), (40, 1000, 2048, "f8", "nk", True, "small", 32, 4),
    (40, 500, 8192, "f8", "nk", True, "small", 32, 8), (100, 4096, 16384, "f8", "nk", True, "small", 128, 4),
    (1500, 4096, 512, "bf16", "nk", True, "pairs", 224, 1)]


@pytest.fixture(scope="module")
def L():
    gbuild.build()
    return gdn.lib()


@pytest.mark.parametrize("M,N,K,dtype,layout,gated,kernel,tokens,splits", CASES)
def test_plan_of_the_cases(L, M, N, K, dtype, layout, gated, kernel, tokens, splits):
    got = gdn.linear_plan(M, N, K, CODES[dtype], weight_layout=layout, gated=gated, sm_count=SMS)
    assert got == (kernel, "in parts" if dtype == "f32" else "as they lie", tokens, splits)


def test_cases_cover_the_splits(L):
    """Pairs that split K two, three and four ways, plain and gated, in both types, on tiles of 64 to 256 tokens."""
    joint = {(c[3], c[5], c[8]) for c in CASES if c[6] == "joint"}
    assert joint == {(t, g, s) for t in ("bf16", "f8") for g in (False, True) for s in (2, 3, 4)}
    assert {c[7] for c in CASES if c[6] == "joint"} == {64, 96, 128, 160, 192, 224, 256}
    assert {c[7] for c in CASES if c[6] == "pairs"} == {64, 96, 128, 160, 192, 224, 256}
    assert {c[7] for c in CASES if c[6] == "small"} == {16, 32, 64, 128}
    assert {c[8] for c in CASES if c[6] == "small"} == {2, 4, 8}


@pytest.mark.parametrize("sms", list(range(1, 161)) + [192, 304])
def test_every_number_of_sms_has_a_plan(L, sms):
    """A device may offer fewer SMs than a GB300 has: a plan within the kernels' limits comes back for all."""
    for dtype in ("bf16", "f8", "f32"):
        for M in (1, 16, 64, 200, 1000, 30000):
            for N in (8, 2048, 20000):
                for K in (64, 1024, 4096, 16384):
                    for gated in (False, True):
                        kernel, _, tokens, splits = gdn.linear_plan(M, N, K, CODES[dtype], weight_layout="nk",
                                                                    gated=gated, sm_count=sms)
                        slabs = -(-K // (128 if dtype == "f8" else 64))
                        if kernel in ("few", "ffma"):
                            assert dtype == "f32" and tokens == splits == 0
                        elif kernel == "small":
                            assert tokens in (16, 32, 64, 128) and splits in (1, 2, 4, 8) and 2 * splits <= max(2, slabs)
                        else:
                            assert tokens in range(64, 257, 32)
                            assert splits == 1 if kernel == "pairs" else splits in (2, 3, 4) and 2 * splits <= slabs


def test_routes(L):
    plan = lambda *a, **kw: gdn.linear_plan(*a, sm_count=SMS, **kw)  # noqa: E731
    assert plan(0, 64, 64) == ("none", "as they lie", 0, 0)
    assert plan(4, 100, 101) == ("few", "as they lie", 0, 0) and plan(40, 100, 101) == ("ffma", "as they lie", 0, 0)
    assert plan(64, 128, 128, force_ffma=True)[0] == "ffma" and plan(64, 128, 128, x_offset=2)[0] == "ffma"
    assert plan(64, 128, 128)[:2] == ("small", "as they lie")
    assert plan(1000, 1001, 1003)[1] == "copied" and plan(1000, 1000, 1000, weight_offset=2)[1] == "copied"
    assert plan(1000, 1000, 1000, gdn.GDN_F32)[1] == "in parts" and plan(1000, 1000, 8192, gdn.GDN_F32)[0] == "ffma"
    assert plan(16384, 2048, 4096)[0] == "pairs" and plan(768, 2048, 8192)[0] == "joint"


def test_refusals(L):
    info = gdn._binding.GdnLinearPlanInfo()
    good = dict(M=4, N=64, K=64, dtype=gdn.GDN_BF16, out_dtype=gdn.GDN_BF16, activation=0, flags=0)
    d = lambda **kw: ctypes.byref(gdn.GdnLinearDims(**dict(good, **kw)))  # noqa: E731
    assert L.gdn_linear_plan(64, 64, d(), SMS, ctypes.byref(info)) == gdn.GDN_OK
    assert L.gdn_linear_plan(64, 64, None, SMS, ctypes.byref(info)) == gdn.GDN_ERR_NULL
    assert L.gdn_linear_plan(64, 64, d(), SMS, None) == gdn.GDN_ERR_NULL
    assert L.gdn_linear_plan(64, 64, d(), 0, ctypes.byref(info)) == gdn.GDN_ERR_DIMS
    assert L.gdn_linear_plan(64, 64, d(N=0), SMS, ctypes.byref(info)) == gdn.GDN_ERR_DIMS
    assert L.gdn_linear_plan(64, 64, d(dtype=9), SMS, ctypes.byref(info)) == gdn.GDN_ERR_UNSUPPORTED
    with pytest.raises(ValueError):
        gdn.linear_plan(4, 64, 64, weight_layout="mn", sm_count=SMS)
    with pytest.raises(gdn.GdnError):
        gdn.linear_plan(4, 64, 64, gdn.GDN_F8E4M3, weight_layout="kn", sm_count=SMS)


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K,dtype,layout,gated,kernel,tokens,splits", CASES)
@pytest.mark.parametrize("full", [False, True])
def test_every_variant(L, M, N, K, dtype, layout, gated, kernel, tokens, splits, full):
    """With everything in the epilogue and bf16 outputs (fp32 in fp32), and with nothing and fp32 outputs."""
    import test_linear_gpu as t
    if torch.cuda.get_device_properties(0).multi_processor_count == SMS:
        assert gdn.linear_plan(M, N, K, CODES[dtype], weight_layout=layout, gated=gated)[0] == kernel
    t._run(gdn, M, N, K, dtype, layout, gated, "silu" if full else "none", bias=full, residual=full,
           out=None if full else "f32")
    assert gdn.device_status(0) == 0


def test_plans_of_fp32_outputs(L):
    """Sums of more than 8 slabs a CTA are worked off in blocks, which have smaller tiles: 192 tokens, 64 in the small
    kernel; shorter ones have bf16 outputs' plans."""
    seen = set()
    for dtype, elems in (("bf16", 64), ("f8", 128)):
        for M in (1, 17, 64, 130, 300, 768, 2000, 16384):
            for N in (64, 1000, 2048, 8192):
                for K in (128, 512, 1024, 2056, 4096, 8192, 16384):
                    if K % 16:
                        continue
                    of = lambda out: gdn.linear_plan(M, N, K, CODES[dtype], out, weight_layout="nk", sm_count=SMS)  # noqa: E731
                    kernel, _, tokens, splits = of(gdn.GDN_F32)
                    slabs = -(-K // elems)
                    share = -(-slabs // splits)
                    if share > 8:
                        assert tokens <= {"pairs": 192, "joint": 192, "small": 64}[kernel]
                        seen.add((dtype, kernel))
                    if slabs <= 8:
                        assert of(gdn.GDN_F32) == of(gdn.GDN_BF16)
    assert seen == {(d, k) for d in ("bf16", "f8") for k in ("small", "pairs", "joint")}
