"""Host-side checks of linear attention's and rotary's entry points and of their binding: every refusal comes
back as its code, or as an exception, before any launch, so no GPU is needed."""
import ctypes
import math

import numpy as np
import pytest
import torch

import gated_delta_rule_20_gb300 as gdn
from gated_delta_rule_20_gb300 import build as gbuild
from oracle import linear_attn as ref


@pytest.fixture(scope="module")
def L():
    gbuild.build()
    return gdn.lib()


# addresses far from one another, for calls that are refused before they are used
Q, K, V, G, LEN, S_IN, S_OUT, OUT, WS = (0x10000000 * (i + 1) for i in range(9))


def dims(B=2, Hk=2, Hv=4, S=64, Dk=128, Dv=128, dtype=gdn.GDN_BF16, flags=0):
    return gdn.make_dims(B, Hk, Hv, S, Dk, Dv, dtype, flags)


def prefill(L, d, q=Q, k=K, v=V, g=G, lengths=None, s_in=S_IN, s_out=S_OUT, out=OUT, ws=None, nbytes=0):
    return L.gdn_linear_attn_prefill(q, k, v, g, lengths, 1.0, s_in, s_out, out, d, ws, nbytes, None)


def step(L, d, q=Q, k=K, v=V, g=G, lengths=None, s_in=S_IN, s_out=S_OUT, out=OUT):
    return L.gdn_linear_attn_step(q, k, v, g, 1.0, s_in, s_out, out, d, None)


@pytest.mark.parametrize("call, S", [(prefill, 64), (step, 1)])
def test_linear_attn_argument_checks(L, call, S):
    d = lambda **kw: dims(**dict(dict(S=S), **kw))  # noqa: E731
    assert call(L, None) == gdn.GDN_ERR_NULL
    assert call(L, d(B=0)) == gdn.GDN_OK and call(L, d(B=0), q=None, out=None, s_out=None) == gdn.GDN_OK
    assert call(L, d(dtype=7)) == gdn.GDN_ERR_UNSUPPORTED and call(L, d(dtype=gdn.GDN_F8E4M3)) == gdn.GDN_ERR_UNSUPPORTED
    assert call(L, d(flags=1 << 5)) == gdn.GDN_ERR_UNSUPPORTED
    assert call(L, d(flags=gdn.GDN_ZERO_INITIAL_STATE)) == gdn.GDN_ERR_UNSUPPORTED  # (a NULL state_in says that)
    for bad in (dict(B=-1), dict(Hk=0), dict(Hv=0), dict(Hk=3), dict(Dk=0), dict(Dv=0), dict(Dk=129), dict(Dv=129),
                dict(S=-1), dict(S=1 << 31), dict(B=1, Hk=1, Hv=1, S=(1 << 31) - 4096), dict(B=1 << 31), dict(B=1 << 29, Hv=8), dict(Hv=1 << 62, B=4, Hk=1)):
        assert call(L, d(**bad)) == gdn.GDN_ERR_DIMS, bad
    if call is step:
        assert call(L, d(S=2)) == gdn.GDN_ERR_DIMS and call(L, d(S=0)) == gdn.GDN_ERR_DIMS
        assert call(L, d(flags=gdn.GDN_ZERO_PADDING)) == gdn.GDN_ERR_UNSUPPORTED      # (there is no padding)
    for name in ("q", "k", "v", "g", "s_out", "out"):
        assert call(L, d(), **{name: None}) == gdn.GDN_ERR_NULL, name
    for name, at in (("q", Q), ("k", K), ("v", V), ("out", OUT)):
        assert call(L, d(), **{name: at + 1}) == gdn.GDN_ERR_ALIGN, name
        assert call(L, d(dtype=gdn.GDN_F32), **{name: at + 2}) == gdn.GDN_ERR_ALIGN, name
    for name, at in (("g", G), ("s_in", S_IN), ("s_out", S_OUT)):
        assert call(L, d(), **{name: at + 2}) == gdn.GDN_ERR_ALIGN, name
    # results that lie over what is read
    for name in ("q", "k", "v", "g", "s_in", "s_out"):
        assert call(L, d(), **{name: OUT}) == gdn.GDN_ERR_UNSUPPORTED, name
    for name in ("q", "k", "v", "g"):
        assert call(L, d(), **{name: S_OUT + 64}) == gdn.GDN_ERR_UNSUPPORTED, name
    assert call(L, d(), s_in=S_OUT + 64) == gdn.GDN_ERR_UNSUPPORTED


def test_linear_attn_prefill_more_checks(L):
    assert prefill(L, dims(), lengths=LEN + 2) == gdn.GDN_ERR_ALIGN
    assert prefill(L, dims(), lengths=OUT) == gdn.GDN_ERR_UNSUPPORTED
    assert prefill(L, dims(), ws=WS + 8, nbytes=1 << 30) == gdn.GDN_ERR_ALIGN
    assert prefill(L, dims(S=0), s_out=None) == gdn.GDN_ERR_NULL
    assert prefill(L, dims(S=0), q=None, k=None, v=None, g=None, out=None, s_in=S_OUT) == gdn.GDN_OK  # in place: no work


def test_linear_attn_segments(L):
    n = lambda d, sms=152: L.gdn_linear_attn_segments(d, sms)  # noqa: E731
    assert n(None) == 0 and n(dims(Hk=3)) == 0 and n(dims(), 0) == 0 and n(dims(flags=1)) == 0
    assert n(dims(S=0)) == 1 and n(dims(B=0)) == 1
    assert n(dims(B=64, Hv=32, S=4096)) == 1                                      # heads enough
    assert n(dims(B=1, S=100000, flags=gdn.GDN_SINGLE_PASS)) == 1
    assert L.gdn_linear_attn_workspace_bytes(None) == 0
    if not torch.cuda.is_available():
        assert L.gdn_linear_attn_workspace_bytes(dims(B=1, S=100000)) == 0


def rotary_dims(B=2, Hq=4, Hk=2, S=8, D=128, R=64, dtype=gdn.GDN_BF16, flags=0, qs=None, ks=None, qo=None, ko=None):
    hm = lambda H: (H * S * D, S * D, D)  # noqa: E731
    return gdn.GdnRotaryDims(B, Hq, Hk, S, D, R, *(qs or hm(Hq)), *(ks or hm(Hk)), *(qo or hm(Hq)), *(ko or hm(Hk)), S, 0,
                             dtype, flags, 1.0)


def test_rotary_argument_checks(L):
    def call(d, q=Q, k=K, f=V, pos=G, qo=OUT, ko=WS):
        return L.gdn_rotary(q, k, f, pos, qo, ko, d, None)
    D = rotary_dims
    assert call(None) == gdn.GDN_ERR_NULL
    assert call(D(B=0)) == gdn.GDN_OK and call(D(S=0)) == gdn.GDN_OK and call(D(Hq=0, Hk=0), f=None) == gdn.GDN_OK
    assert call(D(dtype=gdn.GDN_F8E4M3)) == gdn.GDN_ERR_UNSUPPORTED and call(D(flags=8)) == gdn.GDN_ERR_UNSUPPORTED
    for bad in (dict(B=-1), dict(S=-1), dict(Hq=-1), dict(Hk=-1), dict(R=0), dict(R=63), dict(R=130), dict(D=0),
                dict(D=4098, R=64), dict(Hq=65537), dict(S=1 << 30, B=2), dict(B=1 << 31)):
        assert call(D(**bad)) == gdn.GDN_ERR_DIMS, bad
    for name in ("q", "k", "f", "qo", "ko"):
        assert call(D(), **{name: None}) == gdn.GDN_ERR_NULL, name
    assert call(D(), f=V + 4) == gdn.GDN_ERR_ALIGN and call(D(), pos=G + 4) == gdn.GDN_ERR_ALIGN
    assert call(D(flags=gdn.GDN_ROTARY_POSITIONS_I32), pos=G + 2) == gdn.GDN_ERR_ALIGN
    assert call(D(), q=Q + 1) == gdn.GDN_ERR_ALIGN and call(D(dtype=gdn.GDN_F32), ko=WS + 2) == gdn.GDN_ERR_ALIGN
    # rows of an output over one another, negative strides
    assert call(D(qo=(4 * 8 * 128, 0, 128))) == gdn.GDN_ERR_DIMS
    assert call(D(qo=(4 * 8 * 128, 128, 128))) == gdn.GDN_ERR_DIMS
    assert call(D(qo=(4 * 8 * 128 - 1, 8 * 128, 128))) == gdn.GDN_ERR_DIMS
    assert call(D(ko=(2 * 8 * 128, 8 * 128, 127))) == gdn.GDN_ERR_DIMS
    assert call(D(qs=(4096, -1024, 128))) == gdn.GDN_ERR_DIMS
    # an output over its input, other than in place; over the frequencies
    assert call(D(), qo=Q + 256) == gdn.GDN_ERR_UNSUPPORTED
    assert call(D(qo=(4096, 128, 512)), qo=Q) == gdn.GDN_ERR_UNSUPPORTED
    assert call(D(), f=OUT) == gdn.GDN_ERR_UNSUPPORTED


def test_rotary_refuses_outputs_over_other_operands(L):
    D = rotary_dims
    call = lambda d, q=Q, k=K, pos=G, qo=OUT, ko=WS: L.gdn_rotary(q, k, V, pos, qo, ko, d, None)  # noqa: E731
    same = dict(Hq=2, Hk=2)
    assert call(D(**same), qo=K) == gdn.GDN_ERR_UNSUPPORTED                # q_out over k, k_out over q, one another
    assert call(D(**same), ko=Q) == gdn.GDN_ERR_UNSUPPORTED
    assert call(D(**same), qo=K, ko=Q) == gdn.GDN_ERR_UNSUPPORTED
    assert call(D(**same), qo=WS) == gdn.GDN_ERR_UNSUPPORTED
    assert call(D(**same), q=K, qo=K) == gdn.GDN_ERR_UNSUPPORTED           # q in place while k is the same rows
    assert call(D(**same), pos=OUT + 64) == gdn.GDN_ERR_UNSUPPORTED
    # packed rows of 6 heads (q 4, k 2), in place: k that begins one channel inside q's last head, or whose last
    # head runs into the next token's q
    row = dict(qs=(8 * 768, 128, 768), ks=(8 * 768, 128, 768), qo=(8 * 768, 128, 768), ko=(8 * 768, 128, 768))
    assert call(D(**row), k=Q + 2 * 511, qo=Q, ko=Q + 2 * 511) == gdn.GDN_ERR_UNSUPPORTED
    assert call(D(**row), k=Q + 2 * 513, qo=Q, ko=Q + 2 * 513) == gdn.GDN_ERR_UNSUPPORTED
    assert call(D(**row), k=Q - 2 * 255, qo=Q, ko=Q - 2 * 255) == gdn.GDN_ERR_UNSUPPORTED
    # other strides, which show nothing
    assert call(D(**dict(row, ks=(8 * 700, 128, 700))), k=Q + 1024, qo=Q, ko=WS) == gdn.GDN_ERR_UNSUPPORTED


def test_rotary_refuses_strides_past_64_bits(L):
    D = rotary_dims
    call = lambda d: L.gdn_rotary(Q, K, V, G, OUT, WS, d, None)  # noqa: E731
    far = 1 << 56
    for name in ("qs", "ks", "qo", "ko"):
        assert call(D(**{name: (far + 1, 8 * 128, 128)})) == gdn.GDN_ERR_DIMS, name
    assert call(D(B=3, Hq=1, S=1, R=64, qs=(far // 2 + 1, 128, 128))) == gdn.GDN_ERR_DIMS
    assert call(D(B=1 << 20, Hq=1, Hk=1, S=1, qs=(1 << 40, 128, 128))) == gdn.GDN_ERR_DIMS
    for stride in (-1, far + 1):
        d = D()
        d.position_stride = stride
        assert call(d) == gdn.GDN_ERR_DIMS


def test_bindings_refuse_host_tensors():
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    with pytest.raises(ValueError):
        gdn.linear_attn_prefill(bf(1, 1, 4, 8), bf(1, 1, 4, 8), bf(1, 1, 4, 8), torch.zeros(1), 1.0)
    with pytest.raises(ValueError):
        gdn.linear_attn_step(bf(1, 1, 1, 8), bf(1, 1, 1, 8), bf(1, 1, 1, 8), torch.zeros(1), 1.0, torch.zeros(1, 1, 8, 8))
    with pytest.raises(ValueError):
        gdn.rotary(bf(1, 1, 1, 8), None, torch.zeros(4, dtype=torch.float64))


def test_rotary_frequencies():
    f, amp = gdn.rotary_frequencies(128)
    assert f.dtype == torch.float64 and f.shape == (64,) and amp == 1.0
    want = np.array([10000.0 ** (-2 * i / 128) for i in range(64)])
    assert np.abs(f.numpy() / want - 1).max() < 1e-14
    g, amp = gdn.rotary_frequencies(128, scaling="linear", factor=4.0)
    assert torch.equal(g, f / 4) and amp == 1.0
    g, amp = gdn.rotary_frequencies(128, scaling="ntk", factor=4.0)
    assert g[0] == 1.0 and abs(float(g[-1] / f[-1]) - 0.25) < 1e-12 and amp == 1.0
    g, amp = gdn.rotary_frequencies(128, scaling="yarn", factor=4.0, original_length=4096)
    # pairs that turn more than 32 times over 4096 positions are left, those below one turn are slowed by 4
    turns = 4096 * f / (2 * math.pi)
    assert torch.equal(g[:20], f[:20]) and (turns[:20] > 32).all()
    assert torch.allclose(g[turns < 0.8], f[turns < 0.8] / 4, rtol=1e-14, atol=0)
    assert (g <= f).all() and (g >= f / 4 * (1 - 1e-14)).all() and abs(amp - (0.1 * math.log(4) + 1)) < 1e-15
    g, amp = gdn.rotary_frequencies(128, scaling="bands", factor=8.0, original_length=8192, fast_turns=4.0)
    turns = 8192 * f / (2 * math.pi)
    assert torch.equal(g[turns > 4.0], f[turns > 4.0]) and torch.allclose(g[turns < 1], f[turns < 1] / 8, rtol=1e-14)
    assert amp == 1.0
    for bad in (dict(rotary_dim=3), dict(rotary_dim=0), dict(rotary_dim=8, base=0.0), dict(rotary_dim=8, factor=0.5),
                dict(rotary_dim=8, scaling="yarn"), dict(rotary_dim=8, scaling="other"), dict(rotary_dim=2, scaling="ntk")):
        with pytest.raises(ValueError):
            gdn.rotary_frequencies(**bad)


def test_oracle_linear_attn_hand_worked():
    # one head, Dk = Dv = 1, g = ln(1/2): S = 3, then 3/2 + 2 * 5 = 11.5, then 5.75 - 4 = 1.75
    q, k, v = (np.array(x, dtype=np.float64).reshape(1, 1, 3, 1) for x in ([1, 2, 4], [1, 2, -4], [3, 5, 1]))
    g = np.full((1, 1, 3), math.log(0.5))
    o, s, _ = ref.recurrence(q, k, v, g, 2.0)
    assert np.allclose(o.ravel(), [6.0, 46.0, 14.0], rtol=1e-15) and np.allclose(s.ravel(), [1.75])
    o, s, _ = ref.recurrence(q, k, v, g[0, :, 0], 2.0, state=np.full((1, 1, 1, 1), 4.0), lengths=[2])
    assert np.allclose(o.ravel(), [10.0, 50.0, 0.0]) and np.allclose(s.ravel(), [12.5])


def test_oracle_rotary_hand_worked():
    x = np.array([1.0, 2.0, 3.0, 4.0, 5.0]).reshape(1, 1, 1, 5)
    f = np.array([math.pi / 2, 0.0])
    assert np.allclose(ref.rotary(x, f, np.array([1])).ravel(), [-3, 2, 1, 4, 5])           # pairs (0, 2), (1, 3)
    assert np.allclose(ref.rotary(x, f, np.array([1]), "interleaved").ravel(), [-2, 1, 3, 4, 5])
    # a far position turns as its remainder does, and back again
    y = ref.rotary(x, np.array([2 * math.pi / 1024, 0.25]), np.array([1024 * 1000000 + 256]))
    assert np.allclose(y[..., [0, 2]].ravel(), [-3, 1], atol=1e-6)
    z = ref.rotary(y, np.array([2 * math.pi / 1024, 0.25]), np.array([1024 * 1000000 + 256]), inverse=True)
    assert np.allclose(z, x, atol=1e-12)


@pytest.mark.parametrize("bad", [dict(base=1.0, scaling="yarn"), dict(base=0.5, scaling="yarn"), dict(base=math.inf),
                                 dict(base=math.nan), dict(factor=math.inf, scaling="linear"), dict(factor=math.nan)],
                         ids=str)
def test_rotary_frequencies_that_have_none(bad):
    """The ramp of "yarn" is over log base, which is zero or falls; infinite bases and factors leave no frequency."""
    with pytest.raises(ValueError):
        gdn.rotary_frequencies(16, original_length=4096, **bad)


def test_rotary_frequencies_of_one_base():
    for scaling in (None, "linear", "bands"):  # (bases up to 1 are nobody's, and these forms have no trouble with them)
        f, _ = gdn.rotary_frequencies(16, 1.0, scaling=scaling, factor=2.0, original_length=4096)
        assert torch.isfinite(f).all() and (f > 0).all()
