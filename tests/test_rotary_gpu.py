"""rotary against whole-number angles in fp64 (oracle/linear_attn.py)."""
import numpy as np
import pytest
import torch

import gated_delta_rule_20_gb300 as gdn
from oracle import linear_attn as ref

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def check(got, x, f, pos, dtype, R, layout="half", amplitude=1.0, inverse=False):
    """Each element within: half a step of its type, and for each of the two products cos and sin to 2^-22 of one (their
    function and their angle in fp32), the amplitude's and the product's roundings: 2^-21 of |a| + |b| in all."""
    want = ref.rotary(x, f.cpu().numpy(), pos, layout, amplitude, inverse)
    got = got.double().cpu().numpy()
    a = np.abs(x.double().cpu().numpy())
    size = np.zeros_like(a)
    if layout == "half":
        size[..., :R // 2] = size[..., R // 2:R] = a[..., :R // 2] + a[..., R // 2:R]
    else:
        size[..., 0:R:2] = size[..., 1:R:2] = a[..., 0:R:2] + a[..., 1:R:2]
    most = amplitude * size * 2.0 ** -21 * (1 + HALF[dtype]) + HALF[dtype] * np.abs(want) + 1e-38
    most[..., R:] = 0
    worst = np.max(np.abs(got - want) - most)
    assert worst <= 0, "off by %.3g more than allowed" % worst


def freq(R, base=10000.0):
    return gdn.rotary_frequencies(R, base, device="cuda")[0]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("B, Hq, Hk, S, D, R", [
    (1, 1, 1, 1, 128, 128), (2, 3, 1, 5, 128, 64), (1, 16, 16, 1, 128, 128), (3, 2, 2, 17, 80, 80), (1, 2, 1, 33, 90, 46),
    (2, 1, 2, 7, 5, 2), (1, 1, 1, 9, 2, 2), (2, 2, 1, 40, 256, 84), (70, 4, 0, 1, 64, 32), (1, 2, 1, 700, 96, 24),
    (1, 1, 1, 3, 1000, 998), (1, 65, 1, 2, 64, 64)])
def test_rotary(B, Hq, Hk, S, D, R, dtype, layout):
    gen = torch.Generator().manual_seed(B * S + D)
    q, k = (torch.randn(B, h, S, D, generator=gen).to(TYPES[dtype]).cuda() for h in (Hq, Hk))
    f = freq(R)
    at = torch.randint(0, 1 << 20, (B, 1), generator=gen) + torch.arange(S)
    yq, yk = gdn.rotary(q, k if Hk else None, f, at.cuda(), layout=layout)
    assert yq.is_contiguous() and (yk is None) == (Hk == 0)
    check(yq, q, f, at.numpy(), dtype, R, layout)
    if Hk:
        check(yk, k, f, at.numpy(), dtype, R, layout)
    # in place, int32 positions: the same bits
    a, b = q.clone(), k.clone() if Hk else None
    gdn.rotary(a, b, f, at.to(torch.int32).cuda(), layout=layout, q_out=a, k_out=b)
    assert torch.equal(a, yq) and (not Hk or torch.equal(b, yk))


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_packed_rows(layout):
    """q and k as views into q | k | v rows, into new tensors and in place (v untouched); token-major outputs."""
    B, S, H, D, R = 2, 13, 3, 64, 48
    rows = torch.randn(B, S, 3 * H * D, device="cuda").to(torch.bfloat16)
    before = rows.clone()
    view = lambda r, i: r[..., i * H * D:(i + 1) * H * D].view(B, S, H, D).transpose(1, 2)  # noqa: E731
    f, pos = freq(R), np.arange(S) + 5
    yq, yk = gdn.rotary(view(rows, 0), view(rows, 1), f, first_position=5, layout=layout)
    check(yq, view(rows, 0), f, pos, "bf16", R, layout)
    check(yk, view(rows, 1), f, pos, "bf16", R, layout)
    tm = torch.empty(B, S, H, D, device="cuda", dtype=torch.bfloat16)
    gdn.rotary(view(rows, 0), None, f, torch.arange(5, 5 + S, device="cuda"), layout=layout, q_out=tm.transpose(1, 2))
    assert torch.equal(tm.transpose(1, 2), yq)
    gdn.rotary(view(rows, 0), view(rows, 1), f, first_position=5, layout=layout, q_out=view(rows, 0), k_out=view(rows, 1))
    assert torch.equal(view(rows, 0), yq) and torch.equal(view(rows, 1), yk)
    assert torch.equal(rows[..., 2 * H * D:], before[..., 2 * H * D:])


def test_odd_strides_and_offsets():
    """Rows at odd element offsets and pitches, and an input that is broadcast over the batch and the heads."""
    B, H, S, D, R = 2, 3, 6, 32, 32
    for dt in TYPES:
        buf = torch.randn(B * H * S * (D + 3) + 1, device="cuda").to(TYPES[dt])
        x = buf[1:].view(B, H, S, D + 3)[..., :D]
        f = freq(R)
        for layout in ("half", "interleaved"):
            y, _ = gdn.rotary(x, None, f, layout=layout)
            check(y, x, f, np.arange(S), dt, R, layout)
            one = x[:1, :1].expand(B, H, S, D)
            y, _ = gdn.rotary(one, None, f, layout=layout)
            check(y, one, f, np.arange(S), dt, R, layout)


@pytest.mark.parametrize("start", [0, 1 << 20, (1 << 31) - 5, 1 << 40, -(1 << 33)])
def test_far_positions(start):
    """The angles of far positions are as exact as those of near ones."""
    x = torch.randn(1, 2, 6, 128, device="cuda")
    f = freq(128)
    pos = start + np.arange(6)
    for kw in (dict(first_position=start), dict(positions=torch.from_numpy(pos).cuda())):
        y, _ = gdn.rotary(x, None, f, **kw)
        if abs(start) > 1 << 35:  # (2^-64 of a turn a position)
            want = ref.rotary(x, f.cpu().numpy(), pos)
            assert np.abs(y.double().cpu().numpy() - want).max() < 1e-5
        else:
            check(y, x, f, pos, "f32", 128)


def test_frequencies_of_any_size():
    x = torch.randn(1, 1, 4, 24, device="cuda")
    f = torch.tensor([0.0, 1.0, -0.3, 3.0, 7.5, 1e5, 2.0 ** -40, 1e-300, -4e3, 123456.789, 2 * np.pi, 5e-324],
                     dtype=torch.float64, device="cuda")
    pos = np.array([0, 1, 3, 1000])
    y, _ = gdn.rotary(x, None, f, torch.from_numpy(pos).cuda())
    want = ref.rotary(x, f.cpu().numpy(), pos)
    # 53 bits of a frequency of 1e5 radians leave 2^-36 of a turn; positions to 1000
    assert np.abs(y.double().cpu().numpy() - want).max() < 3e-6
    f[3], f[4] = float("inf"), float("nan")
    z, _ = gdn.rotary(x, None, f, torch.from_numpy(pos).cuda())
    assert torch.equal(z[..., 3], x[..., 3]) and torch.equal(z[..., 16], x[..., 16]) and torch.equal(z[..., 5], y[..., 5])


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_inverse_is_the_gradient(layout):
    """<dy, rotary(x)> differentiates to the inverse of dy: against differences, and against the formula's transpose."""
    D, R, S = 20, 12, 5
    f, amp = freq(R), 1.25
    x, dy = (torch.randn(1, 2, S, D, device="cuda") for _ in range(2))
    dx, _ = gdn.rotary(dy, None, f, layout=layout, amplitude=amp, inverse=True)
    check(dx, dy, f, np.arange(S), "f32", R, layout, amp, True)
    # the map is linear: differences over unit steps are exact up to rounding
    for c in range(D):
        e = torch.zeros_like(x)
        e[..., c] = 1.0
        y, _ = gdn.rotary(e, None, f, layout=layout, amplitude=amp)
        assert torch.allclose((y * dy).sum(-1), dx[..., c], rtol=0, atol=1e-5)
    back, _ = gdn.rotary(gdn.rotary(x, None, f, layout=layout)[0], None, f, layout=layout, inverse=True)
    assert torch.allclose(back, x, rtol=0, atol=4e-6)


def test_refusals():
    x = torch.zeros(2, 2, 4, 16, device="cuda", dtype=torch.bfloat16)
    f = freq(16)
    for bad in (dict(q=x[0]), dict(q=x.transpose(2, 3)), dict(k=x[:1]), dict(k=x.float()), dict(layout="other"),
                dict(positions=torch.zeros(3, dtype=torch.int64, device="cuda")), dict(q_out=x[:1]), dict(q=x.cpu()),
                dict(k_out=x, k=None)):
        with pytest.raises(ValueError):
            gdn.rotary(**dict(dict(q=x, k=x.clone(), inv_freq=f), **bad))
    for bad in (dict(q=x.half()), dict(inv_freq=f.float()), dict(positions=torch.zeros(4, device="cuda"))):
        with pytest.raises(TypeError):
            gdn.rotary(**dict(dict(q=x, k=None, inv_freq=f), **bad))
    with pytest.raises(gdn.GdnError):
        gdn.rotary(x, None, freq(32))                                  # more channels than the head has
    with pytest.raises(gdn.GdnError):
        gdn.rotary(x, None, f, q_out=x[:1, :1].expand(2, 2, 4, 16))    # rows over one another
    flat = torch.zeros(2 * 2 * 4 * 16 + 8, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(gdn.GdnError):
        gdn.rotary(flat[:256].view(2, 2, 4, 16), None, f, q_out=flat[8:].view(2, 2, 4, 16))


def test_more_heads_than_a_grid_has_parts():
    # one token of 2 x 65536 heads: a thread takes two heads, for want of a 65536th row of blocks
    q, k = (torch.randn(1, 65536, 1, 2, generator=torch.Generator().manual_seed(i)).cuda() for i in (1, 2))
    f = freq(2)
    yq, yk = gdn.rotary(q, k, f, first_position=3)
    check(yq, q, f, np.array([3]), "f32", 2)
    check(yk, k, f, np.array([3]), "f32", 2)


def test_heads_of_q_and_k_in_turn_in_place():
    # [B, S, H, 2, D]: every q head beside its k head, and [B, 2, H, S, D]: q's heads before k's within a sequence
    B, S, H, D = 2, 5, 3, 16
    f = freq(D)
    for shape, q_of, k_of in (((B, S, H, 2, D), lambda x: x[:, :, :, 0].transpose(1, 2), lambda x: x[:, :, :, 1].transpose(1, 2)),
                              ((B, 2, H, S, D), lambda x: x[:, 0], lambda x: x[:, 1])):
        x = torch.randn(shape, generator=torch.Generator().manual_seed(len(shape))).cuda()
        was = x.clone()
        gdn.rotary(q_of(x), k_of(x), f, first_position=7, q_out=q_of(x), k_out=k_of(x))
        check(q_of(x), q_of(was), f, np.arange(7, 7 + S), "f32", D)
        check(k_of(x), k_of(was), f, np.arange(7, 7 + S), "f32", D)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_large_frequencies_at_far_positions(layout):
    """inv_freq far above 1, where f = inv_freq / 2 pi mod 1 is off by 1.5 * 2^-64 of a turn times inv_freq: in front of
    cos and sin's own 2^-21 of |a| + |b| the angle's error, 2 pi times that and the position, moves an output by at most
    as much of |a| + |b| again."""
    f = torch.tensor([1.0, 3.7, 1e3, -2.5e4, 1e6, 7e8, -1e10, 3e11], dtype=torch.float64, device="cuda")
    R = 16
    x = torch.randn(1, 2, 5, R, generator=torch.Generator().manual_seed(2)).cuda()
    pos = np.array([0, 1, 1000, (1 << 20) + 1, -(1 << 21)])
    y, _ = gdn.rotary(x, None, f, torch.from_numpy(pos).cuda(), layout=layout)
    want = ref.rotary(x, f.cpu().numpy(), pos, layout)
    a = np.abs(x.double().cpu().numpy())
    ia, ib = (slice(0, 8), slice(8, 16)) if layout == "half" else (slice(0, 16, 2), slice(1, 16, 2))
    angle = 2 * np.pi * 1.5 * 2.0 ** -64 * np.abs(pos)[:, None] * np.maximum(1, np.abs(f.cpu().numpy()))
    for i in (ia, ib):
        most = (a[..., ia] + a[..., ib]) * (2.0 ** -21 + angle) + 2.0 ** -24 * np.abs(want[..., i])
        off = np.abs(y.double().cpu().numpy()[..., i] - want[..., i])
        assert (off <= most).all(), "%.3g times what is allowed" % (off / most).max()
