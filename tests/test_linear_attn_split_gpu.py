"""linear_attn_prefill in segments, over several sequences a CTA, from graphs, other streams and host threads."""
import threading

import numpy as np
import pytest
import torch

import gated_delta_rule_20_gb300 as gdn
from oracle import linear_attn as ref
from test_linear_attn_gpu import TYPES, compare, inputs

pytestmark = pytest.mark.gpu


def call(x, scale=0.1, **kw):
    d = {n: t.cuda() if t is not None else None for n, t in x.items()}
    if kw.get("lengths") is not None:
        kw["lengths"] = torch.tensor(kw["lengths"], dtype=torch.int32, device="cuda")
    return gdn.linear_attn_prefill(d["q"], d["k"], d["v"], d["g"], scale, d["state"], **kw)


def rel(a, b):
    a, b = a.double(), b.double()
    return float((a - b).norm() / b.norm().clamp_min(1e-30))


@pytest.mark.parametrize("B, Hk, Hv, S, Dk, Dv, dtype, decay, lengths", [
    (1, 1, 1, 2000, 128, 128, "bf16", "weak", None),
    (1, 1, 2, 1153, 128, 64, "bf16", "head", None),
    (3, 1, 1, 1500, 64, 128, "bf16", "token", [1500, 700, 0]),
    (2, 1, 1, 1300, 128, 128, "bf16", "none", [1025, 129]),
    (1, 1, 2, 300, 128, 128, "f32", "weak", None),
    (3, 1, 1, 333, 64, 40, "f32", "token", [333, 100, 0]),
    (1, 1, 1, 200, 33, 75, "f32", "head", None),
    (2, 2, 2, 250, 30, 50, "bf16", "token", None)])
def test_segments(B, Hk, Hv, S, Dk, Dv, dtype, decay, lengths):
    """Few sequences: cut into segments, against fp64, from a state and from none, in place, and against one pass."""
    code = gdn.GDN_BF16 if dtype == "bf16" else gdn.GDN_F32
    P = gdn.linear_attn_segments(B, Hk, Hv, S, Dk, Dv, code)
    assert P > 2
    tc = dtype == "bf16" and Dk % 8 == 0 and Dv % 8 == 0
    for start in (True, False):
        x = inputs(B, Hk, Hv, S, Dk, Dv, dtype, decay, start, seed=S)
        out, st, size = ref.recurrence(x["q"], x["k"], x["v"], x["g"], 0.1, x["state"], lengths)
        y = call(x, lengths=lengths)
        # (a segment's start state is rounded once more a segment: 2^-24 of it each, within the bound's margin for one)
        compare(y, (out, st), (size[0], size[1], size[2] + P * size[0], size[3] + P * size[1]), dtype, tc, "segments")
        one = call(x, lengths=lengths, single_pass=True)
        assert rel(y[1], one[1]) < 1e-6 and rel(y[0], one[0]) < (5e-3 if dtype == "bf16" else 1e-6)
    # the workspace: the size that the query says, anything in it before
    need = gdn.linear_attn_workspace_bytes(B, Hk, Hv, S, Dk, Dv, code)
    assert need > 0
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    z = call(x, lengths=lengths, workspace=ws)
    assert torch.equal(z[0], y[0]) and torch.equal(z[1], y[1])
    with pytest.raises(gdn.GdnError) as e:
        call(x, lengths=lengths, workspace=ws[:need - 16])
    assert e.value.code == gdn.GDN_ERR_WORKSPACE


def test_segments_from_the_library_itself():
    """No workspace: the library's own scratch, by the C entry point."""
    x = inputs(1, 1, 1, 1000, 128, 128, "bf16")
    y = call(x)
    d = {n: t.cuda() for n, t in x.items()}
    out, st = torch.empty_like(d["v"]), torch.empty_like(d["state"])
    dims = gdn.make_dims(1, 1, 1, 1000, 128, 128, gdn.GDN_BF16)
    code = gdn.lib().gdn_linear_attn_prefill(d["q"].data_ptr(), d["k"].data_ptr(), d["v"].data_ptr(), d["g"].data_ptr(), None,
                                             0.1, d["state"].data_ptr(), st.data_ptr(), out.data_ptr(), dims, None, 0,
                                             torch.cuda.current_stream().cuda_stream)
    assert code == gdn.GDN_OK
    assert torch.equal(out, y[0]) and torch.equal(st, y[1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_sequences_a_cta(dtype):
    """More sequences than CTAs, of unequal lengths, some of them empty: the pipeline runs through from one to the next."""
    B, Hk, Hv, S, D = 130, 1, 3, 290, 64
    gen = torch.Generator().manual_seed(5)
    lengths = torch.randint(0, S + 1, (B,), generator=gen)
    lengths[::7] = 0
    lengths[3::11] = S
    x = inputs(B, Hk, Hv, S, D, D, dtype, "token", True, seed=9)
    lens = lengths.tolist()
    y = call(x, lengths=lens)
    some = [0, 1, 3, 7, 50, 51, 52, 100, 128, 129]
    part = {n: t[some] if n != "g" or t.dim() == 3 else t for n, t in x.items()}
    out, st, size = ref.recurrence(part["q"], part["k"], part["v"], part["g"], 0.1, part["state"], [lens[i] for i in some])
    compare((y[0][some], y[1][some]), (out, st), size, dtype, dtype == "bf16", "many")
    # and each of them by itself, bit for bit (one pass: the same sums)
    for i in (0, 3, 129):
        one = {n: t[i:i + 1].contiguous() for n, t in x.items()}
        z = call(one, lengths=[lens[i]], single_pass=True)
        assert torch.equal(z[0][0], y[0][i]) and torch.equal(z[1][0], y[1][i])


def test_long_offsets():
    """Rows whose offsets pass 2^31 elements: the last sequence and the last tokens are right."""
    B, S, D = 1, 1 << 20, 64
    Hv = 33  # 33 x 2^20 x 64 = 2.2e9 elements of v and out
    gen = torch.Generator(device="cuda").manual_seed(1)
    q, k = (torch.randn(B, 1, S, D, generator=gen, device="cuda").to(torch.bfloat16) for _ in range(2))
    v = torch.empty(B, Hv, S, D, dtype=torch.bfloat16, device="cuda")
    for h in range(Hv):
        v[:, h].normal_(generator=gen)
    g = torch.full((Hv,), -0.4, device="cuda")
    out, st = gdn.linear_attn_prefill(q, k, v, g, 0.1)
    n = 200  # (e^-80 is left of what came before)
    for h in (0, Hv - 1):
        tail = lambda t, i: t[:, i:i + 1, -n:].cpu()  # noqa: E731
        o, s, size = ref.recurrence(tail(q, 0), tail(k, 0), tail(v, h), g[:1].cpu(), 0.1)
        got = out[:, h:h + 1, -100:]
        compare((got, st[:, h:h + 1]), (o[:, :, -100:], s), (size[0][:, :, -100:], size[1], size[2][:, :, -100:], size[3]), "bf16",
                True, "tail")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_graph_stream_and_threads(dtype):
    """A captured and replayed call; one on another stream; two host threads on streams of their own."""
    x = inputs(1, 1, 2, 900, 64, 64, dtype)
    want = call(x)
    d = {n: t.cuda() for n, t in x.items()}
    scale = 0.1
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = gdn.linear_attn_prefill(d["q"], d["k"], d["v"], d["g"], scale, d["state"], state_out=torch.empty_like(d["state"]),
                                stream=side)
    side.synchronize()
    assert torch.equal(y[0], want[0]) and torch.equal(y[1], want[1])

    out, st = torch.empty_like(d["v"]), torch.empty_like(d["state"])
    with torch.cuda.stream(side):
        gdn.linear_attn_prefill(d["q"], d["k"], d["v"], d["g"], scale, d["state"], out, state_out=st)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdn.linear_attn_prefill(d["q"], d["k"], d["v"], d["g"], scale, d["state"], out, state_out=st)
    for _ in range(3):
        out.fill_(float("nan"))
        st.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(st, want[1])

    errors = []

    def work():
        try:
            s = torch.cuda.Stream()
            for _ in range(20):
                a = gdn.linear_attn_prefill(d["q"], d["k"], d["v"], d["g"], scale, d["state"],
                                            state_out=torch.empty_like(d["state"]), stream=s)
                s.synchronize()
                if not (torch.equal(a[0], want[0]) and torch.equal(a[1], want[1])):
                    errors.append("another result")
        except Exception as e:  # noqa: BLE001
            errors.append(repr(e))
    threads = [threading.Thread(target=work) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors and gdn.device_status(0) == 0


def test_the_same_bits_every_time():
    """Results do not depend on what else runs: the same call, alone and among others, gives the same bits."""
    x = inputs(4, 2, 8, 700, 128, 128, "bf16", "strong")
    want = call(x)
    d = {n: t.cuda() for n, t in x.items()}
    noise = torch.randn(4096, 4096, device="cuda")
    side = torch.cuda.Stream()
    for _ in range(5):
        with torch.cuda.stream(side):
            noise = noise @ noise * 1e-3
        y = gdn.linear_attn_prefill(d["q"], d["k"], d["v"], d["g"], 0.1, d["state"], state_out=torch.empty_like(d["state"]))
        assert torch.equal(y[0], want[0]) and torch.equal(y[1], want[1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_infinities_and_nan_in_the_data(dtype):
    """A NaN in one head's v reaches that head's column alone, from its token on; other heads are bit for bit the same."""
    x = inputs(2, 1, 2, 300, 64, 64, dtype)
    want = call(x)
    x["v"][1, 1, 140, 5] = float("nan")
    y = call(x)
    assert torch.equal(y[0][0], want[0][0]) and torch.equal(y[0][1, 0], want[0][1, 0])
    assert bool(torch.isnan(y[0][1, 1, 140:, 5]).all()) and not bool(torch.isnan(y[0][1, 1, :128, 5]).any())
    keep = [c for c in range(64) if c != 5]
    assert torch.equal(y[0][1, 1][:, keep], want[0][1, 1][:, keep]) and torch.equal(y[1][1, 1][:, keep], want[1][1, 1][:, keep])
    assert bool(torch.isnan(y[1][1, 1, :, 5]).all())


@pytest.mark.parametrize("rounds, rest, S, Dk, Dv, start", [
    (1, 8, 1500, 128, 128, True), (1, 8, 1024, 64, 128, False), (2, 3, 2000, 96, 64, True), (3, 56, 2048, 128, 128, True),
    (1, 76, 1100, 8, 128, True), (4, 1, 3001, 128, 8, True)])
def test_heads_handed_on(rounds, rest, S, Dk, Dv, start):
    """A few heads more than whole rounds of all SMs: they are run in parts by CTAs that hand their states on.  The bits are one
    pass's, with lengths (some end in an early part) and without, in place, from a graph, on two streams at once."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    Hv = rounds * sms + rest
    gen = torch.Generator(device="cuda").manual_seed(S)
    n = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    q, k, v = n(1, 1, S, Dk).bfloat16(), n(1, 1, S, Dk).bfloat16(), n(1, Hv, S, Dv).bfloat16()
    g = -0.2 * torch.rand(1, Hv, S, generator=gen, device="cuda")
    state = n(1, Hv, Dk, Dv) if start else None
    assert gdn.linear_attn_segments(1, 1, Hv, S, Dk, Dv) == 1
    assert gdn.linear_attn_workspace_bytes(1, 1, Hv, S, Dk, Dv) > 0                     # (they are handed on)
    assert gdn.linear_attn_workspace_bytes(1, 1, Hv, S, Dk, Dv, single_pass=True) == 0
    new = lambda: torch.full((1, Hv, Dk, Dv), float("nan"), device="cuda")  # noqa: E731
    call = lambda **kw: gdn.linear_attn_prefill(q, k, v, g, 0.1, state, state_out=new(), **kw)  # noqa: E731
    want = call(single_pass=True)
    for _ in range(3):
        y = call()
        assert torch.equal(y[0], want[0]) and torch.equal(y[1], want[1])
    last = slice(Hv - 1, Hv)
    o, st, size = ref.recurrence(q.cpu(), k.cpu(), v[:, last].cpu(), g[:, last].cpu(), 0.1, state[:, last].cpu() if start else None)
    compare((want[0][:, last], want[1][:, last]), (o, st), size, "bf16", True, "handed on")
    for length in (0, 1, S // 2 - 1, S - 1, 130):
        at = torch.tensor([length], dtype=torch.int32, device="cuda")
        a, b = call(lengths=at), call(lengths=at, single_pass=True)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    if start:
        s = state.clone()
        y = gdn.linear_attn_prefill(q, k, v, g, 0.1, s)
        assert y[1] is s and torch.equal(s, want[1]) and torch.equal(y[0], want[0])
    # two streams at once, each with its own scratch
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    ys = [call(stream=st) for _ in range(3) for st in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(y[0], want[0]) and torch.equal(y[1], want[1]) for y in ys)
    out, st = torch.empty_like(v), new()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdn.linear_attn_prefill(q, k, v, g, 0.1, state, out, state_out=st)
    for _ in range(2):
        out.zero_()
        st.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(st, want[1])
    assert gdn.device_status(0) == 0


@pytest.mark.parametrize("Hv, S, dtype", [(2, 1000, "bf16"), (160, 1100, "bf16"), (2, 300, "f32")])
def test_own_scratch_in_a_graph(Hv, S, dtype):
    """The C entry point without a workspace, captured: segments, heads handed on, and the FMA units' segments, with zeroed padding;
    two graphs of the same call keep their own scratch."""
    code = gdn.GDN_BF16 if dtype == "bf16" else gdn.GDN_F32
    assert gdn.linear_attn_workspace_bytes(1, 1, Hv, S, 64, 64, code) > 0
    gen = torch.Generator(device="cuda").manual_seed(3)
    n = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(TYPES[dtype])  # noqa: E731
    q, k, v, g = n(1, 1, S, 64), n(1, 1, S, 64), n(1, Hv, S, 64), torch.full((Hv,), -0.01, device="cuda")
    at = torch.tensor([S - 70], dtype=torch.int32, device="cuda")
    want = gdn.linear_attn_prefill(q, k, v, g, 0.1, lengths=at)
    dims = gdn.make_dims(1, 1, Hv, S, 64, 64, code, gdn.GDN_HEAD_DECAY | gdn.GDN_ZERO_PADDING)
    graphs = []
    for _ in range(2):
        out, st = torch.empty_like(v), torch.empty_like(want[1])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            assert gdn.lib().gdn_linear_attn_prefill(
                q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), at.data_ptr(), 0.1, None, st.data_ptr(), out.data_ptr(),
                dims, None, 0, torch.cuda.current_stream().cuda_stream) == gdn.GDN_OK
        graphs.append((graph, out, st))
    for _ in range(2):
        for graph, out, st in graphs:
            out.fill_(float("nan"))
            st.fill_(float("nan"))
        for graph, out, st in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for graph, out, st in graphs:
            assert torch.equal(out, want[0]) and torch.equal(st, want[1])
    assert gdn.device_status(0) == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("Dk", [30, 64, 65, 96, 97, 128])
def test_widest_ctas_of_the_fma_units(Dk, dtype):
    """Heads enough for CTAs of 128 columns, whose tokens' shared memory is 48 KB with 65 to 96 rows, at every number of rows."""
    x = inputs(40, 4, 8, 19, Dk, 127, dtype)
    out, st, size = ref.recurrence(x["q"], x["k"], x["v"], x["g"], 0.1, x["state"])
    y = call(x, force_ffma=True)
    compare(y, (out, st), size, dtype, False, "wide")
