"""linear_attn_prefill in bf16 with channels that are no multiple of 8: large calls run on the tensor cores, on padded rows."""
import pytest
import torch

import gated_delta_rule_20_gb300 as gdn
from oracle import linear_attn as ref
from test_linear_attn_gpu import compare, inputs

pytestmark = pytest.mark.gpu


def bytes_of(x, **kw):
    B, Hk, S, Dk = x["q"].shape
    return gdn.linear_attn_workspace_bytes(B, Hk, x["v"].shape[1], S, Dk, x["v"].shape[3], **kw)


@pytest.mark.parametrize("B, Hk, Hv, S, Dk, Dv, decay, lengths", [
    (2, 1, 4, 3300, 77, 75, "token", None),
    (1, 2, 2, 7001, 90, 121, "weak", None),
    (3, 1, 3, 1400, 128, 127, "head", [1400, 700, 0]),
    (4, 2, 4, 1100, 73, 128, "strong", [1100, 1, 129, 1023]),
    (40, 3, 6, 300, 65, 33, "token", None),
    (1, 1, 1, 700, 77, 75, "head", None),
    (8, 4, 4, 100, 33, 35, "token", [100, 0, 1, 31, 32, 33, 99, 64]),
    (64, 16, 32, 2, 100, 100, "token", None),
    (150, 1, 3, 64, 1, 128, "weak", None),
    (300, 1, 1, 90, 128, 1, "token", None)])
def test_padded_rows(B, Hk, Hv, S, Dk, Dv, decay, lengths):
    assert B * Hv * S * Dk * Dv > 3e6
    x = inputs(B, Hk, Hv, S, Dk, Dv, "bf16", decay, True, seed=S)
    need = bytes_of(x, single_pass=True)
    assert need >= 2 * (x["q"].numel() if Dk % 8 else x["v"].numel())
    out, st, size = ref.recurrence(x["q"], x["k"], x["v"], x["g"], 0.1, x["state"], lengths)
    P = gdn.linear_attn_segments(B, Hk, Hv, S, Dk, Dv)
    d = {n: t.cuda() for n, t in x.items()}
    at = torch.tensor(lengths, dtype=torch.int32, device="cuda") if lengths else None
    if lengths:
        for b, n in enumerate(lengths):
            for name in ("q", "k", "v"):
                d[name][b, :, n:] = float("nan")
    call = lambda **kw: gdn.linear_attn_prefill(d["q"], d["k"], d["v"], d["g"], 0.1, d["state"], lengths=at,  # noqa: E731
                                                state_out=torch.full_like(d["state"], float("nan")), **kw)
    y = call()
    compare(y, (out, st), (size[0], size[1], size[2] + P * size[0], size[3] + P * size[1]), "bf16", True, "padded")
    z = call(single_pass=True, workspace=torch.full((need,), 255, dtype=torch.uint8, device="cuda"))
    compare(z, (out, st), size, "bf16", True, "padded, one pass")
    with pytest.raises(gdn.GdnError) as e:
        call(single_pass=True, workspace=torch.zeros(need - 16, dtype=torch.uint8, device="cuda"))
    assert e.value.code == gdn.GDN_ERR_WORKSPACE
    # rows behind a length stay as they were in an out that is given
    given = torch.full_like(d["v"], 7.0)
    w = call(out=given)
    assert w[0] is given and torch.equal(w[1], y[1])
    for b, n in enumerate(lengths or [S] * B):
        assert torch.equal(given[b, :, :n], y[0][b, :, :n]) and bool((given[b, :, n:] == 7.0).all())
    # operands that begin off 16 bytes: the same bits
    off = {n: torch.empty(d[n].numel() + 3, dtype=torch.bfloat16, device="cuda")[3:].view(d[n].shape).copy_(d[n]) for n in "qkv"}
    u = torch.full((d["v"].numel() + 9,), 7.0, dtype=torch.bfloat16, device="cuda")
    if Dk % 8:
        d["q"], d["k"] = off["q"], off["k"]
    if Dv % 8:
        d["v"] = off["v"]
        o = u[5:-4].view(d["v"].shape)
    else:
        o = given
    w = call(out=o)
    for b, n in enumerate(lengths or [S] * B):
        assert torch.equal(o[b, :, :n], y[0][b, :, :n])
    assert torch.equal(w[1], y[1]) and bool((u[:5] == 7.0).all()) and bool((u[-4:] == 7.0).all())
    assert gdn.device_status(0) == 0


def test_what_is_padded():
    need = lambda *s, **kw: gdn.linear_attn_workspace_bytes(*s, single_pass=True, **kw)  # noqa: E731
    assert need(4, 2, 4, 500, 77, 75) > 0 and need(4, 2, 4, 500, 80, 72) == 0
    assert need(4, 2, 4, 500, 77, 75, gdn.GDN_F32) == 0 and need(4, 2, 4, 500, 77, 75, force_ffma=True) == 0
    assert need(1, 1, 1, 500, 77, 75) == 0                                      # small
    assert need(64, 16, 32, 20, 30, 30) == 0 and need(64, 16, 32, 40, 30, 30) > 0   # heads of a few tokens


def test_padded_heads_handed_on_and_graph():
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    Hv, S, Dk, Dv = sms + 8, 1100, 77, 75
    x = inputs(1, 1, Hv, S, Dk, Dv, "bf16", "token", False)
    d = {n: t.cuda() for n, t in x.items() if t is not None}
    call = lambda **kw: gdn.linear_attn_prefill(d["q"], d["k"], d["v"], d["g"], 0.1, **kw)  # noqa: E731
    want = call(single_pass=True)
    y = call()
    assert torch.equal(y[0], want[0]) and torch.equal(y[1], want[1])
    last = slice(Hv - 1, Hv)
    out, st, size = ref.recurrence(x["q"], x["k"], x["v"][:, last], x["g"][:, last], 0.1)
    compare((y[0][:, last], y[1][:, last]), (out, st), size, "bf16", True, "padded, handed on")
    o, s = torch.empty_like(d["v"]), torch.empty_like(want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdn.linear_attn_prefill(d["q"], d["k"], d["v"], d["g"], 0.1, None, o, state_out=s)
    for _ in range(2):
        o.zero_()
        s.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want[0]) and torch.equal(s, want[1])
