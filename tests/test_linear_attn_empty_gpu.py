"""linear_attn_prefill over batches of which most sequences are empty: slots of a server, of which few have a prompt."""
import pytest
import torch

import gated_delta_rule_20_gb300 as gdn

pytestmark = pytest.mark.gpu


def batch(Hv, sms, handed):
    """Which sequences of Hv heads have tokens: every CTA (it takes every sms-th head) meets some, then 100 or more heads
    without a token, some again, 100 or more without, and some at the end.  ``handed``: so many in all that the heads
    left over by whole rounds of the SMs run in parts."""
    some, none = -(-sms // Hv) + 1, -(-100 * sms // Hv)
    live = [True] * some + [False] * none + [True] * some + [False] * none + [True] * some
    while (0 < len(live) * Hv % sms <= sms // 4) != handed or (not handed and len(live) * Hv % sms <= sms // 2):
        live.insert(some, False)
    return live


@pytest.mark.parametrize("S, Hk, Hv, Dk, Dv, handed, ends", [
    (300, 1, 16, 16, 8, False, [300, 257, 1]), (300, 2, 4, 8, 72, False, [300, 128]), (1030, 1, 16, 8, 8, True, [1030, 1030, 300, 700]),
    (1100, 2, 8, 64, 16, True, [1100, 1099])])
@pytest.mark.parametrize("given", [False, True])
def test_long_runs_of_empty_sequences(S, Hk, Hv, Dk, Dv, handed, ends, given):
    """The sequences with tokens have the bits that each has by itself, the empty ones the state that they had; rows behind the
    lengths are zeros in a new out and untouched in one that is given."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    live = batch(Hv, sms, handed)
    B = len(live)
    lengths = [0] * B
    for i, b in enumerate(b for b in range(B) if live[b]):
        lengths[b] = ends[i % len(ends)]
    assert gdn.linear_attn_segments(B, Hk, Hv, S, Dk, Dv) == 1
    assert (gdn.linear_attn_workspace_bytes(B, Hk, Hv, S, Dk, Dv) > 0) == handed
    gen = torch.Generator(device="cuda").manual_seed(S + Dv)
    n = lambda *s: torch.randn(*s, generator=gen, device="cuda").bfloat16()  # noqa: E731
    q, k, v = n(B, Hk, S, Dk), n(B, Hk, S, Dk), n(B, Hv, S, Dv)
    g = -0.3 * torch.rand(B, Hv, S, generator=gen, device="cuda")
    state = torch.randn(B, Hv, Dk, Dv, generator=gen, device="cuda")
    at = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    empty = at == 0
    for x in (q, k, v):
        x[empty] = float("nan")
    for _ in range(3):
        new = torch.full_like(state, float("nan"))
        out = torch.full_like(v, 7.0) if given else None
        out, st = gdn.linear_attn_prefill(q, k, v, g, 0.1, state, out, lengths=at, state_out=new)
        torch.cuda.synchronize()
        assert gdn.device_status(0, clear=True) == 0
        assert torch.equal(st[empty], state[empty])
        rest = 7.0 if given else 0.0
        assert bool((out[empty] == rest).all())
        for b in range(B):
            m = lengths[b]
            if m:
                assert bool((out[b, :, m:] == rest).all())
                one = gdn.linear_attn_prefill(*(x[b:b + 1, :, :m].contiguous() for x in (q, k, v, g)), 0.1, state[b:b + 1],
                                              state_out=torch.empty_like(state[b:b + 1]), single_pass=True)
                assert torch.equal(out[b, :, :m], one[0][0]) and torch.equal(st[b], one[1][0]), "sequence %d" % b


@pytest.mark.parametrize("heads", [1 << 24, 1 << 28])
def test_more_heads_than_waits_are_long(heads):
    """So many heads, of which the first sequence's and the last's have a token, that a walk over a CTA's share would outlast the
    waits behind it: the call ends well, in its time, with the others' states and outputs untouched."""
    Hv, D = 128, 8
    B = heads // Hv
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("needs 100 GB of free device memory")
    gen = torch.Generator(device="cuda").manual_seed(7)
    q, k = (torch.zeros(B, 1, 1, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    v = torch.zeros(B, Hv, 1, D, dtype=torch.bfloat16, device="cuda")
    out = torch.full_like(v, 7.0)
    ends = (0, B - 1)
    for x in (q, k, v):
        for b in ends:
            x[b] = torch.randint(-8, 9, x[b].shape, generator=gen, device="cuda").to(x.dtype)
    g = torch.full((Hv,), -0.5, device="cuda")
    state = torch.zeros(B, Hv, D, D, device="cuda")
    at = torch.zeros(B, dtype=torch.int32, device="cuda")
    at[0] = at[-1] = 1
    gdn.linear_attn_prefill(q, k, v, g, 1.0, state, out, lengths=at)
    torch.cuda.synchronize()
    assert gdn.device_status(0, clear=True) == 0
    for b in ends:
        kv = k[b].float().transpose(-1, -2) * v[b].float()
        # (the FMA units take v by e^0.5 and the state by e^-0.5 in the end: two exponentials, each off by 2 steps, 4 U with U =
        # 2^-24, and three products of U each: 11 U)
        assert bool(((state[b] - kv).abs() <= 11 * 2.0 ** -24 * kv.abs()).all())
        # o = (q . k) v, one term: on the tensor cores the score is rounded to bf16 (up to 8 * 64, 10 bits), by half a step of
        # 2^-8 of it at most, then the output, so that the two are off by (1 + 2^-8)^2 - 1 < 2^-7 + 2^-15 of it
        want = q[b].double() @ kv.double()
        assert bool(((out[b].double() - want).abs() <= (2.0 ** -7 + 2.0 ** -15) * want.abs()).all())
        state[b], out[b] = 0, 7.0
    for part in range(64):  # (a part at a time: comparisons take memory too)
        rows = slice(part * (B // 64), (part + 1) * (B // 64))
        assert bool((state[rows] == 0).all()) and bool((out[rows] == 7.0).all())
