"""The give-up path of linear attention's tensor-core prefill, exercised without a GPU fault.

As in the gated delta rule's test: gdn_test_stall_prefill makes the role that hands out the decays wait on a barrier that
nothing arrives at.  That wait and the other roles' behind it run out after the kernel's own bound, some two seconds;
the call returns, the status word reads GDN_ERR_TIMEOUT, and the next call in the same process has the bits that it had
before: no tensor memory stayed allocated and nothing waits."""
import pytest
import torch

import gated_delta_rule_20_gb300 as gdn
from gated_delta_rule_20_gb300 import _binding as B

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads, S, Dk, Dv, single_pass, lengths", [
    (3, 60, 128, 128, True, None), (2, 1000, 128, 128, False, None),  # a chunk; in segments
    (-8, 1100, 64, 64, False, 900),                                   # heads handed on, zeroed padding
    (6, 1500, 77, 75, True, None)])                                   # padded rows
def test_linear_attn_wait_timeout_reports_and_recovers(heads, S, Dk, Dv, single_pass, lengths):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    Hv = heads if heads > 0 else sms - heads
    gen = torch.Generator(device="cuda").manual_seed(S)
    n = lambda *s: torch.randn(*s, generator=gen, device="cuda").bfloat16()  # noqa: E731
    q, k, v = n(1, 1, S, Dk), n(1, 1, S, Dk), n(1, Hv, S, Dv)
    g = -0.1 * torch.rand(1, Hv, S, generator=gen, device="cuda")
    state = torch.randn(1, Hv, Dk, Dv, generator=gen, device="cuda")
    at = None if lengths is None else torch.tensor([lengths], dtype=torch.int32, device="cuda")

    def call():
        y = gdn.linear_attn_prefill(q, k, v, g, 0.1, state, lengths=at, state_out=torch.full_like(state, float("nan")),
                                    single_pass=single_pass)
        torch.cuda.synchronize()
        return y
    gdn.device_status(0, clear=True)
    want = call()
    assert gdn.device_status(0) == 0
    try:
        B.test_stall_prefill(0, True)
        call()  # returns: no wait is left spinning
        code = gdn.device_status(0, clear=True)
    finally:
        B.test_stall_prefill(0, False)
    assert code == gdn.GDN_ERR_TIMEOUT
    for _ in range(2):
        y = call()
        assert torch.equal(y[0], want[0]) and torch.equal(y[1], want[1])
    assert gdn.device_status(0, clear=True) == 0
