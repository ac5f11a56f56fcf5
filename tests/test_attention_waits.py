"""The attention kernels' bounded waits: no limit on a wait while the CTA moves on,
an end to it once nothing does.
"""
import pytest
import torch

import gated_delta_rule_bwd_gb300 as gdn


def test_selftest_validates_its_argument():
    for clocks in (0, -1, (1 << 26) + 1):
        assert gdn.lib().gdn_attn_wait_selftest(clocks, None) == -1


@pytest.mark.gpu
def test_wait_lasts_while_there_is_progress_and_ends_without():
    """The status is the timeout's only if the slow arrival was waited for and the
    missing one given up; the context goes on."""
    assert gdn.device_status() == 0
    gdn.attn_wait_selftest()
    torch.cuda.synchronize()
    assert gdn.device_status() == -7 and gdn.device_status() == 0
    q, k, v = (torch.randn(1, 300, 2, 64, dtype=torch.bfloat16, device="cuda") for _ in range(3))
    o, lse = gdn.attn_fwd(q, k, v)
    assert o.isfinite().all() and lse.isfinite().all() and gdn.device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("heads", [1, 3])
def test_many_empty_sequences(heads):
    """Long runs of empty sequences between two that are not: the scheduler passes
    over them one by one while the other warps wait."""
    n, T, D = 200001, 200, 64
    q, k, v, do = (torch.randn(1, T, heads, D, dtype=torch.bfloat16, device="cuda") for _ in range(4))
    cu = torch.zeros(n + 1, dtype=torch.int32, device="cuda")
    cu[n // 2:], cu[-1] = 77, T
    few = torch.tensor([0, 77, T], dtype=torch.int32, device="cuda")
    o, lse = gdn.attn_fwd(q, k, v, cu)
    want, want_lse = gdn.attn_fwd(q, k, v, few)
    assert torch.equal(o, want) and torch.equal(lse, want_lse)
    for a, b in zip(gdn.attn_bwd(q, k, v, o, lse, do, cu), gdn.attn_bwd(q, k, v, o, lse, do, few)):
        assert torch.equal(a, b)
    assert gdn.device_status() == 0
