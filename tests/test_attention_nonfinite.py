"""A NaN reaches the rows that it belongs to, whether or not the keys of a call are
split and joined: a query row that holds one, and every row that sees a key that
holds one, are NaN as a whole; all other rows keep their bits.
"""
import ctypes

import pytest
import torch

import gated_delta_rule_bwd_gb300 as gdn

gpu = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
NAN = float("nan")


def randn(seed, *shape, dtype):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def same_but(rows, got, clean):
    """[B, T, ...]: the marked rows [T] are NaN, the others equal `clean`."""
    assert got[:, rows].isnan().all()
    assert torch.equal(got[:, ~rows], clean[:, ~rows])


@gpu
@pytest.mark.parametrize("B,Tq,Tk,H,Hkv,D,dtype,split", [
    (1, 1, 4100, 2, 1, 128, BF16, True), (1, 1400, 1400, 1, 1, 128, BF16, True),
    (1, 300, 2500, 4, 1, 96, BF16, True), (1, 70, 2050, 3, 3, 64, BF16, True), (1, 1500, 700, 1, 1, 64, BF16, True),
    (1, 900, 300, 1, 1, 64, BF16, False), (2, 300, 300, 4, 2, 128, BF16, False), (1, 130, 131, 2, 1, 64, BF16, False),
    (2, 200, 460, 4, 2, 64, F32, False), (1, 5, 700, 2, 1, 72, F32, False), (6, 200, 200, 16, 16, 64, F32, False)])
def test_nan_in_a_prompt(B, Tq, Tk, H, Hkv, D, dtype, split):
    q, k, v = (randn(i, B, t, h, D, dtype=dtype) for i, (t, h) in enumerate(((Tq, H), (Tk, Hkv), (Tk, Hkv))))
    if dtype is BF16:
        s, *_, nseq = gdn._attn_args(q, k, v, None, None, None)
        assert (gdn.lib().gdn_attn_fwd_workspace(ctypes.byref(s), nseq) > 0) == split
    clean, clean_lse = gdn.attn_fwd(q, k, v)
    last = torch.arange(Tq, device="cuda") + Tk - Tq  # a row's last key
    for what, at in (("q", Tq // 2), ("q", slice(None)), ("k", 0), ("k", Tk // 2), ("k", slice(None))):
        x = {"q": q.clone(), "k": k.clone()}
        x[what][:, at] = NAN
        if what == "q":
            rows = torch.zeros(Tq, dtype=torch.bool, device="cuda")
            rows[at] = True
            rows &= last >= 0
        else:
            rows = last >= (at if isinstance(at, int) else 0)
        o, lse = gdn.attn_fwd(x["q"], x["k"], v)
        same_but(rows, o, clean)
        same_but(rows, lse.transpose(1, 2), clean_lse.transpose(1, 2))
    assert gdn.device_status() == 0
