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


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("B,T,S,n,H,Hkv,D", [
    (1, 1, 9000, 8000, 2, 1, 128), (2, 3, 4000, 3500, 8, 1, 64), (1, 2, 30000, 29000, 32, 1, 128),  # split
    (300, 1, 64, 40, 2, 1, 128), (1, 2, 100, 50, 4, 2, 64), (3, 4, 128, 70, 20, 2, 80)])            # whole
def test_nan_in_decode(B, T, S, n, H, Hkv, D, dtype):
    q, k, v = (randn(i, B, T, h, D, dtype=dtype) for i, h in enumerate((H, Hkv, Hkv)))
    kc, vc = (randn(i, B, S, Hkv, D, dtype=dtype) for i in (3, 4))
    lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
    clean = gdn.attn_decode(q, k, v, kc.clone(), vc.clone(), lens)
    for what, at in (("q", T - 1), ("q", slice(None)), ("cache", 0), ("cache", n - 1), ("cache", slice(n)), ("k", T - 1)):
        x = {"q": q.clone(), "cache": kc.clone(), "k": k.clone()}
        x[what][:, at] = NAN
        rows = torch.ones(T, dtype=torch.bool, device="cuda")
        if what in ("q", "k"):
            rows[:] = False
            rows[at] = True
        same_but(rows, gdn.attn_decode(x["q"], x["k"], v, x["cache"], vc.clone(), lens), clean)
    assert gdn.device_status() == 0
