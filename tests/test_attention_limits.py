"""attn_fwd / attn_bwd at the ends of their sizes."""
import ctypes

import pytest
import torch

import gated_delta_rule_bwd_gb300 as gdn

gpu = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("Tq", [0, 5])
def test_key_heads_without_query_heads(Tq, dtype):
    """No query reads the keys: their gradients are zeros, not what lay there."""
    L, n = gdn.lib(), (2, 7, 3, 16)
    q, k = torch.empty(2, Tq, 0, 16, dtype=dtype, device="cuda"), torch.ones(*n, dtype=dtype, device="cuda")
    dk, dv = torch.ones_like(k), torch.ones_like(k)
    s, scale, *_ = gdn._attn_args(q, k, k, None, None, None)
    rc = L.gdn_attn_bwd(ctypes.byref(s), None, k.data_ptr(), k.data_ptr(), scale, None, None, 0, None, None, None, None,
                        dk.data_ptr(), dv.data_ptr(), None, 0, torch.cuda.current_stream().cuda_stream)
    assert rc == 0 and not dk.any() and not dv.any()
    o, lse = gdn.attn_fwd(q, k, k)
    assert o.shape == q.shape and all(not x.any() for x in gdn.attn_bwd(q, k, k, o, lse, o)[1:])


def test_key_heads_without_query_heads_refusals():
    fake, odd = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10008)
    s = gdn.AttnShape(1, 4, 4, 0, 2, 16, 1, (0, 0, 0), (128, 32, 16), (128, 32, 16))
    call = lambda dk, dv: gdn.lib().gdn_attn_bwd(  # noqa: E731
        ctypes.byref(s), None, fake, fake, 0.5, None, None, 0, None, None, None, None, dk, dv, None, 0, None)
    assert call(None, fake) == -1 and call(fake, None) == -1 and call(odd, fake) == -4 and call(fake, odd) == -4


def call(name, packed=False, nseq=0, **sizes):
    """An entry point on made-up pointers: for calls that are refused before a launch."""
    fake = ctypes.c_void_p(0x10000)
    n = dict(B=1, Tq=8, Tk=8, H=16, Hkv=16, D=8) | sizes
    s = gdn.AttnShape(*n.values(), 1, (0, 0, 0), (0, 0, 0), (0, 0, 0))
    cu = fake if packed else None
    f = getattr(gdn.lib(), name)
    if name == "gdn_attn_fwd":
        return f(ctypes.byref(s), fake, fake, fake, 0.5, cu, cu, nseq, fake, fake, fake, 1 << 62, None)
    return f(ctypes.byref(s), fake, fake, fake, 0.5, cu, cu, nseq, *[fake] * 7, 1 << 62, None)


@pytest.mark.parametrize("name", ["gdn_attn_fwd", "gdn_attn_bwd"])
@pytest.mark.parametrize("sizes", [dict(packed=True, nseq=1 << 30, H=16), dict(packed=True, nseq=1 << 27, H=16, Hkv=1),
                                   dict(B=1 << 24, Tq=1, Tk=1, H=128), dict(B=1 << 24, Tq=0, Tk=1, H=128),
                                   dict(Tq=1 << 30, H=17, Hkv=1), dict(Tq=1, Tk=1 << 30, H=128, Hkv=1)])
def test_more_jobs_than_a_grid_has(name, sizes):
    assert call(name, **sizes) == -2


def test_sizes_below_the_limits_have_a_workspace():
    for n in (dict(B=1 << 24, Tq=1, Tk=1, H=127), dict(Tq=1 << 30, H=15, Hkv=1), dict(Tq=8, Tk=1 << 30, H=64, Hkv=1)):
        n = dict(B=1, Tq=8, Tk=8, H=16, Hkv=n["H"], D=8) | n
        s = gdn.AttnShape(*n.values(), 1, (0, 0, 0), (0, 0, 0), (0, 0, 0))
        assert gdn.lib().gdn_attn_bwd_workspace(ctypes.byref(s), 0) == 4 * n["B"] * n["H"] * n["Tq"], n


@pytest.mark.parametrize("B,Tq,Tk,H,D", [(1, 64, 4096, 2, 128), (2, 64, 4096, 2, 128), (1, 1400, 1400, 1, 64)])
def test_workspace_of_a_batch_whatever_nseq(B, Tq, Tk, H, D):
    """A batch call ignores nseq; so does what its workspace query returns at least."""
    s = gdn.AttnShape(B, Tq, Tk, H, 1, D, 1, *[(1 << 20, 1 << 10, 128)] * 3)
    need = lambda nseq: gdn.lib().gdn_attn_fwd_workspace(ctypes.byref(s), nseq)  # noqa: E731
    assert need(0) > 0
    for nseq in (-3, 1, 7, 100000, 1 << 30):
        assert need(nseq) >= need(0), nseq
    if B > 1:
        assert need(7) == need(0)


def test_decode_of_key_heads_without_query_heads_is_refused():
    """It would have to extend the caches, and wrote nothing."""
    fake = ctypes.c_void_p(0x10000)
    s = lambda Hkv: gdn.AttnDecodeShape(1, 1, 8, 0, Hkv, 16, 1, (256, 32, 16), (256, 32, 16))  # noqa: E731
    call = lambda Hkv: gdn.lib().gdn_attn_decode(  # noqa: E731
        ctypes.byref(s(Hkv)), *[fake] * 6, 0.5, fake, None, 0, None)
    assert call(2) == -2 and call(0) == 0


@gpu
def test_heads_without_values_are_refused():
    x, lens = torch.zeros(1, 4, 2, 0, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    with pytest.raises(gdn.GdnError, match="D = 0"):
        gdn.attn_fwd(x, x, x)
    with pytest.raises(gdn.GdnError, match="D = 0"):
        gdn.attn_decode(x, x, x, x, x, lens)
