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
