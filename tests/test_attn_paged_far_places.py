"""attn_paged on a page so long that a token's place times the 16-byte vectors of
its row passes 32 bits."""
import ctypes

import pytest
import torch

import gated_delta_rule_bwd_gb300 as gdn


@pytest.mark.gpu
def test_places_past_2_28():
    """One bf16 head of 128 has 16 vectors a token: place 2^28 + n and place n differ in
    the product's 33rd bit only.  Keys and values are the same memory, zeros but for two
    tokens: the far one's score is |r|^2 scale = 724 above every other's, so that the
    result is its value exactly; the near one, opposite to the query, has no weight."""
    D, page, near = 128, 1 << 29, 37
    far = (1 << 28) + near
    tokens = far + 64
    if torch.cuda.mem_get_info()[0] < 2 * tokens * D + (4 << 30):
        pytest.skip("needs 70 GB of device memory")
    kv = torch.zeros(tokens, D, dtype=torch.bfloat16, device="cuda")
    kv[far], kv[near] = 8, -8
    q = torch.full((1, 1, 1, D), 8, dtype=torch.bfloat16, device="cuda")
    o = torch.empty_like(q)
    table, lens = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([[0]], [tokens - 1]))
    st = (0, D, D)
    c = gdn.PagedCacheDesc(1, page, 1, D, 1, kv.data_ptr(), kv.data_ptr(), None, None, st, st, (0, 0, 0), (0, 0, 0))
    s = gdn.AttnPagedShape(1, 1, 1, 1, 1, 1)
    L = gdn.lib()
    need = L.gdn_attn_paged_workspace(ctypes.byref(s), ctypes.byref(c))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    rc = L.gdn_attn_paged(ctypes.byref(s), ctypes.byref(c), q.data_ptr(), table.data_ptr(), lens.data_ptr(), D ** -0.5, o.data_ptr(),
                          ws.data_ptr(), need, torch.cuda.current_stream().cuda_stream)
    assert rc == 0 and gdn.device_status() == 0
    assert torch.equal(o, q)
