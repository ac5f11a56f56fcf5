"""attn_paged: what is no number in a new token's key or value reaches the rows that
see the token, and no others, whichever kernel takes the call."""
import numpy as np
import pytest
import torch

import gated_delta_rule_bwd_gb300 as gdn
from tests.test_attn_paged import FORMATS, random_cache
from tests.test_kv_cache import i32, places, tables


@pytest.mark.gpu
@FORMATS
@pytest.mark.parametrize("D", [64, 96, 128])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("T,H,Hkv", [(3, 4, 2), (2, 16, 1), (5, 4, 1), (40, 2, 1)])
@pytest.mark.parametrize("page", [16, 64])
def test_new_tokens(page, T, H, Hkv, bad, D, dtype, bits):
    """Two tokens of row 0, in its first key head: the results of the tokens before
    them, of other heads and rows keep every bit; in v the others' 32 values (one value,
    if not in 4 bits) of the head and no more are no numbers."""
    lens = [150, 90, 0]
    held = [n + T for n in lens]
    table, pages = tables(held, page, T)
    cache = random_cache(pages, page, Hkv, D, dtype, bits, T)
    q = torch.randn(len(lens), T, H, D, generator=torch.Generator().manual_seed(T)).to(dtype).cuda()
    before = gdn.attn_paged(q, cache, table, i32(lens))
    G, first = H // Hkv, T // 2
    at = [tuple(int(x[0]) for x in places(np.array([0]), np.array([lens[0] + i]), table, page)) for i in {first, T - 1}]
    k, v = (cache[2], cache[3]) if bits else (cache[0], cache[1])
    for x in (v, k):
        changed = [x[p].clone() for p in at]
        for p in at:
            x[p][0, 1] = bad
        after = gdn.attn_paged(q, cache, table, i32(lens))
        assert gdn.device_status() == 0
        hit = torch.zeros_like(before, dtype=torch.bool)
        if x is v:
            hit[0, first:, :G, slice(32, 64) if bits else 1] = True
            assert not after[hit].isfinite().any()
        else:
            hit[0, first:, :G] = True
            if np.isnan(bad):
                assert after[hit].isnan().all()
        assert torch.equal(after[~hit], before[~hit])
        for p, y in zip(at, changed):
            x[p] = y
