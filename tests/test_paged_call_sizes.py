"""Calls of norm and rotation, pages and attention over them whose sizes pass the
library's 32-bit integers: refused with the library's error, none goes on with the
size's lower bits."""
import pytest
import torch

import gated_delta_rule_bwd_gb300 as gdn

BF16, I32 = torch.bfloat16, torch.int32
BIG = 1 << 31


def test_caches_of_too_many_pages():
    cpu = torch.device("cpu")
    for dtype, extra in ((BF16, 0), (torch.uint8, 2)):
        x = torch.zeros(1, 16, 1, 32, dtype=dtype).expand(BIG, -1, -1, -1)
        steps = torch.zeros(1, 16, 1, 2, dtype=BF16).expand(BIG, -1, -1, -1)
        with pytest.raises(gdn.GdnError, match="integers"):
            gdn._cache_args((x, x, *[steps] * extra), cpu)


@pytest.mark.gpu
def test_too_many_tokens():
    z = lambda *s, dt=BF16: torch.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
    one, n, table = z(1, 1, 1, 8), z(1, dt=I32), z(1, 4, dt=I32)
    many = one.expand(1, BIG, 1, 8)
    cos = z(4, 4, dt=torch.float32)
    cache, codes = gdn.new_paged_cache(4, 16, 1, 8), gdn.new_paged_cache(4, 16, 1, 32, bits=4)
    pages = [x.expand(BIG, -1, -1, -1) for x in (z(1, 16, 1, 8), z(1, 16, 1, 8))]
    steps = [x[:1].expand(BIG, -1, -1, -1) for x in codes]
    four = z(1, 1, 1, 32)
    off = torch.tensor([0, 2], dtype=I32, device="cuda")
    for call in (lambda: gdn.qk_norm_rope_fwd(many, many, cos=cos, sin=cos), lambda: gdn.qk_norm_rope_bwd(many, many, one, one, cos=cos, sin=cos),
                 lambda: gdn.kv_append(many, many, cache, table, n), lambda: gdn.kv_append(one, one, pages, table, n),
                 lambda: gdn.kv_append(many, many, cache, table, n, cu_seqlens=off), lambda: gdn.kv_append(four, four, steps, table, n),
                 lambda: gdn.attn_paged(one, pages, table, n), lambda: gdn.attn_paged(four, steps, table, n),
                 lambda: gdn.attn_paged(torch.empty(1, BIG, 1, 1, dtype=BF16, device="cuda"), gdn.new_paged_cache(4, 16, 1, 1), table, n),
                 lambda: gdn.attn_paged(one, cache, torch.empty(1, BIG, dtype=I32, device="cuda"), n), lambda: gdn.kv_gather(pages, table, off, 2)):
        with pytest.raises(gdn.GdnError):
            call()
    assert gdn.device_status() == 0


@pytest.mark.gpu
def test_gathers_of_too_many_tokens():
    """Nothing is made for them."""
    table, off = torch.zeros(1, 4, dtype=I32, device="cuda"), torch.tensor([0, 2], dtype=I32, device="cuda")
    small = gdn.new_paged_cache(4, 16, 1, 1)
    for total in (-1, (1 << 30) + 1, BIG, 1 << 32, (1 << 32) + 2):
        held = torch.cuda.memory_allocated()
        torch.cuda.reset_peak_memory_stats()
        with pytest.raises(gdn.GdnError):
            gdn.kv_gather(small, table, off, total)
        assert torch.cuda.max_memory_allocated() == held  # nothing is made for it
    k, v = gdn.kv_gather(small, table, off, 2)
    assert k.shape == (1, 2, 1, 1) and gdn.device_status() == 0
