"""4-bit pages where they are used, against plain attention over what kv_gather reads
back from the same pages, so that only the attention differs."""
import numpy as np
import pytest
import torch

import gated_delta_rule_bwd_gb300 as gdn
from oracle import attention as at
from tests.test_examples import load
from tests.test_kv_cache import cu, i32, np64, tables

BF16, F32 = torch.bfloat16, torch.float32


def plain(q, cache, table, lens, rows=None):
    """attn_paged in fp32 torch operations; ``rows``: whose pages each row reads."""
    B, T, H, D = q.shape
    held = (lens + T).tolist()
    k, v = gdn.kv_gather(cache, table if rows is None else table[rows].contiguous(), cu(held), sum(held), dtype=F32)
    o, begin = torch.empty(q.shape, device=q.device), 0
    for b, n in enumerate(held):
        kb, vb = (x[0, begin:begin + n].repeat_interleave(H // x.shape[2], 1) for x in (k, v))
        s = torch.einsum("thd,nhd->htn", q[b].float(), kb) * D ** -0.5
        see = torch.arange(n, device=q.device) <= (n - T + torch.arange(T, device=q.device))[:, None]
        o[b] = torch.einsum("htn,nhd->thd", torch.softmax(s.masked_fill(~see, -torch.inf), -1), vb)
        begin += n
    return o.to(q.dtype)


@pytest.mark.gpu
def test_the_example(monkeypatch):
    """The logits of a text on 4-bit pages are those with plain attention over the same pages,
    within the bf16 roundings along the path (about 16 stored activations, half a step of
    2^-8 each); with each row's pages taken for another's they are not."""
    ex = load("hybrid_layers")
    model = ex.Hybrid()
    ex.train(model, 30)
    gen = torch.Generator().manual_seed(2)
    text = torch.randint(ex.VOCAB, (4, 72), generator=gen).cuda()
    _, memory = model.prompt(text[:, :48], 72)
    runs = {}
    for name, attend in (("kernel", gdn.attn_paged), ("plain", plain),
                         ("other rows", lambda *a: plain(*a, rows=torch.tensor([1, 2, 3, 0], device="cuda")))):
        pages = model.to_pages(memory, bits=4)
        with monkeypatch.context() as m:
            m.setattr(gdn, "attn_paged", attend)
            runs[name] = ex.follow(model, text[:, 48:], pages)
    assert gdn.device_status() == 0
    bound = 16 * 2 ** -8 * runs["plain"].abs().max()
    assert (runs["kernel"] - runs["plain"]).abs().max() <= bound
    assert (runs["other rows"] - runs["plain"]).abs().max() > bound


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_serving(dtype):
    """Prompts, packed and rotated on the way in, then one token per row.  Bounds as for
    attn_paged alone: with bf16 queries 2^-16 + 2e-5 of a = sum p |v| and half a step; 4-bit
    scores are off by the sum of some 32 roundings to fp16 (2^-11 of each second
    weight's part; 6 standard deviations), which moves the result by twice that of a."""
    lens, H, Hkv, D, page = [37, 1, 64, 500], 8, 2, 64, 16
    held = [n + 1 for n in lens]
    table, pages = tables(held, page, 3)
    cache = gdn.new_paged_cache(pages, page, Hkv, D, dtype, 4)
    cos, sin = gdn.rope_table(max(held), D)
    g = torch.Generator().manual_seed(4)
    q, k, v = torch.randn(1, sum(lens), H + 2 * Hkv, D, generator=g).to(dtype).cuda().split([H, Hkv, Hkv], dim=2)
    gdn.kv_append(k, v, cache, table, i32([0] * 4), q, cos, sin, cu_seqlens=cu(lens))
    q, k, v = torch.randn(4, 1, H + 2 * Hkv, D, generator=g).to(dtype).cuda().split([H, Hkv, Hkv], dim=2)
    rq = gdn.kv_append(k, v, cache, table, i32(lens), q, cos, sin)
    o = np64(gdn.attn_paged(rq, cache, table, i32(lens)))
    gk, gv = (np64(x)[0] for x in gdn.kv_gather(cache, table, cu(held), sum(held), dtype=F32))
    assert gdn.device_status() == 0
    e, terms = (2.0 ** -8, 2.0 ** -16) if dtype == BF16 else (0.0, 0.0)
    begin = 0
    for b, n in enumerate(held):
        for h in range(H):
            x, kb, vb = np64(rq)[b, :, h], gk[begin:begin + n, h // 4], gv[begin:begin + n, h // 4]
            ref, _, a = at.attn_fwd(x, kb, vb, D ** -0.5)
            off = 0.0
            if dtype == BF16:
                w = x[0, 0::2] - x[0, 1::2] / 16
                off = 2 * 6 * D ** -0.5 * np.sqrt(np.sum((2.0 ** -11 * w * kb[:, 0::2]) ** 2, -1) / 3).max()
            bound = (terms + 2e-5 + off) * a + e * np.abs(ref) + 2e-5 * np.sqrt(np.mean(ref * ref))
            assert np.all(np.abs(o[b, :, h] - ref) <= bound), (b, h, np.max(np.abs(o[b, :, h] - ref) / bound))
        begin += n
