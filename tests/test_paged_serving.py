"""An attention layer's calls as a program runs them: norm and rotation, prompt
attention, pages, and token by token, against attention over the whole text.

The whole text's attention sees the same bf16 queries and keys (rotation and norm
go row by row), so the bounds are attn_fwd's and attn_paged's own: bf16 weights
off by e = 2^-8 of themselves and a result rounded once, e (a + |o|) with a = sum
p |v|, and fp32 terms of 2e-5.  In 4 bits the oracle attends over the values that
kv_gather reads back, which are what the pages stand for.
"""
import numpy as np
import pytest
import torch

import gated_delta_rule_bwd_gb300 as gdn
from oracle import attention as at
from tests.test_kv_cache import cu, i32, np64, tables

gpu = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
E, F = 2.0 ** -8, 2e-5
H, HKV, D, PAGE = 8, 2, 64, 16


def layer(seed, B, T, dtype):
    """A layer's projections of tokens [B, T], q and k normed and rotated in place of
    their positions 0 ..; all as one call."""
    g = torch.Generator().manual_seed(seed)
    qkv = torch.randn(B, T, H + 2 * HKV, D, generator=g).to(dtype).cuda()
    w = [(1 + 0.2 * torch.randn(D, generator=g)).cuda() for _ in range(2)]
    return qkv, w


def bounds(q, k, v, dtype):
    """Oracle o and its bound for one row: q [n, H, D], k, v [m, HKV, D], causal."""
    o, b = np.zeros(q.shape), np.zeros(q.shape)
    e = E if dtype == BF16 else 0.0
    for h in range(q.shape[1]):
        j = h // (H // HKV)
        o[:, h], _, a = at.attn_fwd(q[:, h], k[:, j], v[:, j], D ** -0.5)
        b[:, h] = (e + F) * a
    return o, b + e * np.abs(o) + F * np.sqrt(np.mean(o * o))


@gpu
@pytest.mark.parametrize("dtype,bits", [(BF16, None), (F32, None), (BF16, 4), (F32, 4)], ids=["bf16", "f32", "bf16-4", "f32-4"])
@pytest.mark.parametrize("fused", [False, True], ids=["norm", "rotated on the way"])
def test_prompt_then_token_by_token(fused, dtype, bits):
    """Prompts of three lengths, packed, into pages; then single tokens, in one
    captured step that is replayed.  ``fused``: no norm, the rotation by kv_append."""
    lens, new = [37, 1, 64], 12
    held = [n + new for n in lens]
    table, pages = tables(held, PAGE)
    cos, sin = gdn.rope_table(max(held), D)
    cache = gdn.new_paged_cache(pages, PAGE, HKV, D, dtype, bits)
    qkv, w = layer(0, 3, max(held), dtype)  # row b's tokens: the first held[b]
    pos = torch.arange(max(held), device="cuda", dtype=torch.int32).expand(3, -1).contiguous()
    q, k, v = qkv.split([H, HKV, HKV], dim=2)
    norm = (None, None) if fused else tuple(w)
    rq, rk = gdn.qk_norm_rope_fwd(q, k, *norm, cos, sin, pos)

    # the prompts, packed
    pick = lambda x: torch.cat([x[b, :n] for b, n in enumerate(lens)])[None]  # noqa: E731
    at0 = torch.cat([pos[b, :n] for b, n in enumerate(lens)])[None]
    pq, pk = gdn.qk_norm_rope_fwd(pick(q), pick(k), *norm, cos, sin, at0)
    assert torch.equal(pq, pick(rq)) and torch.equal(pk, pick(rk))
    o, _ = gdn.attn_fwd(pq, pk, pick(v), cu_seqlens=cu(lens))
    zero = i32([0, 0, 0])
    if fused:
        same = gdn.kv_append(pick(k), pick(v), cache, table, zero, pick(q), cos, sin, cu_seqlens=cu(lens))
        assert torch.equal(same, pq)
    else:
        gdn.kv_append(pk, pick(v), cache, table, zero, cu_seqlens=cu(lens))

    # token by token, a captured step
    n = i32(lens)
    tok = torch.zeros(3, 1, H + 2 * HKV, D, dtype=dtype, device="cuda")
    out = torch.zeros(3, 1, H, D, dtype=dtype, device="cuda")

    def step():
        sq, sk, sv = tok.split([H, HKV, HKV], dim=2)
        if fused:
            sq = gdn.kv_append(sk, sv, cache, table, n, sq, cos, sin)
        else:
            sq, sk = gdn.qk_norm_rope_fwd(sq, sk, *norm, cos, sin, n[:, None])
            gdn.kv_append(sk, sv, cache, table, n)
        out.copy_(gdn.attn_paged(sq, cache, table, n))
        n.add_(1)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        step()
    steps = []
    for i in range(new):
        tok.copy_(torch.stack([qkv[b, lens[b] + i] for b in range(3)])[:, None])
        g.replay()
        steps.append(out.clone())
    torch.cuda.synchronize()
    assert gdn.device_status() == 0 and n.tolist() == held

    gk, gv = gdn.kv_gather(cache, table, cu(held), sum(held), dtype=dtype)
    if bits is None:
        whole = lambda x: torch.cat([x[b, :m] for b, m in enumerate(held)])[None]  # noqa: E731
        assert torch.equal(gk, whole(rk)) and torch.equal(gv, whole(v))
    begin = 0
    for b, m in enumerate(held):
        kb, vb = np64(gk)[0, begin:begin + m], np64(gv)[0, begin:begin + m]
        begin += m
        ref, bound = bounds(np64(rq)[b, :m], kb, vb, dtype)
        if bits == 4:  # see attn_paged's own test
            bound += 1e-4 * D ** -0.5 * np.max(np.abs(np64(rq)[b, :m]).sum(-1)) * np.abs(kb).max() * np.abs(vb).max()
        got = np64(torch.cat([s[b] for s in steps]))
        err = np.abs(got - ref[lens[b]:]) - bound[lens[b]:]
        assert err.max() <= 0, (b, err.max())
        if bits is None:  # the prompt's attention saw the same keys
            first = sum(lens[:b])
            assert np.all(np.abs(np64(o)[0, first:first + lens[b]] - ref[:lens[b]]) <= bound[:lens[b]])


@gpu
@pytest.mark.parametrize("bits", [None, 4])
def test_a_prompt_goes_on(bits):
    """The second piece of two prompts: appended, all keys read back, attn_fwd over
    them; the last token's row is also attn_paged's."""
    first, piece = [50, 3], [21, 40]
    held = [a + b for a, b in zip(first, piece)]
    table, pages = tables(held, PAGE, 5)
    cos, sin = gdn.rope_table(max(held), D)
    cache = gdn.new_paged_cache(pages, PAGE, HKV, D, BF16, bits)
    qkv, _ = layer(1, 1, sum(first) + sum(piece), BF16)
    q, k, v = qkv.split([H, HKV, HKV], dim=2)
    n0 = sum(first)
    gdn.kv_append(k[:, :n0], v[:, :n0], cache, table, i32([0, 0]), cos=cos, sin=sin, cu_seqlens=cu(first))
    rq = gdn.kv_append(k[:, n0:], v[:, n0:], cache, table, i32(first), q[:, n0:], cos, sin, cu_seqlens=cu(piece))
    gk, gv = gdn.kv_gather(cache, table, cu(held), sum(held))
    o, _ = gdn.attn_fwd(rq, gk, gv, cu_seqlens=cu(piece), cu_seqlens_k=cu(held))
    assert gdn.device_status() == 0
    qb = kb = 0
    last = []
    for b, (m, p) in enumerate(zip(held, piece)):
        ref, bound = bounds(np64(rq)[0, qb:qb + p], np64(gk)[0, kb:kb + m], np64(gv)[0, kb:kb + m], BF16)
        assert np.all(np.abs(np64(o)[0, qb:qb + p] - ref) <= bound)
        qb, kb = qb + p, kb + m
        last.append((ref[-1], bound[-1], rq[0, qb - 1]))
    one = gdn.attn_paged(torch.stack([x[2] for x in last])[:, None].contiguous(), cache, table, i32([m - 1 for m in held]))
    for b, (ref, bound, _) in enumerate(last):
        slack = 0 if bits is None else 1e-3 * np.abs(np64(gv)).max()  # fp32 sums of scores from codes
        assert np.all(np.abs(np64(one)[b, 0] - ref) <= bound + slack)


@gpu
def test_training_step():
    """Norm, rotation and attention of packed sequences under autograd: the gradient
    of the whole is the composition of the calls' own, and of torch's in fp32."""
    lens = [33, 7, 90]
    T = sum(lens)
    qkv, w = layer(2, 1, T, F32)
    pos = torch.cat([torch.arange(n) for n in lens]).int()[None].cuda()
    cos, sin = gdn.rope_table(max(lens), D)
    do = torch.randn(1, T, H, D, generator=torch.Generator().manual_seed(3)).cuda()
    x = qkv.detach().requires_grad_()
    ws = [t.detach().requires_grad_() for t in w]
    q, k, v = x.split([H, HKV, HKV], dim=2)
    rq, rk = gdn.qk_norm_rope(q, k, *ws, cos, sin, pos)
    o = gdn.attention(rq, rk, v.contiguous(), cu_seqlens=cu(lens))
    got = torch.autograd.grad(o, [x, *ws], do)

    def plain(x, wq, wk):
        q, k, v = x.double().split([H, HKV, HKV], dim=2)
        c, s = cos.double()[pos.long()][:, :, None], sin.double()[pos.long()][:, :, None]

        def nr(t, w):
            t = t * (t.square().mean(-1, keepdim=True) + gdn.NORM_EPS).rsqrt() * w.double()
            a, b = t.chunk(2, -1)
            return torch.cat([a * c - b * s, b * c + a * s], -1)
        q, k = nr(q, wq), nr(k, wk)
        seq = torch.repeat_interleave(torch.arange(3), torch.tensor(lens)).cuda()
        see = (seq[:, None] == seq[None]) & torch.ones(T, T, dtype=torch.bool, device="cuda").tril()
        k, v = k.repeat_interleave(H // HKV, 2), v.repeat_interleave(H // HKV, 2)
        z = torch.einsum("bihd,bjhd->bhij", q, k) * D ** -0.5
        return torch.einsum("bhij,bjhd->bihd", torch.softmax(z.masked_fill(~see, -torch.inf), -1), v)
    y = [t.detach().clone().requires_grad_() for t in (qkv, *w)]
    want = torch.autograd.grad(plain(*y), y, do.double())
    for a, b in zip(got, want):
        # fp32 throughout: some 2e-5 of absolute sums (attention's bound) over gradients of the same order
        assert (a.double() - b).norm() <= 1e-4 * b.norm()


@gpu
def test_backward_in_a_graph_beside_an_eager_one():
    """A step's backward is captured while an eager pass of the same leaves is alive."""
    qkv, w = layer(4, 1, 40, BF16)
    cos, sin = gdn.rope_table(40, D)
    x = qkv.detach().requires_grad_()

    def loss():
        q, k, _ = x.split([H, HKV, HKV], dim=2)
        a, b = gdn.qk_norm_rope(q, k, *w, cos, sin)
        return a.float().square().sum() + b.float().sum()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        eager = loss()
        want, = torch.autograd.grad(loss(), x)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        got, = torch.autograd.grad(loss(), x)
    got.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    again, = torch.autograd.grad(eager, x)
    assert torch.equal(again, want)


@gpu
def test_calls_refuse_another_current_device(monkeypatch):
    """Every call asks for its stream, and that refuses; nothing is launched."""
    z = lambda *s, dt=BF16: torch.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
    q, k, w, c = z(1, 4, 2, 64), z(1, 4, 1, 64), z(64, dt=F32), z(8, 32, dt=F32)
    cache = gdn.new_paged_cache(4, 16, 1, 64, bits=4)
    table, n = z(1, 4, dt=torch.int32), z(1, dt=torch.int32)
    calls = (lambda: gdn.qk_norm_rope_fwd(q, k, w, w, c, c), lambda: gdn.qk_norm_rope_bwd(q, k, q, k, w, w, c, c),
             lambda: gdn.qk_norm_rope(q, k, w, w), lambda: gdn.kv_append(k, k, cache, table, n, q, c, c),
             lambda: gdn.kv_gather(cache, table, i32([0, 3]), 3), lambda: gdn.attn_paged(q, cache, table, n))
    with gdn.KernelTimer() as t:
        monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
        for call in calls:
            with pytest.raises(gdn.GdnError, match="current device"):
                call()
        monkeypatch.undo()
    assert t.launches == 0


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_gradients_between_boundaries_and_second_derivatives(dtype):
    """A gradient that starts on no 16-byte boundary is as good as a copy; a second
    derivative is refused."""
    qkv, w = layer(6, 1, 19, dtype)
    cos, sin = gdn.rope_table(19, D)
    x = qkv.detach().requires_grad_()

    def rows():
        q, k, _ = x.split([H, HKV, HKV], dim=2)
        return [t.flatten() for t in gdn.qk_norm_rope(q, k, *w, cos, sin)]
    n = sum(t.numel() for t in rows())
    do = torch.randn(n + 3, generator=torch.Generator().manual_seed(7)).to(dtype).cuda()
    want, = torch.autograd.grad((torch.cat(rows()) * do[3:]).sum(), x)
    got, = torch.autograd.grad((torch.cat([do[:3], *rows()]) * do).sum(), x)
    assert torch.equal(got, want)
    first, = torch.autograd.grad(torch.cat(rows()).float().square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="differentiate twice"):
        (first.float().square().sum() + x.float().sum()).backward()
    assert gdn.device_status() == 0
