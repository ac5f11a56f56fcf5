"""attn_paged against the fp64 oracle, element by element.

The oracle attends over the values that the pages stand for (4-bit codes times
steps, exact in bf16).  Bounds as for the form on a contiguous cache: a bf16
weight that feeds the tensor cores is off by e = 2^-8 of itself (4 bits: the
probability times the value's step is that weight, rounded once) and the result
is rounded once, so o is within e (a + |o|), a = sum p |v|; fp32 terms add 2e-5 of
the absolute sums.  Scores from 4-bit keys are products with codes + 136 less 136
times the sum of q: fp32 sums about 45 times the size of the result, 32 terms per
step, 45 * 32 * 2^-24 < 1e-4 of sum |q||k| in the worst case, which moves a
probability by as much (the scores here are below 10 in sum |q||k| scale).
"""
import ctypes

import numpy as np
import pytest
import torch

import gated_delta_rule_bwd_gb300 as gdn
from oracle import attention as at
from oracle import paging as pg
from tests.test_kv_cache import cache_desc, i32, np64, places, tables, BAD_CACHES

gpu = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
E, F = 2.0 ** -8, 2e-5
FORMATS = pytest.mark.parametrize("dtype,bits", [(BF16, None), (F32, None), (BF16, 4), (F32, 4)],
                                  ids=["bf16", "f32", "bf16-4", "f32-4"])


def random_cache(pages, page, Hkv, D, dtype, bits, seed, unused=False):
    """A cache full of normal values (``unused``: of NaN, codes of any kind)."""
    g = torch.Generator().manual_seed(seed)
    cache = gdn.new_paged_cache(pages, page, Hkv, D, dtype, bits)
    for x in cache:
        if x is None:
            continue
        if x.dtype == torch.uint8:
            n = torch.randn(*x.shape, 2, generator=g).mul(3).round().clamp(-7, 7).add(8).to(torch.uint8)
            x.copy_(n[..., 0] | n[..., 1] << 4)
        elif bits == 4:
            x.copy_(torch.randint(16, 32, x.shape, generator=g) / 64)
        else:
            x.copy_(torch.randn(x.shape, generator=g).to(dtype))
    return cache


def seen(cache, table, b, n, page):
    """Row b's first n tokens' k and v [n, Hkv, D] in fp64."""
    p = places(np.full(n, b), np.arange(n), table, page)
    p = tuple(torch.tensor(x, device="cuda").long() for x in p)
    if cache[0].dtype != torch.uint8:
        return np64(cache[0][p]), np64(cache[1][p])
    return tuple(pg.values(cache[i][p].cpu().numpy(), np64(cache[2 + i][p])) for i in range(2))


def reference(q, cache, table, lens, page, scale):
    B, T, H, D = q.shape
    G = H // cache[0].shape[2]
    e = E if q.dtype == BF16 else 0.0
    ref, bound = np.zeros(q.shape), np.zeros(q.shape)
    q = np64(q)
    for b, n in enumerate(lens):
        if n < 0:
            continue
        k, v = seen(cache, table, b, n + T, page)
        for h in range(H):
            o, _, a = at.attn_fwd(q[b, :, h], k[:, h // G], v[:, h // G], scale)
            ref[b, :, h], bound[b, :, h] = o, (e + F) * a
            if cache[0].dtype == torch.uint8:
                bound[b, :, h] += 1e-4 * scale * np.max(np.abs(q[b, :, h]) @ np.abs(k[:, h // G]).T) * a
    rms = np.sqrt(np.mean(ref * ref)) if ref.size else 0.0
    return ref, bound + e * np.abs(ref) + F * rms


def check(lens, T, H, Hkv, D, page, dtype, bits, seed=0, scale=None, change=None):
    held = [max(n, 0) + T for n in lens]
    table, pages = tables(held, page, seed)
    q = torch.randn(len(lens), T, H, D, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()
    cache = random_cache(pages, page, Hkv, D, dtype, bits, seed + 1)
    if change is not None:
        cache, table, q = change(cache, table, q)
    ref, bound = reference(q, cache, table, lens, page, D ** -0.5 if scale is None else scale)
    o = gdn.attn_paged(q, cache, table, i32(lens), scale)
    assert gdn.device_status() == 0
    got = np64(o)
    assert got.shape == ref.shape and np.all(np.isfinite(got))
    err = np.abs(got - ref) - bound
    i = np.unravel_index(np.argmax(err), err.shape)
    assert err[i] <= 0, f"{got[i]:.6e} for {ref[i]:.6e} at {i}, bound {bound[i]:.2e}"
    return o, q, cache, table


@gpu
@FORMATS
@pytest.mark.parametrize("H,Hkv,D", [(8, 2, 128), (4, 4, 64), (6, 1, 96), (16, 1, 128), (40, 1, 64), (2, 2, 32), (3, 1, 128)])
@pytest.mark.parametrize("T", [1, 3])
@pytest.mark.parametrize("page", [16, 64])
def test_sizes(page, T, H, Hkv, D, dtype, bits):
    check([0, 1, 62, 63, 64, 130, 700, -1], T, H, Hkv, D, page, dtype, bits, seed=D + T)


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("H,Hkv,D", [(6, 1, 80), (2, 1, 33), (2, 2, 8), (1, 1, 1), (4, 2, 120)])
def test_other_head_sizes(H, Hkv, D, dtype):
    check([0, 5, 200, 64], 2, H, Hkv, D, 16, dtype, None, seed=D)


@gpu
@FORMATS
@pytest.mark.parametrize("page", [1, 2, 4, 8, 32, 256, 4096])
def test_page_sizes(page, dtype, bits):
    check([0, 17, 300], 1, 4, 2, 64, page, dtype, bits, seed=page)


@gpu
@FORMATS
def test_one_long_row_among_short_ones(dtype, bits):
    """Rows that are split over many CTAs, and rows of one piece."""
    check([30000, 3, 0, 5000], 2, 8, 2, 128, 64, dtype, bits, seed=2)


@gpu
@FORMATS
def test_many_rows(dtype, bits):
    r = np.random.default_rng(3)
    check([int(x) for x in r.integers(0, 300, 200)], 1, 4, 2, 64, 16, dtype, bits, seed=3, scale=0.2)


@gpu
@FORMATS
@pytest.mark.parametrize("layout", ["tokens_first", "one_layer", "wide_table"])
def test_layouts(layout, dtype, bits):
    def change(cache, table, q):
        cache = [x for x in cache if x is not None]
        if layout == "tokens_first":
            cache = [x.contiguous() for x in cache]
        elif layout == "one_layer":
            cache = [torch.stack([x, x, x], 1)[:, 1] for x in cache]
        else:
            table = torch.cat([table, table, table], 1)[:, :table.shape[1]]
        return cache, table, q
    check([0, 100, 77], 1, 4, 2, 128, 32, dtype, bits, seed=4, change=change)


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_cache_between_boundaries(dtype):
    def change(cache, table, q):
        flat = [torch.cat([x.flatten()[:1], x.flatten()])[1:].view(x.shape) for x in (y.contiguous() for y in cache[:2])]
        return flat, table, q
    check([0, 100, 77], 1, 4, 2, 128, 32, dtype, None, seed=4, change=change)


@gpu
@FORMATS
def test_slots_past_the_row_are_not_read(dtype, bits):
    """They hold NaN (codes with NaN steps); shared pages serve two rows."""
    lens, T, page = [0, 5, 64, 70], 2, 16

    def change(cache, table, q):
        for b, n in enumerate(lens):
            last = n + T
            if last % page:
                p = int(table[b, last // page])
                for x in cache[2:] if bits else cache[:2]:
                    x[p, last % page:] = float("nan")
        return cache, table, q
    o, q, cache, table = check(lens, T, 4, 2, 64, page, dtype, bits, seed=5, change=change)
    table2 = table.clone()
    table2[2] = table[3]  # row 2 as a reader of row 3's pages
    a = gdn.attn_paged(q, cache, table2, i32(lens))
    b = gdn.attn_paged(q[2:3].contiguous(), cache, table[3:4], i32(lens[2:3]))
    assert torch.allclose(a[2], b[0], rtol=2 ** -7, atol=2 ** -7) and torch.equal(a[1], o[1])


@gpu
@FORMATS
def test_nan_reaches_its_rows_only(dtype, bits):
    lens, page = [150, 90, 40], 16
    o, q, cache, table = check(lens, 1, 4, 2, 64, page, dtype, bits, seed=6)
    p = int(table[1, 2])
    if bits:
        cache[2][p, 3, 1, 0] = float("nan")  # a key of row 1, head 1
    else:
        cache[0][p, 3, 1, 5] = float("nan")
    got = gdn.attn_paged(q, cache, table, i32(lens))
    assert got[1, 0, 2:].isnan().all()
    got[1, 0, 2:] = o[1, 0, 2:]
    assert torch.equal(got, o)
    q[0, 0, 0, 7] = float("nan")
    q[2, 0, 1, 7] = float("inf")
    got = gdn.attn_paged(q, cache, table, i32(lens))
    assert got[0, 0, 0].isnan().all() and not got[2, 0, 1].isfinite().all()
    assert torch.equal(got[0, 0, 1:], o[0, 0, 1:]) and torch.equal(got[2, 0, 0], o[2, 0, 0]) and torch.equal(got[2, 0, 2:], o[2, 0, 2:])


@gpu
@FORMATS
@pytest.mark.parametrize("rise", [False, True])
def test_moving_maximum(rise, dtype, bits):
    """Scores that climb or fall by 100 along the keys: earlier sums are scaled down,
    or later ones vanish.  Scores of 100 are off by 100 * 2^-23 in fp32, 4 bits: by
    1e-4 of them in the worst case, 1e-2 of a probability: relative L2 2e-2."""
    n, D, page = 600, 64, 16
    table, pages = tables([n], page)
    q = torch.zeros(1, 1, 2, D, device="cuda", dtype=dtype)
    q[..., 0] = 8.0
    cache = random_cache(pages, page, 1, D, dtype, bits, 7)
    slot = np.arange(n)
    p = tuple(torch.tensor(x, device="cuda").long() for x in places(np.zeros(n, int), slot, table, page))
    ramp = torch.tensor(slot if rise else slot[::-1].copy(), device="cuda") / n * 100
    if bits:
        c = cache[0][p]
        c[:, 0, 0] = (c[:, 0, 0] & 0xf0) | 15  # code 7 of the first value
        cache[0][p] = c
        s = cache[2][p]
        s[:, 0, 0] = (ramp / 7).to(torch.float8_e5m2).to(BF16)
        cache[2][p] = s
    else:
        k = cache[0][p]
        k[:, 0, 0] = ramp.to(dtype)
        cache[0][p] = k
    ref, _ = reference(q, cache, table, [n - 1], page, D ** -0.5)
    o = np64(gdn.attn_paged(q, cache, table, i32([n - 1])))
    assert gdn.device_status() == 0
    assert np.linalg.norm(o - ref) <= (2e-2 if dtype == BF16 or bits else 3e-4) * np.linalg.norm(ref)


@gpu
@FORMATS
@pytest.mark.parametrize("size", [1e-30, 1e6, 1e30])
def test_sizes_of_values(size, dtype, bits):
    """Very small and very large keys against queries that make up for it, and
    values of that size: nothing leaves fp32's or bf16's range on the way."""
    lens, page, D = [100, 7], 16, 64

    def change(cache, table, q):
        for x in (cache[2:] if bits else cache[:2]):
            x.mul_(size)
        return cache, table, (q.float() / size).to(dtype)
    check(lens, 1, 4, 2, D, page, dtype, bits, seed=8, change=change)


@gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("order", ["rising", "falling", "mixed", "by group"])
def test_steps_of_many_sizes(order, D):
    """4 bits: steps of values from 2^-12 to 2^12 of one another, along the sequence or
    from one 32 values to the next.  The fp16 weights' absolute error, 2^-30 of the
    largest step of a value's 32, is far below the bound's 2^-9 of the weighted sum,
    in which every key has its part."""
    lens, page = [700, 45, 31, 3000], 16
    held = [n + 1 for n in lens]

    def change(cache, table, q):
        g = torch.Generator().manual_seed(3)
        for b, n in enumerate(held):
            at_ = tuple(torch.tensor(x, device="cuda").long() for x in places(np.full(n, b), np.arange(n), table, page))
            e = torch.linspace(-12, 12, n)[:, None, None].expand(n, 2, D // 32).round()
            if order == "falling":
                e = -e
            elif order == "mixed":
                e = torch.randint(-12, 13, e.shape, generator=g)
            elif order == "by group":
                e = torch.linspace(-12, 12, D // 32).round().expand(e.shape)
            cache[3][at_] = cache[3][at_] * torch.exp2(e.float()).cuda().to(cache[3].dtype)
        return cache, table, q
    check(lens, 1, 8, 2, D, page, BF16, 4, seed=21, change=change)


@gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_step_that_is_no_number(bad, D):
    """4 bits: such a step of a value reaches its own 32 values of its key head, and
    leaves the others as they were."""
    lens, page = [300, 20], 16
    held = [n + 1 for n in lens]
    table, pages = tables(held, page, 22)
    q = torch.randn(2, 1, 8, D, generator=torch.Generator().manual_seed(22)).to(BF16).cuda()
    cache = random_cache(pages, page, 2, D, BF16, 4, 23)
    o = gdn.attn_paged(q, cache, table, i32(lens))
    p = places(np.array([0]), np.array([150]), table, page)
    cache[3][int(p[0][0]), int(p[1][0]), 1, 1] = bad
    x = gdn.attn_paged(q, cache, table, i32(lens))
    assert gdn.device_status() == 0
    hit = torch.zeros_like(o, dtype=torch.bool)
    hit[0, :, 4:, 32:64] = True
    assert not torch.isfinite(x[hit]).any()
    assert torch.equal(x[~hit], o[~hit])


@gpu
@FORMATS
def test_same_bits_streams_and_graphs(dtype, bits):
    lens = [3000, 1, 333, -1]
    o, q, cache, table = check(lens, 1, 8, 2, 128, 64, dtype, bits, seed=9)
    n = i32(lens)
    need = torch.full((1 << 24,), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        a = gdn.attn_paged(q, cache, table, n, workspace=need)
    st.synchronize()
    assert torch.equal(a, o)
    g, h = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):  # two graphs that share a workspace, replayed one after the other
        a = gdn.attn_paged(q, cache, table, n, workspace=need)
    with torch.cuda.graph(h):
        b = gdn.attn_paged(q, cache, table, n, workspace=need)
    a.zero_(), b.zero_()
    g.replay(), h.replay()
    torch.cuda.synchronize()
    assert torch.equal(a, o) and torch.equal(b, o)
    n.copy_(i32([5, 2999, -1, 64]))  # other lengths for the same graph
    g.replay()
    c = gdn.attn_paged(q, cache, torch.where(table > 1 << 20, table[:1], table), i32([5, -1, -1, -1]))
    torch.cuda.synchronize()
    assert torch.equal(a[0], c[0]) and not a[2].any()
    gdn.device_status()  # the longer row's table has entries of no page


@gpu
@FORMATS
def test_bad_rows_are_reported(dtype, bits):
    D, page = 64, 8
    cache = random_cache(6, page, 1, D, dtype, bits, 10)
    q = torch.ones(3, 2, 2, D, device="cuda", dtype=dtype)
    table = i32([[0, 1], [2, 3], [4, 5]])
    good = gdn.attn_paged(q, cache, table, i32([14, 3, -5]))
    assert gdn.device_status() == 0 and good[:2].any() and not good[2].any()
    for n in (15, 1 << 30, (1 << 31) - 1):
        o = gdn.attn_paged(q, cache, table, i32([14, 3, n]))
        assert gdn.device_status() == -8 and gdn.device_status() == 0
        assert torch.equal(o, good)
    for n in (6, -1, 1 << 30, -(1 << 31)):
        bad = i32([[0, 1], [2, 3], [4, n]])
        o = gdn.attn_paged(q, cache, bad, i32([14, 3, 8]))
        assert gdn.device_status() == -9 and gdn.device_status() == 0
        assert torch.equal(o[:2], good[:2])
    o = gdn.attn_paged(q, cache, i32([[0, 1], [2, 77], [99, 99]]), i32([14, 3, -1]))  # entries of no token
    assert gdn.device_status() == 0 and torch.equal(o, good)


@gpu
@pytest.mark.parametrize("bits", [None, 4])
def test_offsets_past_32_bits(bits):
    """The last pages of a cache of more than 2^32 bytes."""
    Hkv, D, page = 8, 128, 256
    n = (1 << 32) // (Hkv * page * (D if bits is None else D // 2)) + 3
    small = random_cache(2, page, Hkv, D, BF16, bits, 11)
    cache = gdn.new_paged_cache(n, page, Hkv, D, BF16, bits)
    for x, y in zip(cache, small):
        if x is not None:
            x[n - 2:].copy_(y)
    q = torch.randn(1, 1, 16, D, generator=torch.Generator().manual_seed(1)).to(BF16).cuda()
    a = gdn.attn_paged(q, cache, i32([[n - 1, n - 2]]), i32([400]))
    b = gdn.attn_paged(q, small, i32([[1, 0]]), i32([400]))
    assert gdn.device_status() == 0 and torch.equal(a, b) and a.any()


@gpu
def test_as_on_a_contiguous_cache():
    """The same values as attn_decode's within the bounds of both."""
    lens, T, H, Hkv, D, page = [130, 5], 1, 8, 2, 128, 64
    o, q, cache, table = check(lens, T, H, Hkv, D, page, BF16, None, seed=12)
    S = 160
    kc, vc = (torch.zeros(2, S, Hkv, D, dtype=BF16, device="cuda") for _ in range(2))
    new = []
    for b, n in enumerate(lens):
        p = tuple(torch.tensor(x, device="cuda").long() for x in places(np.full(n + T, b), np.arange(n + T), table, page))
        kc[b, :n + T], vc[b, :n + T] = cache[0][p], cache[1][p]
        new.append((kc[b, n:n + T].clone(), vc[b, n:n + T].clone()))
    k, v = (torch.stack([x[i] for x in new]) for i in range(2))
    want = gdn.attn_decode(q, k, v, kc, vc, i32(lens))
    _, bound = reference(q, cache, table, lens, page, D ** -0.5)
    assert np.all(np.abs(np64(o) - np64(want)) <= 2 * bound)


@gpu
@FORMATS
def test_empty(dtype, bits):
    cache = random_cache(2, 16, 1, 64, dtype, bits, 0)
    for B, T, H in ((0, 1, 2), (2, 0, 2)):
        q = torch.empty(B, T, H, 64, dtype=dtype, device="cuda")
        assert gdn.attn_paged(q, cache, i32([[0]] * B).view(B, -1) if B else torch.empty(0, 1, dtype=torch.int32, device="cuda"),
                              i32([0] * B)).shape == q.shape
    q = torch.ones(2, 1, 2, 64, dtype=dtype, device="cuda")
    o = gdn.attn_paged(q, cache, torch.empty(2, 0, dtype=torch.int32, device="cuda"), i32([-1, -1]))
    assert gdn.device_status() == 0 and not o.any()


# ------------------------------------------------------------------ refusals (host side)

FAKE = ctypes.c_void_p(0x10000)  # never dereferenced


def call(c=None, B=2, T=1, H=2, dtype=1, most=4, stride=4, q=FAKE, table=FAKE, lens=FAKE, scale=0.5, o=FAKE, ws=None, n=0):
    c = cache_desc() if c is None else c
    s = gdn.AttnPagedShape(B, T, H, dtype, most, stride)
    return gdn.lib().gdn_attn_paged(ctypes.byref(s), ctypes.byref(c), q, table, lens, scale, o, ws, n, None)


@pytest.mark.parametrize("kw,status", BAD_CACHES, ids=str)
def test_caches_that_are_refused(kw, status):
    assert call(cache_desc(**kw)) == status


def test_refusals():
    odd = lambda n: ctypes.c_void_p(0x10000 + n)  # noqa: E731
    for kw in (dict(B=-1), dict(T=-1), dict(H=-1), dict(H=0), dict(H=70000), dict(H=3, c=cache_desc(Hkv=2)), dict(c=cache_desc(Hkv=0)),
               dict(B=70000), dict(B=20000, H=4, c=cache_desc(Hkv=4)), dict(T=300000), dict(most=-1), dict(most=1 << 27), dict(stride=-1)):
        assert call(**kw) == -2, kw
    assert call(dtype=0) == -3 and call(dtype=2) == -3 and call(cache_desc(format=0)) == -3
    for x in (0.0, -1.0, float("nan"), float("inf")):
        assert call(scale=x) == -1
    for kw in (dict(q=None), dict(table=None), dict(lens=None), dict(o=None)):
        assert call(**kw) == -1, kw
    for kw in (dict(q=odd(8)), dict(o=odd(8)), dict(ws=odd(8)), dict(lens=odd(2)), dict(table=odd(2))):
        assert call(**kw) == -4, kw
    assert call() == -5
    s, c = gdn.AttnPagedShape(2, 1, 2, 1, 4, 4), cache_desc()
    need = gdn.lib().gdn_attn_paged_workspace(ctypes.byref(s), ctypes.byref(c))
    assert need > 0 and call(ws=FAKE, n=need - 1) == -5
    assert call(B=0, q=None) == 0 and call(T=0, q=None) == 0
    assert gdn.lib().gdn_attn_paged_workspace(None, ctypes.byref(c)) == 0
    assert gdn.lib().gdn_attn_paged_workspace(ctypes.byref(s), None) == 0


def test_binding_refuses_cpu_tensors():
    q = torch.zeros(1, 1, 2, 32)
    cache = gdn.new_paged_cache(2, 8, 1, 32, torch.float32, device="cpu")
    with pytest.raises(gdn.GdnError, match="CUDA"):
        gdn.attn_paged(q, cache, torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32))


@gpu
def test_binding_refusals():
    z = lambda *s, dt=BF16: torch.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
    q, t, n = z(2, 1, 2, 64), z(2, 4, dt=torch.int32), z(2, dt=torch.int32)
    c, f = gdn.new_paged_cache(8, 16, 1, 64), gdn.new_paged_cache(8, 16, 1, 64, bits=4)
    for bad in (lambda: gdn.attn_paged(q.float(), c, t, n), lambda: gdn.attn_paged(q.half(), f, t, n), lambda: gdn.attn_paged(q[..., :32], c, t, n),
                lambda: gdn.attn_paged(z(2, 2, 2, 64).transpose(1, 2), c, t, n), lambda: gdn.attn_paged(z(2, 1, 3, 64), gdn.new_paged_cache(8, 16, 2, 64), t, n),
                lambda: gdn.attn_paged(q, c, t[:1], n), lambda: gdn.attn_paged(q, c, t.long(), n), lambda: gdn.attn_paged(q, c, t, n[:1]),
                lambda: gdn.attn_paged(q, c, t, n.long()), lambda: gdn.attn_paged(q, c, t.t().contiguous().t(), n), lambda: gdn.attn_paged(q, f[:3], t, n),
                lambda: gdn.attn_paged(q, c, t, n, scale=0.0), lambda: gdn.attn_paged(q, (c.k, c.v[..., ::2]), t, n)):
        with pytest.raises(gdn.GdnError):
            bad()
    assert gdn.device_status() == 0
