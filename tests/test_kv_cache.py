"""kv_append and kv_gather against the fp64 oracle.

Rotation is two products and a sum, each rounded to fp32: within 3 * 2^-24 <
F = 2e-7 of |a c| + |b s|, and bf16 adds half a step, 2^-8 of the value.  4-bit
storage: the step is amax / 7 within 2^-5 of itself (5 significant bits), and a
value lies within half a step of what it is stored as, each up to F of the
group's largest magnitude, by which the rotated value differs from the oracle's.
The codes are also those of the same formula with each operation rounded to fp32,
bit for bit.
"""
import ctypes

import numpy as np
import pytest
import torch

import gated_delta_rule_bwd_gb300 as gdn
from oracle import paging as pg

gpu = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
F = 2e-7
TYPES = pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])


def np64(t):
    return t.detach().double().cpu().numpy()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def cu(n):
    return i32(np.concatenate([[0], np.cumsum(n)]).astype(int).tolist())


def tables(held, page, seed=0, spare=2):
    """A block table of pages in no order for rows that hold that many tokens;
    entries of no page are out of range."""
    each = [-(-n // page) for n in held]
    order = np.random.default_rng(seed).permutation(sum(each) + spare)
    t = np.full((len(held), max(each + [1])), 1 << 30)
    at = 0
    for b, n in enumerate(each):
        t[b, :n] = order[at:at + n]
        at += n
    return i32(t.tolist()), sum(each) + spare


def inputs(B, T, H, Hkv, D, dtype, seed=0, fused=False):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g).to(dtype).cuda()  # noqa: E731
    if fused:
        return r(B, T, H + 2 * Hkv, D).split([H, Hkv, Hkv], dim=2)
    return r(B, T, H, D), r(B, T, Hkv, D), r(B, T, Hkv, D)


def filled(cache):
    """The cache with old contents that must survive."""
    for x in cache:
        if x is not None:
            x.copy_(torch.full_like(x, 77) if x.dtype == torch.uint8 else torch.full_like(x, 5.5))
    return cache


def places(row, slot, table, page):
    t = table.cpu().numpy()
    return t[row, slot // page], slot % page


def turned(x, slot, cos, sin, interleaved):
    """Tokens x [n, heads, D] in fp64, rotated, and the absolute terms."""
    if cos is None:
        return x, np.abs(x)
    c, s = np64(cos)[slot][:, None], np64(sin)[slot][:, None]
    ia, ib = pg.pairs(2 * c.shape[-1], interleaved)
    a = np.abs(x)
    m = a.copy()
    m[..., ia], m[..., ib] = a[..., ia] * np.abs(c) + a[..., ib] * np.abs(s), a[..., ib] * np.abs(c) + a[..., ia] * np.abs(s)
    return pg.rotate(x, c, s, interleaved), m


def stored(x):
    """Codes [.., D / 2] and steps of fp32 values, each operation in fp32."""
    x = x.astype(np.float32).reshape(*x.shape[:-1], -1, 32)
    step = np.abs(x).max(-1) * np.float32(1 / 7)
    step = ((step.view(np.int32) + 0x40000) & np.int32(-0x80000)).view(np.float32)
    s = step[..., None]
    n = np.clip(np.rint(x / np.where(s > 0, s, np.float32(1))) * (s > 0), -7, 7).astype(np.int32) + 8
    n = n.reshape(*n.shape[:-2], -1).astype(np.uint8)
    return n[..., 0::2] | n[..., 1::2] << 4, step


def fp32_turned(x, slot, cos, sin, interleaved):
    if cos is None:
        return x
    c, s = cos.cpu().numpy()[slot][:, None], sin.cpu().numpy()[slot][:, None]
    ia, ib = pg.pairs(2 * c.shape[-1], interleaved)
    y = x.copy()
    y[..., ia], y[..., ib] = x[..., ia] * c - x[..., ib] * s, x[..., ib] * c + x[..., ia] * s
    return y


def check(new, used, H, Hkv, D, page, dtype, bits=None, R=None, interleaved=False, packed=None, fused=False, seed=0,
          change=None):
    """Appends new[b] tokens behind used[b] and compares the whole cache."""
    R = D if R is None else R
    packed = len(set(new)) > 1 if packed is None else packed
    held = [a + b for a, b in zip(new, used)]
    table, pages = tables(held, page, seed)
    B, T = (1, sum(new)) if packed else (len(new), new[0])
    q, k, v = inputs(B, T, H, Hkv, D, dtype, seed, fused)
    cos, sin = gdn.rope_table(max(held), R) if R else (None, None)
    cache = filled(gdn.new_paged_cache(pages, page, Hkv, D, dtype, bits))
    if change is not None:
        cache, k, v = change(cache, k, v)
    want = [np.array(np64(x)) for x in cache if x is not None]
    lens = i32(used)
    qo = gdn.kv_append(k, v, cache, table, lens, q=q if H else None, cos=cos, sin=sin, interleaved=interleaved,
                       cu_seqlens=cu(new) if packed else None)
    assert gdn.device_status() == 0 and lens.tolist() == list(used)
    row = np.repeat(np.arange(len(new)), new)
    slot = np.concatenate([np.arange(a, a + b) for a, b in zip(used, new)]).astype(int)
    at = places(row, slot, table, page)
    flat = lambda x: np64(x).reshape(-1, *x.shape[2:])  # noqa: E731
    e = 2.0 ** -8 if dtype == BF16 else 0.0
    if H:
        y, m = turned(flat(q), slot, cos, sin, interleaved)
        assert np.all(np.abs(flat(qo) - y) <= F * m + e * np.abs(y))
        if R and not packed and len(set(used)) == 1:
            pos = i32([[used[0] + t for t in range(T)]] * B)
            same = gdn.qk_norm_rope_fwd(q, k, cos=cos, sin=sin, positions=pos, interleaved=interleaved)
            assert torch.equal(same[0], qo)
            if bits is None:
                for b in range(B):
                    a = [torch.tensor(x[b * T:(b + 1) * T], device="cuda") for x in at]
                    assert torch.equal(cache[0][a[0], a[1]], same[1][b])
    else:
        assert qo is None
    for i, (x, c, s) in enumerate(((k, cos, sin), (v, None, None))):
        y, m = turned(flat(x), slot, c, s, interleaved)
        got = np64(cache[i])
        if bits is None:
            assert np.all(np.abs(got[at] - y) <= (F * m if c is not None else 0) + (e * np.abs(y) if c is not None else 0))
        else:
            x32 = x.float().cpu().numpy().reshape(-1, Hkv, D)
            codes, steps = stored(fp32_turned(x32, slot, c, s, interleaved))
            steps_got = np64(cache[2 + i])
            assert np.array_equal(steps_got[at], steps) and np.array_equal(got[at], codes)
            back = pg.values(got[at].astype(np.uint8), steps_got[at])
            amax = np.abs(y).reshape(-1, Hkv, D // 32, 32).max(-1)
            wide = lambda z: np.repeat(z, 32, -1)  # noqa: E731
            off = F * m.reshape(-1, Hkv, D // 32, 32).max(-1) if c is not None else 0 * amax
            assert np.all(np.abs(steps_got[at] - amax / 7) <= (amax + off) / 7 * (2.0 ** -5 + 1e-6) + off)
            assert np.all(np.abs(back - y) <= wide(steps_got[at] * (0.5 + 1e-6) + off))
            want[2 + i][at] = steps_got[at]
        want[i][at] = got[at]
        assert np.array_equal(got, want[i])  # all other slots as they were
        if bits is not None:
            assert np.array_equal(np64(cache[2 + i]), want[2 + i])
    # and back out
    k2, v2 = gdn.kv_gather(cache, table, cu(held), sum(held))
    assert gdn.device_status() == 0
    row = np.repeat(np.arange(len(new)), held)
    slot = np.concatenate([np.arange(n) for n in held]).astype(int)
    at = places(row, slot, table, page)
    for i, x in enumerate((k2, v2)):
        assert x.shape == (1, sum(held), Hkv, D)
        y = want[i][at] if bits is None else pg.values(want[i][at].astype(np.uint8), want[2 + i][at])
        assert np.array_equal(np64(x)[0], y)
    if bits is not None:
        k3, v3 = gdn.kv_gather(cache, table, cu(held), sum(held), dtype=F32)
        assert torch.equal(k3, k2.float()) and torch.equal(v3, v2.float())


@gpu
@TYPES
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("H,Hkv,D,R", [(8, 2, 128, 128), (0, 1, 64, 64), (4, 4, 64, 32), (2, 1, 33, 32), (3, 3, 80, 40),
                                       (0, 2, 128, 0), (1, 1, 1, 0), (2, 2, 96, 96), (16, 1, 128, 64)])
@pytest.mark.parametrize("new,used", [([1] * 5, [0, 7, 8, 31, 100]), ([3, 1, 40, 0, 17], [0, 63, 5, 9, 64]), ([70], [13])])
def test_append(new, used, H, Hkv, D, R, interleaved, dtype):
    check(new, used, H, Hkv, D, 16, dtype, R=R, interleaved=interleaved, fused=len(new) > 1, seed=D + len(new))


@gpu
@TYPES
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("H,Hkv,D,R", [(8, 2, 128, 128), (0, 1, 64, 64), (4, 4, 64, 32), (0, 2, 128, 0), (2, 1, 96, 48),
                                       (3, 3, 32, 32), (1, 2, 128, 20)])
@pytest.mark.parametrize("new,used", [([1] * 5, [0, 7, 8, 31, 100]), ([3, 1, 40, 0, 17], [0, 63, 5, 9, 64]), ([70], [13])])
def test_append_4_bits(new, used, H, Hkv, D, R, interleaved, dtype):
    check(new, used, H, Hkv, D, 16, dtype, 4, R=R, interleaved=interleaved, fused=len(new) > 1, seed=D + len(new))


@gpu
@pytest.mark.parametrize("bits", [None, 4])
@pytest.mark.parametrize("page", [1, 2, 64, 1024])
def test_page_sizes(page, bits):
    check([5, 130, 1], [3, 60, 1], 2, 2, 64, page, BF16, bits, seed=page)


@gpu
@pytest.mark.parametrize("bits", [None, 4])
def test_many_tokens(bits):
    """More tokens than warps at once, more heads than a warp's rows on their way."""
    check([3000, 1, 257], [0, 900, 5], 24, 3, 128, 64, BF16, bits, seed=1)


@gpu
@TYPES
@pytest.mark.parametrize("bits", [None, 4])
@pytest.mark.parametrize("layout", ["tokens_first", "one_layer", "odd_k", "expanded_v", "one_page"])
def test_layouts(layout, bits, dtype):
    """Caches with tokens outside heads, one layer's part of a larger tensor, and
    tokens that start between 16-byte boundaries."""
    def change(cache, k, v):
        cache = [x for x in cache if x is not None]
        if layout == "tokens_first":
            cache = [x.contiguous() for x in cache]
        elif layout == "one_layer":
            cache = [torch.stack([x, x, x], 1)[:, 1] for x in cache]
        elif layout == "odd_k":
            k, v = (torch.cat([x[..., :1], x, x[..., :2]], -1)[..., 1:1 + x.shape[-1]] for x in (k, v))
        elif layout == "expanded_v":
            v = v[:, :, :1].expand(v.shape)
        else:
            cache = [x[:, :, :, :] for x in cache]
        return cache, k, v
    new, used = ([4, 9, 30], [0, 17, 2]) if layout != "one_page" else ([2], [3])
    check(new, used, 3, 2, 64, 8, dtype, bits, seed=5, change=change)
    if bits is None:  # a cache on no 16-byte boundary
        def odd(cache, k, v):
            flat = [torch.cat([x.flatten()[:1], x.flatten()])[1:].view(x.shape) for x in (y.contiguous() for y in cache[:2])]
            return flat, k, v
        check(new, used, 3, 2, 64, 8, dtype, None, seed=5, change=odd)


@gpu
@pytest.mark.parametrize("bits", [None, 4])
def test_rows_that_are_not_in_use(bits):
    """A negative length, tokens behind the last sequence: nothing is stored, q is 0,
    and no error; a captured graph serves batches of different fill."""
    Hkv, D, page = 2, 64, 16
    table, pages = tables([40, 40, 40], page)
    q, k, v = inputs(1, 12, 4, Hkv, D, BF16, 3)
    cos, sin = gdn.rope_table(40, D)
    cache, want = (filled(gdn.new_paged_cache(pages, page, Hkv, D, BF16, bits)) for _ in range(2))
    lens, offs = i32([5, -1, 8]), i32([0, 4, 6, 9])
    g = torch.cuda.CUDAGraph()
    gdn.kv_append(k, v, cache, table, i32([-1, -7, -1 << 31]), q, cos, sin, cu_seqlens=offs)
    assert all(torch.equal(a, b) for a, b in zip(cache, want) if a is not None)
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        qo = gdn.kv_append(k, v, cache, table, lens, q, cos, sin, cu_seqlens=offs)
    for n, o in (([5, -1, 8], [0, 4, 6, 9]), ([0, 0, -1], [0, 1, 1, 1]), ([-1, 3, 3], [0, 0, 12, 12]), ([1, 1, 1], [0, 0, 0, 0])):
        lens.copy_(i32(n)), offs.copy_(i32(o))
        qo.fill_(9)
        g.replay()
        assert gdn.device_status() == 0
        for b in range(3):
            sl = slice(o[b], o[b + 1])
            if n[b] < 0:
                assert not qo[:, sl].any()
                continue
            one = gdn.kv_append(k[:, sl], v[:, sl], want, table[b:b + 1], i32(n[b:b + 1]), q[:, sl], cos, sin)
            assert torch.equal(one, qo[:, sl])
        assert not qo[:, o[3]:].any()
        assert all(torch.equal(a, b) for a, b in zip(cache, want) if a is not None)


@gpu
@pytest.mark.parametrize("bits", [None, 4])
def test_bad_rows_are_reported(bits):
    """Lengths past the table, slots past the angles, pages that are not there: the
    token is left out, the status word tells, and others go in."""
    Hkv, D, page = 1, 64, 8
    q, k, v = inputs(3, 2, 2, Hkv, D, BF16, 3)
    cos, sin = gdn.rope_table(16, D)
    table = i32([[0, 1], [2, 3], [4, 5]])
    fresh = lambda: filled(gdn.new_paged_cache(6, page, Hkv, D, BF16, bits))  # noqa: E731
    want = fresh()
    gdn.kv_append(k[:1], v[:1], want, table[:1], i32([3]), q[:1], cos, sin)
    for lens, status in (([3, 15, -1], -8), ([3, 1 << 30, (1 << 31) - 1], -8)):
        cache = fresh()
        qo = gdn.kv_append(k, v, cache, table, i32(lens), q, cos, sin)
        assert gdn.device_status() == status and gdn.device_status() == 0
        assert not qo[1:].any() and qo[0].any()
        assert all(torch.equal(a, b) for a, b in zip(cache, want) if a is not None)
    cache = fresh()  # angles for four positions only
    gdn.kv_append(k, v, cache, table, i32([2, 3, -1]), q, cos[:4].contiguous(), sin[:4].contiguous())
    assert gdn.device_status() == -8
    assert cache[0][2, 3].ne(5.5 if bits is None else 77).any() and torch.equal(cache[0][2, 4], want[0][2, 4])
    for page_no in (6, -1, 1 << 30, -(1 << 31)):
        cache = fresh()
        bad = i32([[0, 1], [page_no, 3], [4, 5]])
        qo = gdn.kv_append(k, v, cache, bad, i32([3, 0, -1]), q, cos, sin)
        assert gdn.device_status() == -9 and gdn.device_status() == 0
        assert qo[1].any()  # it is rotated all the same
        assert all(torch.equal(a, b) for a, b in zip(cache, want) if a is not None)
        a, b = gdn.kv_gather(cache, bad, cu([5, 3, 0]), 8)
        assert gdn.device_status() == -9
        assert not a[0, 5:].any() and not b[0, 5:].any() and a[0, :5].any()
    # offsets that do not rise: reported, and nothing outside the arrays
    packed = [x.reshape(1, 6, -1, D) for x in (k, v, q)]
    for o in ([0, 4, 2, 6], [1, 2, 3, 6], [0, 2, 4, 7], [0, -5, 4, 6], [0, 2, 1 << 30, 6]):
        gdn.kv_append(packed[0], packed[1], fresh(), table, i32([0, 0, 0]), packed[2], cos, sin, cu_seqlens=i32(o))
        assert gdn.device_status() == -8, o
        gdn.kv_gather(cache, table, i32(o), 6)
        assert gdn.device_status() == -8, o
    gdn.kv_gather(cache, table, i32([0, 2, 4, 5]), 6)
    assert gdn.device_status() == -8
    gdn.kv_gather(cache, table, i32([0, 17, 17, 17]), 17)  # longer than its pages
    assert gdn.device_status() == -8


@gpu
@TYPES
def test_values_that_4_bits_do_not_hold(dtype):
    """A NaN or infinity makes its 32 values NaN and no others; the largest and the
    smallest magnitudes, and zeros."""
    D = 64
    _, k, v = inputs(1, 6, 0, 1, D, dtype, 4)
    big = torch.finfo(dtype).max
    k[0, 0, 0, 3], k[0, 1, 0, 40], k[0, 1, 0, 41] = float("nan"), float("inf"), float("-inf")
    k[0, 2] = 0
    k[0, 3] = big
    k[0, 4] = 1e-44 if dtype == F32 else 2.0 ** -133
    k[0, 5, 0, :32] = torch.linspace(-2.0 ** -130, 2.0 ** -130, 32).to(dtype)
    cache = gdn.new_paged_cache(1, 8, 1, D, dtype, 4)
    table = i32([[0]])
    gdn.kv_append(k, v, cache, table, i32([0]))
    a, b = gdn.kv_gather(cache, table, i32([0, 6]), 6, dtype=F32)
    assert gdn.device_status() == 0
    nan = torch.zeros(6, 2, dtype=torch.bool, device="cuda")
    nan[0, 0] = nan[1, 1] = True
    assert torch.equal(a[0, :, 0].view(6, 2, 32).isnan().all(-1), nan) and torch.equal(a[0, :, 0].view(6, 2, 32).isnan().any(-1), nan)
    assert not a[0, 2].any() and a[0, 3].isfinite().all() and b.isfinite().all()
    codes, steps = stored(k[0, 2:].float().cpu().numpy())
    assert np.array_equal(cache[0][0, 2:6].cpu().numpy(), codes) and np.array_equal(np64(cache[2][0, 2:6]), steps)


@gpu
def test_gather_leaves_nothing_out():
    """Rows of no tokens, one long row, more heads than a CTA's run of tokens."""
    for held, Hkv, D, dtype in (([0, 0, 7, 0], 1, 8, BF16), ([5000], 2, 128, BF16), ([3, 9], 300, 128, F32), ([1] * 50, 1, 33, BF16),
                                ([77, 1], 3, 20, F32)):
        table, pages = tables(held, 32)
        cache = gdn.PagedCache(*(torch.randn(pages, 32, Hkv, D, device="cuda").to(dtype) for _ in range(2)))
        k, v = gdn.kv_gather(cache, table, cu(held), sum(held))
        assert gdn.device_status() == 0
        row = np.repeat(np.arange(len(held)), held)
        slot = np.concatenate([np.arange(n) for n in held]).astype(int)
        at = tuple(torch.tensor(x, device="cuda").long() for x in places(row, slot, table, 32))
        assert torch.equal(k[0], cache.k[at]) and torch.equal(v[0], cache.v[at])
    k, v = gdn.kv_gather(cache, table, i32([0, 0, 0]), 0)
    assert k.shape == (1, 0, 3, 20)


@gpu
@pytest.mark.parametrize("bits", [None, 4])
def test_offsets_past_32_bits(bits):
    """A cache of more than 2^32 bytes and, in elements, more than 2^31."""
    Hkv, D, page = 8, 128, 256
    n = (1 << 32) // (Hkv * page * (D if bits is None else D // 2)) + 3
    cache = gdn.new_paged_cache(n, page, Hkv, D, BF16, bits)
    _, k, v = inputs(1, 300, 0, Hkv, D, BF16, 6)
    table = i32([[n - 1, n - 2]])
    gdn.kv_append(k, v, cache, table, i32([100]))
    a, b = gdn.kv_gather(cache, table, i32([0, 400]), 400)
    assert gdn.device_status() == 0 and not a[0, :100].any()
    if bits is None:
        assert torch.equal(a[0, 100:], k[0]) and torch.equal(b[0, 100:], v[0])
    else:
        small = gdn.new_paged_cache(2, page, Hkv, D, BF16, bits)
        gdn.kv_append(k, v, small, i32([[0, 1]]), i32([0]))
        c, d = gdn.kv_gather(small, i32([[0, 1]]), i32([0, 300]), 300)
        assert torch.equal(a[0, 100:], c[0]) and torch.equal(b[0, 100:], d[0])
    assert not any(x[:n - 2].any() for x in cache[:2])


@gpu
def test_streams():
    q, k, v = inputs(2, 40, 4, 2, 64, BF16, 8)
    cos, sin = gdn.rope_table(50, 64)
    table = i32([[0, 1, 2, 3], [7, 6, 5, 4]])
    caches = [gdn.new_paged_cache(8, 16, 2, 64, BF16, 4) for _ in range(2)]
    a = gdn.kv_append(k, v, caches[0], table, i32([3, 0]), q, cos, sin)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        b = gdn.kv_append(k, v, caches[1], table, i32([3, 0]), q, cos, sin)
        r = gdn.kv_gather(caches[1], table, i32([0, 43, 83]), 83)
    st.synchronize()
    assert torch.equal(a, b) and all(torch.equal(x, y) for x, y in zip(*caches))
    assert all(torch.equal(x, y) for x, y in zip(r, gdn.kv_gather(caches[0], table, i32([0, 43, 83]), 83)))


# ------------------------------------------------------------------ refusals (host side)

FAKE = ctypes.c_void_p(0x10000)  # never dereferenced


def cache_desc(pages=4, page=16, Hkv=1, D=64, format=1, k=0x10000, ks=0x10000, st=(1024, 64, 64), ss=(32, 2, 2)):
    return gdn.PagedCacheDesc(pages, page, Hkv, D, format, k, 0x10000, ks, 0x10000, st, st, ss, ss)


def append(c=None, B=2, T=3, H=2, R=64, P=8, il=0, dtype=1, rows=2, most=4, stride=4, qs=(0, 0, 0), k=FAKE, v=FAKE, q=FAKE, cos=FAKE,
           sin=FAKE, table=FAKE, lens=FAKE, cu=None, qo=FAKE):
    c = cache_desc() if c is None else c
    s = gdn.KvAppendShape(B, T, H, R, P, il, dtype, rows, most, stride, qs, (0, 0, 0), (0, 0, 0))
    return gdn.lib().gdn_kv_append(ctypes.byref(s), ctypes.byref(c), k, v, q, cos, sin, table, lens, cu, qo, None)


def gather(c=None, table=FAKE, rows=2, most=4, stride=4, cu=FAKE, total=5, dtype=1, k=FAKE, v=FAKE):
    c = cache_desc() if c is None else c
    return gdn.lib().gdn_kv_gather(ctypes.byref(c), table, rows, most, stride, cu, total, dtype, k, v, None)


BAD_CACHES = [(dict(pages=-1), -2), (dict(page=0), -2), (dict(page=24), -2), (dict(page=-16), -2), (dict(Hkv=-1), -2), (dict(Hkv=70000), -2),
              (dict(D=0), -2), (dict(D=129), -2), (dict(format=2, D=48), -2), (dict(st=(-1, 64, 64)), -2), (dict(format=3), -3),
              (dict(format=-1), -3), (dict(k=None), -1), (dict(k=0x10001), -4), (dict(format=2, ks=None), -1), (dict(format=2, k=0x10008), -4),
              (dict(format=2, ks=0x10008), -4), (dict(format=2, st=(1024, 40, 64)), -4), (dict(format=2, ss=(32, 3, 2)), -4),
              (dict(format=2, ss=(32, -2, 2)), -2)]


@pytest.mark.parametrize("kw,status", BAD_CACHES, ids=str)
def test_caches_that_are_refused(kw, status):
    assert append(cache_desc(**kw)) == status and gather(cache_desc(**kw)) == status


def test_append_refusals():
    ARG, SHAPE, DTYPE, ALIGN = -1, -2, -3, -4
    odd = lambda n: ctypes.c_void_p(0x10000 + n)  # noqa: E731
    for kw in (dict(B=-1, rows=-1), dict(T=-1), dict(H=-1), dict(H=70000), dict(R=66), dict(R=3), dict(P=-1), dict(rows=3), dict(cu=FAKE),
               dict(B=1, rows=-1, cu=FAKE), dict(most=-1), dict(most=1 << 27), dict(stride=-4), dict(qs=(0, -1, 0)), dict(B=1 << 20, rows=1 << 20, T=1 << 20)):
        assert append(**kw) == SHAPE, kw
    assert append(dtype=0) == DTYPE and append(dtype=2) == DTYPE and append(cache_desc(format=0)) == DTYPE
    for kw in (dict(k=None), dict(v=None), dict(q=None), dict(qo=None), dict(cos=None), dict(sin=None), dict(R=0), dict(table=None), dict(lens=None)):
        assert append(**kw) == ARG, kw
    for kw in (dict(k=odd(1)), dict(v=odd(1)), dict(q=odd(1)), dict(cos=odd(2)), dict(sin=odd(1)), dict(table=odd(2)), dict(lens=odd(2)),
               dict(B=1, cu=odd(2)), dict(qo=odd(8))):
        assert append(**kw) == ALIGN, kw
    assert append(B=0, rows=0) == 0 and append(T=0, k=None) == 0
    c = ctypes.byref(cache_desc())
    assert gdn.lib().gdn_kv_append(None, c, *[FAKE] * 10) == ARG
    s = gdn.KvAppendShape()
    assert gdn.lib().gdn_kv_append(ctypes.byref(s), None, *[FAKE] * 10) == ARG


def test_gather_refusals():
    odd = lambda n: ctypes.c_void_p(0x10000 + n)  # noqa: E731
    for kw in (dict(rows=-1), dict(most=-1), dict(most=1 << 27), dict(stride=-1), dict(total=-1), dict(total=(1 << 30) + 1)):
        assert gather(**kw) == -2, kw
    assert gather(dtype=0) == -3 and gather(dtype=2) == -3
    for kw in (dict(table=None), dict(cu=None), dict(k=None), dict(v=None)):
        assert gather(**kw) == -1, kw
    for kw in (dict(table=odd(2)), dict(cu=odd(1)), dict(k=odd(8)), dict(v=odd(4))):
        assert gather(**kw) == -4, kw
    assert gather(total=0, k=None, v=None) == 0


def test_binding_refuses_on_the_cpu():
    k = torch.zeros(1, 4, 1, 32)
    cache = gdn.new_paged_cache(2, 8, 1, 32, torch.float32, device="cpu")
    n, t = torch.zeros(1, dtype=torch.int32), torch.zeros(1, 2, dtype=torch.int32)
    with pytest.raises(gdn.GdnError, match="CUDA"):
        gdn.kv_append(k, k, cache, t, n)
    with pytest.raises(gdn.GdnError, match="CUDA"):
        gdn.kv_gather(cache, t, n, 0)
    for kw in (dict(bits=8), dict(page=12), dict(page=0), dict(dtype=torch.float16), dict(D=48, bits=4)):
        with pytest.raises(gdn.GdnError):
            gdn.new_paged_cache(**{**dict(pages=1, page=8, Hkv=1, D=32, device="cpu"), **kw})
    four = gdn.new_paged_cache(2, 8, 3, 64, bits=4, device="cpu")
    assert [tuple(x.shape) for x in four] == [(2, 8, 3, 32)] * 2 + [(2, 8, 3, 2)] * 2


@gpu
def test_binding_refusals():
    z = lambda *s, dt=BF16: torch.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
    k, q, t, n = z(2, 3, 1, 64), z(2, 3, 2, 64), z(2, 4, dt=torch.int32), z(2, dt=torch.int32)
    c = gdn.new_paged_cache(8, 16, 1, 64)
    f = gdn.new_paged_cache(8, 16, 1, 64, bits=4)
    x = z(8, 32, dt=F32)
    off = z(3, dt=torch.int32)
    for call in (lambda: gdn.kv_append(k, k[:, :2], c, t, n), lambda: gdn.kv_append(k, k.float(), c, t, n), lambda: gdn.kv_append(k.float(), k.float(), c, t, n),
                 lambda: gdn.kv_append(k, k, c, t, n.long()), lambda: gdn.kv_append(k, k, c, t, n[:1]), lambda: gdn.kv_append(k, k, c, t[:1], n),
                 lambda: gdn.kv_append(k, k, c, t.long(), n), lambda: gdn.kv_append(k, k, c, t[0], n), lambda: gdn.kv_append(k, k, c[:1], t, n),
                 lambda: gdn.kv_append(k, k, (c.k, c.v[:, :8]), t, n), lambda: gdn.kv_append(k, k, (c.k, c.v.float()), t, n),
                 lambda: gdn.kv_append(k, k, (f.k, f.v), t, n), lambda: gdn.kv_append(k, k, (f.k, f.v, f.k_scale, f.v_scale[..., :1]), t, n),
                 lambda: gdn.kv_append(k, k, (f.k, f.v, f.k_scale.float(), f.v_scale), t, n), lambda: gdn.kv_append(z(2, 3, 2, 64), z(2, 3, 2, 64), c, t, n),
                 lambda: gdn.kv_append(k[..., :32], k[..., :32], c, t, n), lambda: gdn.kv_append(k, k, c, t, n, q[:, :2]),
                 lambda: gdn.kv_append(k, k, c, t, n, q.float()), lambda: gdn.kv_append(k, k, c, t, n, q, x), lambda: gdn.kv_append(k, k, c, t, n, q, x, x[:4]),
                 lambda: gdn.kv_append(k, k, c, t, n, cu_seqlens=off), lambda: gdn.kv_append(k, k, c, t.cpu(), n),
                 lambda: gdn.kv_append(k, k, [y.cpu() for y in c[:2]], t, n), lambda: gdn.kv_append(k, k, (c.k[:, :12], c.v[:, :12]), t, n),
                 lambda: gdn.kv_gather(c, t, off[:2], 4), lambda: gdn.kv_gather(c, t, off, 4, dtype=F32), lambda: gdn.kv_gather(f, t, off, 4, dtype=torch.half)):
        with pytest.raises(gdn.GdnError):
            call()
    assert gdn.device_status() == 0
