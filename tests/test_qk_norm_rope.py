"""qk_norm_rope_fwd / _bwd against the fp64 oracle, element by element.

The oracle sees the same bytes.  Everything is fp32 and rounded once: a norm's
sum has at most 5 terms per lane and 5 levels of lanes (value by value: the
same), each rounding at most 2^-24 of absolute sums, its square root a few more,
the products of norm and rotation five: a value is within 20 * 2^-24 < F = 2e-6
of the absolute terms of its formula, and e = 2^-8 of itself in bf16.  The
backward has the rotation's, the norm's and a second sum's errors: 2 F.  dw adds
one row after another, at most 1000 of them here in a lane's, a CTA's and the
CTAs' sums together: 1000 * 2^-24 < 6e-5 of the absolute sum.
"""
import ctypes

import numpy as np
import pytest
import torch

import gated_delta_rule_bwd_gb300 as gdn
from oracle import paging as pg

gpu = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
F = 2e-6
TYPES = pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])


def np64(t):
    return t.detach().double().cpu().numpy()


def inputs(B, T, H, Hkv, D, dtype, seed=0, fused=False):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g).to(dtype).cuda()  # noqa: E731
    if fused:
        q, k, _ = r(B, T, H + 2 * Hkv, D).split([H, Hkv, Hkv], dim=2)
    else:
        q, k = r(B, T, H, D), r(B, T, Hkv, D)
    w = [(1 + 0.3 * torch.randn(D, generator=g)).cuda() for _ in range(2)]
    return q, k, w, r(B, T, H, D), r(B, T, Hkv, D)


def check(q, k, w, dqo, dko, cos, sin, pos=None, interleaved=False, eps=1e-6):
    """One call of each against the oracle."""
    B, T = q.shape[:2]
    wq, wk = w if w is not None else (None, None)
    how = dict(cos=cos, sin=sin, positions=pos, interleaved=interleaved, eps=eps)
    out = gdn.qk_norm_rope_fwd(q, k, wq, wk, **how)
    grad = gdn.qk_norm_rope_bwd(q, k, dqo, dko, wq, wk, **how)
    assert gdn.device_status() == 0
    e = 2.0 ** -8 if q.dtype == BF16 else 0.0
    at = np.broadcast_to(np.arange(T), (B, T)) if pos is None else pos.cpu().numpy()
    c, s = (None, None) if cos is None else (np64(cos)[at][:, :, None], np64(sin)[at][:, :, None])
    for i, (x, dy) in enumerate(((q, dqo), (k, dko))):
        x, dy, wi = np64(x), np64(dy), None if w is None else np64(w[i])
        y = pg.norm_rope(x, wi, c, s, eps, interleaved)
        m = np.abs(pg.norm_rope(x, wi, None, None, eps))
        a = m.copy()
        if c is not None:  # |a c| + |b s| for the first halves, |b c| + |a s| for the second
            ia, ib = pg.pairs(2 * c.shape[-1], interleaved)
            a[..., ia] = m[..., ia] * np.abs(c) + m[..., ib] * np.abs(s)
            a[..., ib] = m[..., ib] * np.abs(c) + m[..., ia] * np.abs(s)
        dx, dw, ax, aw = pg.norm_rope_bwd(x, wi, c, s, dy, eps, interleaved)
        for name, got, want, bound in (("y", out[i], y, F * a), ("dx", grad[i], dx, 2 * F * ax)):
            got = np64(got)
            assert got.shape == want.shape
            err = np.abs(got - want) - bound - e * np.abs(want) - 1e-37
            assert not err.size or err.max() <= 0, (name, "qk"[i], err.max())
        if w is None:
            assert grad[2 + i] is None
        else:
            assert grad[2 + i].shape == wi.shape
            assert np.all(np.abs(np64(grad[2 + i]) - dw) <= 6e-5 * aw), ("dw", "qk"[i])
    return out, grad


@gpu
@TYPES
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("H,Hkv,D,R", [(2, 2, 128, 128), (8, 1, 64, 64), (3, 1, 80, 80), (5, 3, 128, 64), (2, 1, 96, 48),
                                       (1, 1, 8, 8), (2, 1, 33, 20), (1, 1, 1, 0), (4, 2, 2, 2), (3, 2, 64, 6),
                                       (16, 4, 128, 0), (2, 1, 127, 126), (4, 2, 24, 16)])
@pytest.mark.parametrize("B,T", [(1, 1), (2, 37), (3, 130)])
def test_sizes(B, T, H, Hkv, D, R, interleaved, dtype):
    q, k, w, dq, dk = inputs(B, T, H, Hkv, D, dtype, seed=T + D)
    cos, sin = gdn.rope_table(T, R) if R else (None, None)
    check(q, k, w, dq, dk, cos, sin, interleaved=interleaved)
    if R:
        check(q, k, None, dq, dk, cos, sin, interleaved=interleaved)


@gpu
@TYPES
def test_packed_positions_and_views(dtype):
    """Positions of packed sequences; q and k as views of one projection."""
    n = [5, 1, 200, 64]
    q, k, w, dq, dk = inputs(1, sum(n), 4, 2, 128, dtype, seed=3, fused=True)
    pos = torch.cat([torch.arange(100 * i, 100 * i + x) for i, x in enumerate(n)]).int()[None].cuda()
    cos, sin = gdn.rope_table(400, 128)
    a, _ = check(q, k, w, dq, dk, cos, sin, pos)
    b = gdn.qk_norm_rope_fwd(q.contiguous(), k.contiguous(), *w, cos, sin, pos)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@gpu
@TYPES
@pytest.mark.parametrize("layout", ["heads_first", "sliced_tokens", "expanded", "odd_base", "odd_tables"])
def test_layouts(layout, dtype):
    T, H, D = 50, 3, 64
    q, k, w, dq, dk = inputs(2, T, H, H, D, dtype, seed=11)
    cos, sin = gdn.rope_table(T, D)
    if layout == "heads_first":
        q, k = (x.transpose(1, 2).contiguous().transpose(1, 2) for x in (q, k))
    elif layout == "sliced_tokens":
        q, k = (torch.cat([x, x], 1)[:, 7:7 + T] for x in (q, k))
    elif layout == "expanded":
        k = k[:, :, :1].expand(2, T, H, D)
    elif layout == "odd_base":
        q, k = (torch.cat([x[..., :1], x, x[..., :2]], -1)[..., 1:1 + D] for x in (q, k))
    else:  # weights and tables that start between 16-byte boundaries
        w = [torch.cat([x[:1], x])[1:] for x in w]
        cos = torch.cat([cos.flatten()[:1], cos.flatten()])[1:].view(cos.shape)
    check(q, k, w, dq, dk, cos, sin)


@gpu
@TYPES
def test_far_positions(dtype):
    """A million positions in the table; the angles are the table's."""
    q, k, w, dq, dk = inputs(2, 3, 2, 1, 64, dtype, seed=4)
    cos, sin = gdn.rope_table(1 << 20, 64)
    pos = torch.tensor([[0, 1, (1 << 20) - 1], [999999, 524287, 7]], dtype=torch.int32, device="cuda")
    check(q, k, w, dq, dk, cos, sin, pos)
    at = np.arange((1 << 20) - 3, 1 << 20)[:, None] * 10000.0 ** (-np.arange(0, 64, 2) / 64)
    # the table itself: an angle below 2^20 is off by 2^-33 in 64 bits, a value by half a step of fp32
    assert np.abs(np64(cos[-3:]) - np.cos(at)).max() <= 2 ** -24 + 2 ** -32
    assert np.abs(np64(sin[-3:]) - np.sin(at)).max() <= 2 ** -24 + 2 ** -32


@gpu
@TYPES
@pytest.mark.parametrize("D", [64, 33])
def test_positions_outside_the_tables(D, dtype):
    """Rows of zeros, no gradient, and the status word; other tokens are as ever."""
    q, k, w, dq, dk = inputs(1, 4, 2, 1, D, dtype, seed=5)
    R = D // 2 * 2
    cos, sin = gdn.rope_table(10, R)
    pos = torch.tensor([[3, 10, -1, 9]], dtype=torch.int32, device="cuda")
    good = torch.tensor([[3, 0, 0, 9]], dtype=torch.int32, device="cuda")
    for eps in (1e-6, 0.0):
        y = gdn.qk_norm_rope_fwd(q, k, *w, cos, sin, pos, eps=eps)
        assert gdn.device_status() == -8 and gdn.device_status() == 0
        g = gdn.qk_norm_rope_bwd(q, k, dq, dk, *w, cos, sin, pos, eps=eps)
        assert gdn.device_status() == -8
        want = gdn.qk_norm_rope_fwd(q, k, *w, cos, sin, good, eps=eps)
        sel = [0, 3]
        s = lambda x: x[:, sel].contiguous()  # noqa: E731
        gw = gdn.qk_norm_rope_bwd(s(q), s(k), s(dq), s(dk), *w, cos, sin, s(good), eps=eps)
        for a, b, d, e in zip(y, want, g[:2], gw[:2]):
            assert not a[:, 1:3].any() and not d[:, 1:3].any()
            assert torch.equal(a[:, sel], b[:, sel]) and torch.equal(d[:, sel], e)
        for a, b in zip(g[2:], gw[2:]):  # the same terms, in another order of lanes
            assert torch.allclose(a, b, rtol=1e-5, atol=1e-5)


@gpu
@TYPES
@pytest.mark.parametrize("D", [64, 33])
def test_tokens_that_are_not_in_use(D, dtype):
    """Negative positions, as in a padded batch: zeros, no gradient, no error, whatever
    the rows hold."""
    q, k, w, dq, dk = inputs(1, 5, 2, 1, D, dtype, seed=15)
    cos, sin = gdn.rope_table(8, D // 2 * 2)
    pos = torch.tensor([[0, -1, 7, -(1 << 31), 3]], dtype=torch.int32, device="cuda")
    use = [0, 2, 4]
    q[:, [1, 3]], dq[:, [1, 3]], k[:, 1], dk[:, 3] = float("nan"), float("inf"), float("nan"), float("nan")
    for x in (w, (None, None)):
        y = gdn.qk_norm_rope_fwd(q, k, *x, cos, sin, pos)
        g = gdn.qk_norm_rope_bwd(q, k, dq, dk, *x, cos, sin, pos)
        assert gdn.device_status() == 0
        s = lambda t: t[:, use].contiguous()  # noqa: E731
        yw = gdn.qk_norm_rope_fwd(s(q), s(k), *x, cos, sin, s(pos))
        gw = gdn.qk_norm_rope_bwd(s(q), s(k), s(dq), s(dk), *x, cos, sin, s(pos))
        for a, b in zip((*y, *g[:2]), (*yw, *gw[:2])):
            assert torch.equal(a[:, use], b) and not a[:, [1, 3]].any()
        for a, b in zip(g[2:], gw[2:]):
            assert a is b is None or torch.allclose(a, b, rtol=1e-5, atol=1e-5)


@gpu
@TYPES
@pytest.mark.parametrize("D", [64, 31])
def test_zero_rows_and_other_rows_nan(D, dtype):
    """A row of zeros gives zeros and a finite gradient; a NaN stays in its row."""
    q, k, w, dq, dk = inputs(1, 9, 2, 1, D, dtype, seed=6)
    R = D // 2 * 2
    cos, sin = gdn.rope_table(9, R)
    clean = gdn.qk_norm_rope_fwd(q, k, *w, cos, sin)
    q[0, 3, 1] = 0
    q[0, 5, 0, D // 2] = float("nan")
    q[0, 6, 1, 0] = float("inf")
    y = gdn.qk_norm_rope_fwd(q, k, *w, cos, sin)
    assert not y[0][0, 3, 1].any() and y[0][0, 5, 0].isnan().all() and y[0][0, 6, 1].isnan().any()
    keep = torch.ones(9, 2, dtype=torch.bool, device="cuda")
    keep[3, 1] = keep[5, 0] = keep[6, 1] = False
    assert torch.equal(y[0][0][keep], clean[0][0][keep]) and torch.equal(y[1], clean[1])
    q[0, 5, 0], q[0, 6, 1] = 1, 1
    g = gdn.qk_norm_rope_bwd(q, k, dq, dk, *w, cos, sin)
    assert all(x.isfinite().all() for x in g)


@gpu
def test_unrotated_values_see_no_angle():
    """Infinite values past R do not become NaN by an angle of zero."""
    q = torch.full((1, 2, 1, 64), float("inf"), device="cuda")
    cos, sin = gdn.rope_table(2, 32)
    for il in (False, True):
        y, _ = gdn.qk_norm_rope_fwd(q, q, cos=cos, sin=sin, interleaved=il)
        assert y[..., 32:].isinf().all()


@gpu
@TYPES
def test_many_tokens(dtype):
    """More tokens than warps at once; and the same bits every time."""
    q, k, w, dq, dk = inputs(2, 4100, 3, 1, 64, dtype, seed=7)
    cos, sin = gdn.rope_table(4100, 64)
    out, grad = check(q, k, w, dq, dk, cos, sin)
    again = gdn.qk_norm_rope_bwd(q, k, dq, dk, *w, cos, sin)
    assert all(torch.equal(a, b) for a, b in zip(grad, again))


@gpu
def test_streams_graphs_and_workspace():
    q, k, w, dq, dk = inputs(2, 70, 4, 2, 128, BF16, seed=8)
    cos, sin = gdn.rope_table(70, 128)
    want = gdn.qk_norm_rope_fwd(q, k, *w, cos, sin), gdn.qk_norm_rope_bwd(q, k, dq, dk, *w, cos, sin)
    ws = torch.full((1 << 20,), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        got = gdn.qk_norm_rope_fwd(q, k, *w, cos, sin), gdn.qk_norm_rope_bwd(q, k, dq, dk, *w, cos, sin, workspace=ws)
    st.synchronize()
    assert all(torch.equal(a, b) for x, y in zip(got, want) for a, b in zip(x, y))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = gdn.qk_norm_rope_fwd(q, k, *w, cos, sin), gdn.qk_norm_rope_bwd(q, k, dq, dk, *w, cos, sin)
    for x in got:
        for t in x:
            t.zero_()
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for x, y in zip(got, want) for a, b in zip(x, y))


@gpu
def test_autograd():
    """The wrapper's gradients against differences, and weights without gradients."""
    q, k, w, dq, dk = inputs(1, 21, 2, 1, 32, F32, seed=9)
    cos, sin = gdn.rope_table(21, 32)
    x = [t.detach().clone().requires_grad_() for t in (q, k, *w)]
    yq, yk = gdn.qk_norm_rope(*x, cos, sin, interleaved=True)
    ((yq * dq).sum() + (yk * dk).sum()).backward()

    def loss(*y):
        a, b = gdn.qk_norm_rope_fwd(*y, cos, sin, interleaved=True)
        return float((np64(a) * np64(dq)).sum() + (np64(b) * np64(dk)).sum())
    r = np.random.default_rng(0)
    with torch.no_grad():
        for i, t in enumerate(x):
            d = torch.tensor(r.normal(size=t.shape), dtype=F32, device="cuda")
            h = 1e-2
            up, down = ([u if j != i else t + s * h * d for j, u in enumerate(x)] for s in (1, -1))
            num, ana = (loss(*up) - loss(*down)) / (2 * h), float((t.grad.double() * d.double()).sum())
            # h^2 / 6 times a third derivative of order the gradient's, over a direction of norm sqrt(n)
            assert abs(num - ana) <= 1e-3 * (abs(ana) + np.sqrt(t.numel()) * 4), (i, num, ana)
    yq, yk = gdn.qk_norm_rope(x[0], k, *w, cos, sin)
    x[0].grad = None
    yq.sum().backward()  # no gradient reaches yk
    assert x[0].grad.isfinite().all()


@gpu
@TYPES
def test_empty(dtype):
    cos, sin = gdn.rope_table(4, 16)
    w = [torch.ones(16, device="cuda")] * 2
    for B, T, H, Hkv in ((0, 4, 2, 1), (2, 0, 2, 1), (1, 4, 0, 0)):
        q, k = torch.empty(B, T, H, 16, dtype=dtype, device="cuda"), torch.empty(B, T, Hkv, 16, dtype=dtype, device="cuda")
        y = gdn.qk_norm_rope_fwd(q, k, *w, cos, sin)
        g = gdn.qk_norm_rope_bwd(q, k, q, k, *w, cos, sin)
        assert y[0].shape == q.shape and not g[2].any() and not g[3].any()
    q, k, w, dq, dk = inputs(1, 4, 2, 1, 16, dtype)
    none = k[:, :, :0]
    y = gdn.qk_norm_rope_fwd(q, none, *w, cos, sin)
    g = gdn.qk_norm_rope_bwd(q, none, dq, none, *w, cos, sin)
    assert torch.equal(y[0], gdn.qk_norm_rope_fwd(q, k, *w, cos, sin)[0]) and not g[3].any() and g[2].any()
    assert gdn.device_status() == 0


# ------------------------------------------------------------------ refusals (host side)

FAKE = ctypes.c_void_p(0x10000)  # never dereferenced


def shape(B=1, T=8, H=2, Hkv=1, D=16, R=16, P=8, il=0, dtype=1, qs=(256, 32, 16), ks=(128, 16, 16)):
    return gdn.QkRopeShape(B, T, H, Hkv, D, R, P, il, dtype, qs, ks)


def fwd(s, q=FAKE, k=FAKE, wq=FAKE, wk=FAKE, eps=1e-6, cos=FAKE, sin=FAKE, pos=None, qo=FAKE, ko=FAKE):
    return gdn.lib().gdn_qk_norm_rope_fwd(ctypes.byref(s), q, k, wq, wk, eps, cos, sin, pos, qo, ko, None)


def bwd(s, ws=FAKE, n=1 << 30, wq=FAKE, wk=FAKE, dwq=FAKE, dq=FAKE, dqo=FAKE):
    return gdn.lib().gdn_qk_norm_rope_bwd(ctypes.byref(s), FAKE, FAKE, wq, wk, 1e-6, FAKE, FAKE, None, dqo, FAKE, dq, FAKE,
                                          dwq, FAKE, ws, n, None)


def test_refusals():
    ARG, SHAPE, DTYPE, ALIGN, WS = -1, -2, -3, -4, -5
    odd = lambda n: ctypes.c_void_p(0x10000 + n)  # noqa: E731
    for kw in (dict(D=0), dict(D=129), dict(R=17), dict(R=3), dict(R=-2), dict(B=-1), dict(T=-1), dict(H=-1), dict(H=70000),
               dict(Hkv=70000), dict(B=1 << 20, T=1 << 20), dict(qs=(-1, 32, 16)), dict(ks=(0, 0, -1)), dict(P=-1),
               dict(B=1 << 30, T=1, H=1 << 10)):
        assert fwd(shape(**kw)) == SHAPE, kw
    for t in (2, 3, -1):
        assert fwd(shape(dtype=t)) == DTYPE
    for kw in (dict(q=None), dict(k=None), dict(wq=None), dict(wk=None), dict(cos=None), dict(sin=None), dict(qo=None),
               dict(ko=None), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf"))):
        assert fwd(shape(), **kw) == ARG, kw
    none = dict(cos=None, sin=None)
    assert fwd(shape(R=0), **none, wq=None, wk=None) == ARG and fwd(shape(R=0), **none, pos=FAKE) == ARG
    assert fwd(shape(R=0)) == ARG  # tables without pairs
    for kw in (dict(q=odd(1)), dict(k=odd(1)), dict(wq=odd(2)), dict(cos=odd(2)), dict(pos=odd(2)), dict(qo=odd(8)), dict(ko=odd(4))):
        assert fwd(shape(), **kw) == ALIGN, kw
    assert fwd(shape(B=0), q=None, k=None, qo=None, ko=None) == 0
    assert gdn.lib().gdn_qk_norm_rope_fwd(None, *[FAKE] * 4, 1e-6, *[FAKE] * 5, None) == ARG
    need = gdn.lib().gdn_qk_norm_rope_bwd_workspace(ctypes.byref(shape()))
    assert need > 0 and gdn.lib().gdn_qk_norm_rope_bwd_workspace(None) == 0
    assert bwd(shape(), None) == WS and bwd(shape(), FAKE, need - 1) == WS and bwd(shape(), odd(8)) == ALIGN
    assert bwd(shape(), dwq=None) == ARG and bwd(shape(), dq=None) == ARG and bwd(shape(), dqo=odd(4)) == ALIGN


def test_binding_refuses_cpu_tensors():
    q = torch.zeros(1, 4, 2, 16)
    with pytest.raises(gdn.GdnError, match="CUDA"):
        gdn.qk_norm_rope_fwd(q, q, cos=q, sin=q)
    with pytest.raises(gdn.GdnError):
        gdn.rope_table(4, 3, device="cpu")


@gpu
def test_binding_refusals():
    z = lambda *s, dt=BF16: torch.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
    q, k, w = z(1, 4, 2, 16), z(1, 4, 1, 16), z(16, dt=F32)
    c = z(4, 8, dt=F32)
    p = torch.zeros(1, 4, dtype=torch.int32, device="cuda")
    for call in (lambda: gdn.qk_norm_rope_fwd(q, k), lambda: gdn.qk_norm_rope_fwd(q, k, w), lambda: gdn.qk_norm_rope_fwd(q, k, w, w, c),
                 lambda: gdn.qk_norm_rope_fwd(q, k, w, w, c, c[:3]), lambda: gdn.qk_norm_rope_fwd(q, k, w, w, c.bfloat16(), c.bfloat16()),
                 lambda: gdn.qk_norm_rope_fwd(q, k, w, w, z(4, 9, dt=F32), z(4, 9, dt=F32)), lambda: gdn.qk_norm_rope_fwd(q, k, w, w[:8]),
                 lambda: gdn.qk_norm_rope_fwd(q, k[:, :3], w, w), lambda: gdn.qk_norm_rope_fwd(q, k.float(), w, w),
                 lambda: gdn.qk_norm_rope_fwd(q, k, w, w, positions=p), lambda: gdn.qk_norm_rope_fwd(q, k, w, w, c, c, p.long()),
                 lambda: gdn.qk_norm_rope_fwd(q, k, w, w, c, c, p[0]), lambda: gdn.qk_norm_rope_fwd(q, k, w.cpu(), w.cpu()),
                 lambda: gdn.qk_norm_rope_fwd(q.transpose(2, 3), k, w, w), lambda: gdn.qk_norm_rope_fwd(q.half(), k.half(), w, w),
                 lambda: gdn.qk_norm_rope_bwd(q, k, q, q, w, w), lambda: gdn.qk_norm_rope_bwd(q, k, q.float(), k, w, w),
                 lambda: gdn.qk_norm_rope_fwd(q, k, w, w, eps=-1.0), lambda: gdn.qk_norm_rope_fwd(q, k, w, w, z(4, 0, dt=F32), z(4, 0, dt=F32))):
        with pytest.raises(gdn.GdnError):
            call()
    assert gdn.device_status() == 0
