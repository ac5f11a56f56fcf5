"""layer_norm_fwd / layer_norm_bwd against the fp64 oracle, element by element.

The kernels compute in fp32 and round each output once.  fp32: a row's sums of
D terms are off by a few 2^-24 sqrt(D) of their RMS, below 1e-5 for D <= 2^16,
and x - mean by 2^-23 of |x|: 2e-5 |ref| + 2e-5 rms.  bf16 outputs add half a
step, 2^-8 |ref|.  dweight and dbias are fp32 sums over the rows: 2e-5 of the
sum of their absolute terms, where x - mean counts as |x| + |mean| (it may cancel).
"""
import ctypes

import numpy as np
import pytest
import torch

import gated_delta_rule_bwd_gb300 as gdn
from oracle import attention as at

gpu = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
EPS = 1e-6
F = 2e-5


def np64(t):
    return t.detach().double().cpu().numpy()


def near(name, got, ref, bound):
    got = np64(got)
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    err = np.abs(got - ref)
    if ref.size:
        i = np.unravel_index(np.argmax(err - bound), ref.shape)
        assert np.all(err <= bound), f"{name}: {got[i]:.6e} for {ref[i]:.6e} at {i}"


def make(rows, D, dtype, seed=0, mean=0.5, std=1.0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x, dy = (r(rows, D) * std + mean).to(dtype).cuda(), r(rows, D).to(dtype).cuda()
    return x, (1 + 0.1 * r(D)).cuda(), (0.1 * r(D)).cuda(), dy


def compare(x, w, b, dy, eps=EPS):
    bf = x.dtype == BF16
    y, mean, rstd = gdn.layer_norm_fwd(x, w, b, eps)
    dx, dw, db = gdn.layer_norm_bwd(x, w, mean, rstd, dy)
    D = x.shape[-1]
    x2, dy2 = np64(x).reshape(-1, D), np64(dy).reshape(-1, D)
    w2, b2 = np64(w), None if b is None else np64(b)
    ry, rm, rr = at.layer_norm_fwd(x2, w2, b2, eps)
    rx, rw, rb = at.layer_norm_bwd(x2, w2, dy2, eps)
    rms = lambda a: np.sqrt(np.mean(a * a)) if a.size else 0.0  # noqa: E731
    h = 2.0 ** -8 if bf else 0.0
    near("y", y.reshape(-1, D), ry, (h + F) * np.abs(ry) + F * rms(ry))
    near("dx", dx.reshape(-1, D), rx, (h + F) * np.abs(rx) + F * (rms(rx) + rms(rr)))
    near("mean", mean.reshape(-1), rm, F * (np.abs(rm) + rms(x2)))
    near("rstd", rstd.reshape(-1), rr, F * rr)
    near("dw", dw, rw, F * (np.abs(dy2) * (np.abs(x2) + np.abs(rm)[:, None]) * rr[:, None]).sum(0))
    near("db", db, rb, F * np.abs(dy2).sum(0))
    return y, dx, dw, db


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("D", [1, 2, 7, 8, 100, 128, 257, 1000, 1024, 2048, 2056, 4100, 8192, 16384])
@pytest.mark.parametrize("rows", [1, 5, 700])
def test_against_oracle(rows, D, dtype):
    compare(*make(rows, D, dtype, seed=D + rows), eps=1e-6 if D > 2 else 1e-2)


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_many_rows_and_the_widest(dtype):
    compare(*make(20001, 96, dtype, seed=1))
    compare(*make(3, 65536, dtype, seed=2))


@gpu
def test_no_bias_shapes_and_no_rows():
    x, w, b, dy = make(24, 512, BF16, seed=3)
    compare(x, w, None, dy)
    y, *_ = gdn.layer_norm_fwd(x.view(2, 3, 4, 512), w, b)
    assert y.shape == (2, 3, 4, 512) and torch.equal(y.view(24, 512), gdn.layer_norm_fwd(x, w, b)[0])
    y, mean, rstd = gdn.layer_norm_fwd(x[:0], w, b)
    dx, dw, db = gdn.layer_norm_bwd(x[:0], w, mean, rstd, dy[:0])
    assert y.numel() == 0 and dx.numel() == 0 and not dw.any() and not db.any()


@gpu
def test_far_mean():
    """The variance is taken about the mean: a mean of 100 standard deviations
    costs 100 2^-24, not its square."""
    x, w, b, dy = make(50, 1024, F32, seed=4, mean=100.0)
    y, mean, rstd = gdn.layer_norm_fwd(x, w, b, EPS)
    ry, rm, rr = at.layer_norm_fwd(np64(x), np64(w), np64(b), EPS)
    # x - mean: the mean's own error, a few 100 2^-24
    near("y", y, ry, 1e-4 + F * np.abs(ry))
    near("rstd", rstd, rr, 1e-4 * rr)


@gpu
def test_constant_rows_and_non_finite_rows():
    """A constant row has y = bias; a NaN stays in its own row."""
    x, w, b, dy = make(6, 256, F32, seed=5)
    x[2] = 3.0
    x[4, 17] = float("nan")
    y, mean, rstd = gdn.layer_norm_fwd(x, w, b, EPS)
    assert torch.equal(y[2], b)
    assert y[4].isnan().all() and y[[0, 1, 2, 3, 5]].isfinite().all()
    dx, dw, db = gdn.layer_norm_bwd(x, w, mean, rstd, dy)
    assert dx[4].isnan().all() and dx[[0, 1, 2, 3, 5]].isfinite().all()


@gpu
def test_same_bits_every_time():
    x, w, b, dy = make(3001, 1024, BF16, seed=6)
    a, c = compare(x, w, b, dy), compare(x, w, b, dy)
    assert all(torch.equal(s, t) for s, t in zip(a, c))


@gpu
def test_autograd_and_differences():
    x, w, b, dy = make(5, 40, F32, seed=7)
    t = [u.requires_grad_() for u in (x, w, b)]
    (gdn.layer_norm(*t) * dy).sum().backward()
    loss = lambda *u: float((np64(gdn.layer_norm_fwd(*u)[0]) * np64(dy)).sum())  # noqa: E731
    r = np.random.default_rng(0)
    with torch.no_grad():
        for i, u in enumerate(t):
            d = torch.tensor(r.normal(size=u.shape), dtype=F32, device="cuda")
            h = 1e-2
            v = [z.clone() for z in t]
            v[i] = u + h * d
            up = loss(*v)
            v[i] = u - h * d
            num, ana = (up - loss(*v)) / (2 * h), float((u.grad.double() * d.double()).sum())
            assert abs(num - ana) <= 1e-3 * (abs(ana) + np.sqrt(dy.numel())), (i, num, ana)


def test_refusals():
    FAKE, odd = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10008)
    L = gdn.lib()
    s = lambda rows=4, D=64, dt=1: ctypes.byref(gdn.NormShape(rows, D, dt))  # noqa: E731
    fwd = lambda sh, x=FAKE, w=FAKE, b=None, y=FAKE, eps=1e-6: L.gdn_layer_norm_fwd(  # noqa: E731
        sh, x, w, b, y, None, None, eps, None)
    assert fwd(s(D=0)) == -2 and fwd(s(D=65537)) == -2 and fwd(s(rows=-1)) == -2
    assert fwd(s(dt=2)) == -3 and fwd(s(), eps=-1.0) == -1 and fwd(s(), eps=float("nan")) == -1
    assert fwd(s(), x=None) == -1 and fwd(s(), w=None) == -1 and fwd(s(), y=odd) == -4
    assert fwd(s(rows=0), x=None) == 0 and fwd(None) == -1
    need = L.gdn_layer_norm_bwd_workspace(s())
    bwd = lambda ws, n, dw=FAKE: L.gdn_layer_norm_bwd(  # noqa: E731
        s(), FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, dw, None, ws, n, None)
    assert need > 0 and bwd(None, 0) == -5 and bwd(FAKE, need - 1) == -5 and bwd(FAKE, need, None) == -1
    with pytest.raises(gdn.GdnError):
        gdn.layer_norm_fwd(torch.zeros(2, 8), torch.zeros(8))
