"""Scores that climb (or fall) by some 100 along the keys, so that the running
maximum moves all the way and rows, warps and parts are joined at very different
maxima; against the fp64 oracle, element by element.

Bounds as in test_attention.py (e = 2^-8 for bf16, F = 2e-5), and on top what large
scores cost: a score is a sum of D <= 128 fp32 terms with the absolute sum A, off by
about sqrt(128) 2^-24 A, and its exponent's factor c by 2^-24 of itself: d = 2^-18 A
takes four times that.  A probability is off by d of itself and so is their sum: o by
2 d sum p |v|, lse by d.
"""
import numpy as np
import pytest
import torch

import gated_delta_rule_bwd_gb300 as gdn
from oracle import attention as at

gpu = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
E, F, DELTA = 2.0 ** -8, 2e-5, 2.0 ** -18


def np64(t):
    return t.detach().double().cpu().numpy()


def sloped(seed, B, Tq, Tk, H, Hkv, D, dtype, falling):
    """q near one direction per key head, k along it from -50 to 50 in the score."""
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    u = r(Hkv, D).sign()
    slope = torch.linspace(-50, 50, Tk) * (-1 if falling else 1) * D ** -0.5
    q = u.repeat_interleave(H // Hkv, 0) + 0.3 * r(B, Tq, H, D)
    k = slope[:, None, None] * u + 0.3 * r(B, Tk, Hkv, D)
    return [x.to(dtype).cuda() for x in (q, k, r(B, Tk, Hkv, D))]


def expect(q, k, v, bf16):
    """One head: o, lse and their bounds."""
    scale = q.shape[1] ** -0.5
    o, lse, a = at.attn_fwd(q, k, v, scale)
    d = DELTA * scale * (np.abs(q) @ np.abs(k).T).max(1)
    e = E if bf16 else 0.0
    return o, lse, (e + F + 2 * d[:, None]) * a + e * np.abs(o) + F * np.sqrt(np.mean(o * o)), F * (1 + np.abs(lse)) + d


def near(name, got, ref, bound):
    err = np.abs(np64(got) - ref) - bound
    i = np.unravel_index(np.argmax(err), err.shape)
    assert err[i] <= 0, f"{name}: {float(got[i]):.6e} for {ref[i]:.6e} at {i}, bound {bound[i]:.2e}"


@gpu
@pytest.mark.parametrize("falling", [False, True], ids=["climbing", "falling"])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("Tq,Tk,H,Hkv,D", [(300, 300, 4, 2, 128), (70, 2050, 3, 1, 64), (1, 4100, 2, 1, 128),
                                           (260, 3000, 2, 2, 80), (1500, 1500, 1, 1, 64)])
def test_prompt(Tq, Tk, H, Hkv, D, dtype, falling):
    q, k, v = sloped(Tk, 1, Tq, Tk, H, Hkv, D, dtype, falling)
    o, lse = gdn.attn_fwd(q, k, v)
    for h in range(H):
        ro, rl, bo, bl = expect(np64(q[0, :, h]), np64(k[0, :, h * Hkv // H]), np64(v[0, :, h * Hkv // H]), dtype is BF16)
        near("lse", lse[0, h], rl, bl)
        near("o", o[0, :, h], ro, bo)
    assert gdn.device_status() == 0


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_large_random_scores_have_an_exact_lse(dtype):
    """Scores up to about 300 in no order."""
    g = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn(1, 1500, h, 128, generator=g) for h in (2, 1, 1))
    q, k, v = (8 * q).to(dtype).cuda(), (8 * k).to(dtype).cuda(), v.to(dtype).cuda()
    o, lse = gdn.attn_fwd(q, k, v)
    for h in range(2):
        ro, rl, bo, bl = expect(np64(q[0, :, h]), np64(k[0, :, 0]), np64(v[0, :, 0]), dtype is BF16)
        near("lse", lse[0, h], rl, bl)
        near("o", o[0, :, h], ro, bo)


@gpu
@pytest.mark.parametrize("falling", [False, True], ids=["climbing", "falling"])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("B,T,n,H,Hkv,D", [
    (3, 3, 125, 4, 1, 128), (2, 1, 127, 32, 1, 64), (2, 2, 90, 4, 2, 80),      # a row whole in a CTA
    (1, 3, 8000, 4, 1, 128), (1, 1, 8000, 32, 1, 128), (2, 3, 5000, 20, 2, 64)])  # split over many
def test_decode(B, T, n, H, Hkv, D, dtype, falling):
    q, k, v = sloped(n, B, T, n + T, H, Hkv, D, dtype, falling)
    kc, vc = (torch.full((B, n + T + 5, Hkv, D), float("nan"), dtype=dtype, device="cuda") for _ in range(2))
    kc[:, :n], vc[:, :n] = k[:, :n], v[:, :n]
    lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
    o = gdn.attn_decode(q, k[:, n:].contiguous(), v[:, n:].contiguous(), kc, vc, lens)
    for b in range(B):
        for h in range(H):
            ro, _, bo, _ = expect(np64(q[b, :, h]), np64(k[b, :, h * Hkv // H]), np64(v[b, :, h * Hkv // H]), dtype is BF16)
            near("o", o[b, :, h], ro, bo)
    assert gdn.device_status() == 0
