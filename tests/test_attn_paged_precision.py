"""attn_paged to the precision that its kernels hold, against the fp64 oracle.

With bf16 queries a probability meets its value in two bf16 terms.  The first is off
by up to 2^-8 of it, the second by 2^-8 of what the first leaves: 2^-16.  Values of 4
bits are exact in bf16.  fp32 terms are F = 2e-5 of the absolute sums (scores below 10
in sum |q||k| scale, off by some 8 * 2^-23 of that, and the sums).  So o is within
(2^-16 + F) a of the oracle, a = sum p |v|, before it is rounded, and E = 2^-8 of itself
after.  Against 16-bit pages that is all.

Scores from 4-bit keys with bf16 queries: the weight of every second value,
w = q0 - q1 / 16, is rounded to fp16, 2^-11 of it at most, and reaches the score as that
part of w k0; some 64 such errors of either sign: 6 standard deviations of their
sum, each evenly spread.  The offset of 1024 (1160 at most with the codes' own) makes
the fp32 sums over 32 values 1160 steps sum |w| large: 4 roundings of 2^-24 each.
fp32 queries are multiplied as fp32 numbers: F alone.
"""
import numpy as np
import pytest
import torch

import gated_delta_rule_bwd_gb300 as gdn
from oracle import attention as at
from tests.test_attn_paged import random_cache, seen
from tests.test_attn_paged_weights import compare, scored
from tests.test_kv_cache import i32, np64, tables

gpu = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
E, F, TERMS = 2.0 ** -8, 2e-5, 2.0 ** -16


def oracle(q, cache, table, lens, page, scale):
    """o and a = sum p |v| of every row in fp64."""
    B, T, H, D = q.shape
    G = H // cache[0].shape[2]
    o, a = np.zeros(q.shape), np.zeros(q.shape)
    q = np64(q)
    for b, n in enumerate(lens):
        if n >= 0:
            k, v = seen(cache, table, b, n + T, page)
            for h in range(H):
                o[b, :, h], _, a[b, :, h] = at.attn_fwd(q[b, :, h], k[:, h // G], v[:, h // G], scale)
    return o, a


def setting(lens, T, H, Hkv, D, page, dtype, bits, seed):
    table, pages = tables([max(n, 0) + T for n in lens], page, seed)
    q = torch.randn(len(lens), T, H, D, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()
    return q, random_cache(pages, page, Hkv, D, dtype, bits, seed + 1), table


@gpu
@pytest.mark.parametrize("dtype,bits", [(BF16, None), (F32, None), (F32, 4)], ids=["bf16", "f32", "f32-4"])
@pytest.mark.parametrize("H,Hkv,D", [(8, 2, 128), (4, 4, 64), (6, 1, 96), (40, 1, 64), (16, 1, 128)])
@pytest.mark.parametrize("T", [1, 3])
@pytest.mark.parametrize("page", [16, 64])
def test_elements(page, T, H, Hkv, D, dtype, bits):
    lens = [0, 1, 62, 63, 64, 130, 700, 3000, -1]
    q, cache, table = setting(lens, T, H, Hkv, D, page, dtype, bits, 41 + D + T)
    o, a = oracle(q, cache, table, lens, page, D ** -0.5)
    got = np64(gdn.attn_paged(q, cache, table, i32(lens)))
    assert gdn.device_status() == 0
    bound = (TERMS + F) * a + E * np.abs(o) if dtype == BF16 else F * (a + np.sqrt(np.mean(o * o)))
    assert np.all(np.abs(got - o) <= bound), np.max(np.abs(got - o) / (bound + 1e-30))


@gpu
@pytest.mark.parametrize("bits", [None, 4])
@pytest.mark.parametrize("H,D", [(4, 128), (4, 64), (16, 128), (16, 64), (40, 128)])
@pytest.mark.parametrize("n,page", [(1, 16), (33, 16), (700, 16), (3000, 64)])
def test_values(n, page, H, D, bits):
    """Scores that both caches hold exactly, of 24 sizes."""
    r = np.random.default_rng(n + D)
    scores = r.choice([0.0] + [s * c * 2.0 ** -x for s in (1, -1) for c in (5, 6, 7) for x in (1, 2, 3, 6)], n)
    cache, table, q, _ = scored(scores, H, D, page, bits, 42)
    compare(q, cache, table, n, page)


@gpu
@pytest.mark.parametrize("D", [64, 128])
def test_scores_in_4_bits(D):
    """Two keys with values of 1 and -1: o = tanh of half the difference of their scores,
    which is near 0 for some, where the output's rounding hides nothing."""
    B, H, Hkv, page = 128, 16, 4, 16
    q, cache, table = setting([1] * B, 1, H, Hkv, D, page, BF16, 4, 43)
    first = table[:, 0].long()
    for n, code in ((0, 12), (1, 4)):  # 4 and -4, in steps of 1 / 4
        cache[1][first, n] = code | code << 4
    cache[3].fill_(0.25)
    got = np64(gdn.attn_paged(q, cache, table, i32([1] * B)))[:, 0, :, 0]
    assert gdn.device_status() == 0
    near = 0
    for b in range(B):
        k, _ = seen(cache, table, b, 2, page)
        step = np.repeat(np64(cache[2][first[b], :2]), 32, -1)
        for h in range(H):
            x, kh, sh = np64(q)[b, 0, h], k[:, h // (H // Hkv)], step[:, h // (H // Hkv)]
            ref = np.tanh((kh[0] - kh[1]) @ x * D ** -0.5 / 2)
            w = x[0::2] - x[1::2] / 16
            off = 6 * np.sqrt(np.sum((2.0 ** -11 * w * kh[:, 0::2]) ** 2, -1) / 3)
            off += 4 * 2.0 ** -24 * 1160 * np.sum((np.abs(w) + np.abs(x[1::2]) / 16) * sh[:, 0::2], -1)
            bound = E * abs(ref) + TERMS + F + off.sum() * D ** -0.5 / 2
            assert abs(got[b, h] - ref) <= bound, (b, h, got[b, h], ref, bound)
            near += abs(ref) < 0.05
    assert near > 20


def excess(got, o):
    """The error over that of the oracle's result rounded to bf16."""
    rounded = np64(torch.tensor(o).to(BF16))
    return np.linalg.norm(got - o) / np.linalg.norm(rounded - o)


@gpu
@pytest.mark.parametrize("bits", [None, 4])
@pytest.mark.parametrize("D", [64, 128])
def test_on_the_whole(D, bits):
    """What stands beside the output's rounding (about 1.6e-3 of the result) adds 5 % to its
    error at most: a third of it, as of independent errors.  Two terms leave 1e-5, the
    scores of 4-bit keys about 2e-4; one bf16 term would add a third."""
    lens, page = [700, 3000, 100, 1500], 64
    q, cache, table = setting(lens, 1, 16, 4, D, page, BF16, bits, 44)
    o, _ = oracle(q, cache, table, lens, page, D ** -0.5)
    got = np64(gdn.attn_paged(q, cache, table, i32(lens)))
    assert gdn.device_status() == 0
    assert excess(got, o) <= 1.05


def test_one_term_would_fail():
    """The oracle with probabilities rounded to bf16 once, as a kernel that fed
    only that to its products, is outside both bounds."""
    r = np.random.default_rng(45)
    n, D, H = 700, 64, 16
    k, v = r.standard_normal((n, D)), r.standard_normal((n, D))
    k, v = (np64(torch.tensor(x).to(BF16)) for x in (k, v))
    q = np64(torch.tensor(r.standard_normal((H, D))).to(BF16))
    s = q @ k.T * D ** -0.5
    p = np.exp(s - s.max(-1, keepdims=True))
    total = p.sum(-1, keepdims=True)
    o, a = p @ v / total, p @ np.abs(v) / total
    for terms, good in ((1, False), (2, True)):
        hi = np64(torch.tensor(p).to(BF16))
        w = hi if terms == 1 else hi + np64(torch.tensor(p - hi).to(BF16))
        got = np64(torch.tensor(w @ v / total).to(BF16))
        assert bool(np.all(np.abs(got - o) <= (TERMS + F) * a + E * np.abs(o))) is good
        assert bool(excess(got, o) <= 1.05) is good
