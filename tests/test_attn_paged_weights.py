"""attn_paged where keys differ widely in weight and in size of value.

A probability meets its value in two bf16 terms, which leave 2^-16 of it, whatever
the other keys' are, and fp32 terms are F = 2e-5 of the absolute sums: o is within
(2^-16 + F) a of the oracle, a = sum p |v|, and half a step of bf16 (2^-8) of the
result.  The scores here are exact: one value of q is not 0, and keys hold their
code's multiple of a power of two (16-bit pages: such a value) against it.
"""
import numpy as np
import pytest
import torch

import gated_delta_rule_bwd_gb300 as gdn
from oracle import attention as at
from tests.test_attn_paged import random_cache, seen
from tests.test_kv_cache import i32, np64, places, tables

gpu = pytest.mark.gpu
BF16 = torch.bfloat16
E, F = 2.0 ** -8, 2e-5


def scored(scores, H, D, page, bits, seed):
    """A cache of one key head whose keys have these scores (a power of two times a
    code) for every row of q, and whose values are random; with its table, and where
    the keys lie."""
    n = len(scores)
    table, pages = tables([n], page, seed)
    cache = random_cache(pages, page, 1, D, BF16, bits, seed)
    at_ = tuple(torch.tensor(x, device="cuda").long() for x in places(np.zeros(n, int), np.arange(n), table, page))
    q = torch.zeros(1, 1, H, D, dtype=BF16, device="cuda")
    q[..., 0] = 8
    k0 = torch.tensor(np.asarray(scores) / 8, device="cuda")  # scale = 1
    if bits is None:
        k = cache[0][at_]
        k[:, 0, 0] = k0.to(BF16)
        cache[0][at_] = k
        return cache, table, q, at_
    code, step = torch.zeros_like(k0), torch.ones_like(k0)
    for c in (7, 6, 5):  # k0 = sign c 2^x
        x = k0.abs() / c
        hit = torch.frexp(x).mantissa == 0.5
        code[hit], step[hit] = (torch.sign(k0) * c)[hit], x[hit]
    assert torch.equal(code * step, k0)
    codes, steps = cache[0][at_], cache[2][at_]
    codes[:, 0, 0] = (codes[:, 0, 0] & 0xf0) | (code + 8).to(torch.uint8)
    steps[:, 0, 0] = step.to(BF16)
    cache[0][at_], cache[2][at_] = codes, steps
    return cache, table, q, at_


def compare(q, cache, table, n, page):
    """q [B, 1, H, D]: all rows of the batch are the same n keys."""
    B = q.shape[0]
    o = gdn.attn_paged(q, cache, table.expand(B, -1), i32([n - 1] * B), scale=1.0)
    assert gdn.device_status() == 0
    k, v = seen(cache, table, 0, n, page)
    for h in range(q.shape[2]):
        ref, _, a = at.attn_fwd(np64(q)[0, :, h], k[:, 0], v[:, 0], 1.0)
        got = np64(o)[:, 0, h]
        # weights below fp32's smallest normal number may be taken for 0: n of them at most
        over = np.abs(got - ref) - (2.0 ** -16 + F) * a - E * np.abs(ref) - n * 2.0 ** -126 * np.abs(v).max()
        assert over.max() <= 0, (h, over.max(), np.linalg.norm(got[0] - ref) / np.linalg.norm(ref))


@gpu
@pytest.mark.parametrize("bits", [None, 4])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B,H", [(1, 4), (150, 4), (150, 16)])
@pytest.mark.parametrize("far", [4, 16, 24])
@pytest.mark.parametrize("where", [64, 205, 1101])
def test_a_large_value_without_weight(where, far, B, H, D, bits):
    """8192 keys, one 10 above the rest in its score with a value of 0, and one whose value is
    2^far times the others' and whose score is 112 below theirs: it adds nothing.  Warps
    take every fourth 32 keys, so that the two are one warp's; with 150 rows it has some
    700 keys."""
    n, page = 8192, 64
    scores = np.zeros(n)
    scores[77], scores[where] = 10, -112
    cache, table, q, at_ = scored(scores, H, D, page, bits, 31)
    v = cache[1] if bits is None else cache[3]
    peak, big = tuple(x[77] for x in at_), tuple(x[where] for x in at_)
    v[peak] = 0
    v[big] = v[big] * 2.0 ** far
    compare(q.expand(B, -1, -1, -1).contiguous(), cache, table, n, page)


@gpu
@pytest.mark.parametrize("bits", [None, 4])
def test_rows_that_attend_to_different_sizes(bits):
    """One head attends to a value 2^30 times the others', the next seven to the rest."""
    n, page, D = 700, 16, 128
    scores = np.zeros(n)
    scores[300] = 112
    cache, table, q, at_ = scored(scores, 8, D, page, bits, 32)
    v = cache[1] if bits is None else cache[3]
    big = tuple(x[300] for x in at_)
    v[big] = v[big] * 2.0 ** 30
    q[0, 0, 1:] = -q[0, 0, 1:]
    compare(q, cache, table, n, page)


@gpu
@pytest.mark.parametrize("bits", [None, 4])
@pytest.mark.parametrize("T,H", [(3, 4), (3, 8), (40, 2)])
def test_a_large_value_of_a_later_token(T, H, bits):
    """New tokens before it do not see it: their results do not change by a bit."""
    D, page, n = 128, 16, 500
    table, pages = tables([n], page, 33)
    cache = random_cache(pages, page, 1, D, BF16, bits, 33)
    q = torch.randn(1, T, H, D, generator=torch.Generator().manual_seed(33)).to(BF16).cuda()
    lens = i32([n - T])
    before = gdn.attn_paged(q, cache, table, lens)
    at_ = tuple(int(x[0]) for x in places(np.array([0]), np.array([n - 1]), table, page))
    v = cache[1] if bits is None else cache[3]
    v[at_] = v[at_] * 2.0 ** 24
    after = gdn.attn_paged(q, cache, table, lens)
    assert gdn.device_status() == 0
    assert torch.equal(after[:, :-1], before[:, :-1]) and not torch.equal(after[:, -1], before[:, -1])
