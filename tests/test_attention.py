"""attn_fwd, attn_bwd and attn_decode against the fp64 oracle, element by element.

The oracle sees the same bytes (bf16 values upcast).  Bounds, with e = 2^-8 for
bf16 (half a step, relative) and the oracle's sums of absolute terms:

* fp32 inputs: everything is fp32.  An exponential's argument (below about 20)
  is off by a few 2^-24 of itself, so a probability by a few 1e-6 of itself,
  and a sum of n terms adds at most about sqrt(n) 2^-24 of their absolute sum:
  2e-5 of the absolute sum.  ds = p (dp - delta) is a difference of two such
  sums (it is 0 in exact arithmetic where a query sees one key), so the
  absolute sums of dp and of delta count for dq and dk.
* bf16 inputs: a probability that feeds the tensor cores is off by e of itself
  and the result is rounded once, so o is within e (a + |o|), a = sum p |v|;
  dv within e (sum p |do| + |dv|).  delta = do . o is made from the rounded o:
  it is off by at most d = sum |do| e (a + |o|) (and the fp32 2e-5), so ds by p d, and ds is
  rounded once more: dq within e (sum |ds||k| + |dq|) + d sum p |k|, dk the
  same with the rows' own d.  The fp32 terms above come on top.
* lse is fp32 in both: 2e-5.
"""
import ctypes

import numpy as np
import pytest
import torch

import gated_delta_rule_bwd_gb300 as gdn
from oracle import attention as at

gpu = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
E = 2.0 ** -8
F = 2e-5


def np64(t):
    return t.detach().double().cpu().numpy()


def inputs(B, tq, tk, H, Hkv, D, dtype, seed=0, fused=False, device="cuda"):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g).to(dtype)  # noqa: E731
    if fused:  # q, k, v as views of one projection
        q, k, v = r(B, tq, H + 2 * Hkv, D).to(device).split([H, Hkv, Hkv], dim=2)
    else:
        q, k, v = (x.to(device) for x in (r(B, tq, H, D), r(B, tk, Hkv, D), r(B, tk, Hkv, D)))
    return q, k, v, r(B, tq, H, D).to(device)


def reference(q, k, v, do, lq, lk, scale, bf16):
    """Oracle outputs and bounds; lq, lk the lengths of the row's sequences."""
    q, k, v, do = map(np64, (q, k, v, do))
    B, tq, H, D = q.shape
    Hkv = k.shape[2]
    G = H // Hkv
    ref = {"o": np.zeros_like(q), "lse": np.zeros((B, H, tq)), "dq": np.zeros_like(q),
           "dk": np.zeros_like(k), "dv": np.zeros_like(v)}
    bound = {n: np.zeros_like(x) for n, x in ref.items()}
    e = E if bf16 else 0.0
    for b in range(B):
        q0 = k0 = 0
        for n, m in zip(lq, lk):
            iq, ik = slice(q0, q0 + n), slice(k0, k0 + m)
            q0, k0 = q0 + n, k0 + m
            for h in range(H):
                a = q[b, iq, h], k[b, ik, h // G], v[b, ik, h // G]
                o, lse, av = at.attn_fwd(*a, scale)
                dq, dk, dv, ab = at.attn_bwd(*a, do[b, iq, h], scale)
                ref["o"][b, iq, h], ref["lse"][b, h, iq], ref["dq"][b, iq, h] = o, lse, dq
                ref["dk"][b, ik, h // G] += dk
                ref["dv"][b, ik, h // G] += dv
                d = (np.abs(do[b, iq, h]) * (e + F) * (av + np.abs(o))).sum(1)
                bound["o"][b, iq, h] = (e + F) * av
                bound["dq"][b, iq, h] = (e + F) * ab["dq"] + d[:, None] * ab["pk"] + F * ab["cq"]
                bound["dk"][b, ik, h // G] += (e + F) * ab["dk"] + ab["pq"](d) + F * ab["ck"]
                bound["dv"][b, ik, h // G] += (e + F) * ab["dv"]
    for n, x in ref.items():
        if n == "lse":
            bound[n] = F * (1 + np.abs(np.where(np.isfinite(x), x, 0)))
        elif x.size:
            bound[n] += e * np.abs(x) + F * np.sqrt(np.mean(x * x))
    return ref, bound


def check(got, ref, bound):
    for n, x in got.items():
        x, r = np64(x), ref[n]
        assert x.shape == r.shape, (n, x.shape, r.shape)
        if not r.size:
            continue
        inf = ~np.isfinite(r)
        assert np.array_equal(x[inf], r[inf]), f"{n}: other non-finite values"
        assert np.all(np.isfinite(x[~inf])), f"{n}: non-finite values"
        err = np.abs(np.where(inf, 0, x) - np.where(inf, 0, r)) - bound[n]
        i = np.unravel_index(np.argmax(err), err.shape)
        assert err[i] <= 0, f"{n}: {x[i]:.6e} for {r[i]:.6e} at {i}, bound {bound[n][i]:.2e}"


def cu(lengths):
    return torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32, device="cuda")


def run(q, k, v, do, lq=None, lk=None, scale=None):
    c = {} if lq is None else {"cu_seqlens": cu(lq)}
    if lk is not None and lk != lq:
        c["cu_seqlens_k"] = cu(lk)
    o, lse = gdn.attn_fwd(q, k, v, scale=scale, **c)
    dq, dk, dv = gdn.attn_bwd(q, k, v, o, lse, do, scale=scale, **c)
    assert gdn.device_status() == 0
    return {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv}


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("H,Hkv,D", [(2, 2, 128), (4, 1, 64), (6, 2, 80), (2, 1, 33), (1, 1, 1), (3, 3, 8)])
@pytest.mark.parametrize("T", [1, 2, 63, 64, 65, 127, 128, 129, 300])
def test_one_length(T, H, Hkv, D, dtype):
    q, k, v, do = inputs(2, T, T, H, Hkv, D, dtype, seed=T)
    ref, bound = reference(q, k, v, do, [T], [T], D ** -0.5, dtype == BF16)
    check(run(q, k, v, do), ref, bound)


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("lq,lk", [([5, 61, 33], None), ([1, 0, 257, 3, 128], None),
                                   ([0, 0, 7], None), ([17, 130, 1], [300, 130, 513]),
                                   ([9, 200, 40], [4, 0, 150]), ([0, 3], [70, 3]), ([1] * 40, None)])
@pytest.mark.parametrize("H,Hkv,D,fused", [(4, 2, 128, True), (2, 1, 64, False), (4, 1, 96, True)])
def test_packed(lq, lk, H, Hkv, D, fused, dtype):
    """Empty sequences, rows without keys (fewer keys than queries), keys from
    before, sequences that start and end inside a tile."""
    fused = fused and lk is None
    q, k, v, do = inputs(1, sum(lq), sum(lk or lq), H, Hkv, D, dtype, seed=len(lq), fused=fused)
    ref, bound = reference(q, k, v, do, lq, lk or lq, D ** -0.5, dtype == BF16)
    check(run(q, k, v, do, lq, lk), ref, bound)


@gpu
@pytest.mark.parametrize("lq,lk,H,Hkv,D", [
    ([1], [4100], 2, 1, 128), ([70], [2050], 3, 3, 64), ([260], [3000], 2, 2, 80),
    ([1400], [1400], 1, 1, 128), ([300], [2500], 4, 1, 96),
    ([5, 130, 0, 2], [1500, 131, 70, 6000], 2, 1, 128), ([3000, 40], [1400, 40], 1, 1, 64)])
def test_few_queries_and_many_keys(lq, lk, H, Hkv, D):
    """Keys in parts that are joined: parts without keys for some rows, for a
    whole short sequence, and rows that see no key in any part."""
    q, k, v, do = inputs(1, sum(lq), sum(lk), H, Hkv, D, BF16, seed=len(lq))
    s, *_, nseq = gdn._attn_args(q, k, v, cu(lq), cu(lk), None)
    assert gdn.lib().gdn_attn_fwd_workspace(ctypes.byref(s), nseq) > 0
    ref, bound = reference(q, k, v, do, lq, lk, D ** -0.5, True)
    got = run(q, k, v, do, *((lq, lk) if len(lq) > 1 else ()))
    check(got, ref, bound)
    # another packed sequence's NaN reaches no row
    for bad, rows in ((slice(lk[0]), slice(lq[0], None)), (slice(-lk[-1], None), slice(-lq[-1]))):
        if len(lq) > 1:
            k2, v2 = k.clone(), v.clone()
            k2[:, bad] = v2[:, bad] = float("nan")
            o, lse = gdn.attn_fwd(q, k2, v2, cu(lq), cu(lk))
            assert torch.equal(o[:, rows], got["o"][:, rows])
            assert torch.equal(lse[:, :, rows], got["lse"][:, :, rows])


@gpu
@pytest.mark.parametrize("dtype,D", [(F32, 64), (F32, 72), (BF16, 65)], ids=["f32", "f32-72", "bf16-65"])
def test_more_jobs_than_fit(dtype, D):
    """CUDA-core kernels with whole jobs to a CTA (shorter calls share them)."""
    q, k, v, do = inputs(6, 200, 200, 16, 16, D, dtype)
    ref, bound = reference(q, k, v, do, [200], [200], D ** -0.5, dtype == BF16)
    check(run(q, k, v, do), ref, bound)


@gpu
def test_batch_rows_in_groups():
    """Batches of many rows go out in groups of rows, the last one smaller."""
    q, k, v, do = inputs(19, 300, 300, 16, 16, 64, BF16)
    ref, bound = reference(q, k, v, do, [300], [300], 64 ** -0.5, True)
    check(run(q, k, v, do), ref, bound)


@gpu
def test_workspace_of_parts():
    """A workspace that is too small or missing is refused before a launch."""
    q, k, v, _ = inputs(1, 64, 4096, 2, 2, 128, BF16)
    s, scale, *_ = gdn._attn_args(q, k, v, None, None, None)
    L, need = gdn.lib(), gdn.lib().gdn_attn_fwd_workspace(ctypes.byref(s), 0)
    o, lse = torch.empty_like(q), torch.empty(1, 2, 64, device="cuda")
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    call = lambda ptr, n: L.gdn_attn_fwd(  # noqa: E731
        ctypes.byref(s), q.data_ptr(), k.data_ptr(), v.data_ptr(), scale, None, None, 0,
        o.data_ptr(), lse.data_ptr(), ptr, n, None)
    assert call(None, need) == -5 and call(ws.data_ptr(), need - 1) == -5
    given, given_lse = gdn.attn_fwd(q, k, v, workspace=ws)
    own, own_lse = gdn.attn_fwd(q, k, v)
    assert torch.equal(given, own) and torch.equal(given_lse, own_lse)


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("Tq,Tk", [(1, 700), (130, 1), (64, 0), (0, 5), (200, 460)])
def test_other_numbers_of_keys(Tq, Tk, dtype):
    q, k, v, do = inputs(2, Tq, Tk, 4, 2, 64, dtype, seed=Tq)
    ref, bound = reference(q, k, v, do, [Tq], [Tk], 0.2, dtype == BF16)
    check(run(q, k, v, do, scale=0.2), ref, bound)


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_long_and_large_scores(dtype):
    """Many tiles, and scores up to about 300: the running maximum moves.  Such
    an argument is off by a few 300 2^-24 of itself, some 1e-4 of a probability:
    relative L2 3e-4 per output (bf16 inputs: the mixers' bar, 2e-2)."""
    q, k, v, do = inputs(1, 1500, 1500, 2, 1, 128, dtype, seed=3)
    q, k = q * 8, k * 8
    ref, _ = reference(q, k, v, do, [1500], [1500], 128 ** -0.5, dtype == BF16)
    for n, x in run(q, k, v, do).items():
        err = np.linalg.norm(np64(x) - ref[n]) / np.linalg.norm(ref[n])
        assert err <= (2e-2 if dtype == BF16 else 3e-4), (n, err)


@gpu
@pytest.mark.parametrize("layout", ["heads_first", "sliced_tokens", "expanded", "odd_base", "reversed_batch"])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_strides(layout, dtype):
    T, H, D = 150, 2, 64
    q, k, v, do = inputs(2, T, T, H, H, D, dtype, seed=11)
    if layout == "heads_first":  # [B, H, T, D] memory
        q, k, v = (x.transpose(1, 2).contiguous().transpose(1, 2) for x in (q, k, v))
    elif layout == "sliced_tokens":
        q, k, v = (torch.cat([x, x], 1)[:, 7:7 + T] for x in (q, k, v))
    elif layout == "expanded":  # one key head seen as two
        k, v = k[:, :, :1].expand(2, T, H, D), v[:, :, :1].expand(2, T, H, D)
    elif layout == "odd_base":  # rows that start between 16-byte boundaries
        wide = lambda x: torch.cat([x[..., :1], x, x[..., :2]], -1)[..., 1:1 + D]  # noqa: E731
        q, k, v = map(wide, (q, k, v))
    else:
        q, k, v = (x.repeat(2, 1, 1, 1)[::2] for x in (q, k, v))
    ref, bound = reference(q, k, v, do, [T], [T], D ** -0.5, dtype == BF16)
    check(run(q, k, v, do), ref, bound)


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_other_sequences_do_not_reach_in(dtype):
    """NaN and infinities in one packed sequence change no other's values."""
    lq = [70, 45, 200]
    q, k, v, do = inputs(1, sum(lq), sum(lq), 4, 2, 64, dtype, seed=5)
    clean = run(q, k, v, do, lq)
    bad = [x.clone() for x in (q, k, v, do)]
    for x, y in zip(bad, (float("nan"), float("inf"), float("nan"), float("-inf"))):
        x[:, 70:115] = y
    got = run(*bad, lq)
    for n in clean:
        for sl in (slice(0, 70), slice(115, None)):
            a, b = (clean[n][..., sl], got[n][..., sl]) if n == "lse" else (clean[n][:, sl], got[n][:, sl])
            assert torch.equal(a, b), n


@gpu
def test_same_bits_every_time_and_on_another_stream():
    lq = [700, 1, 333]
    q, k, v, do = inputs(1, sum(lq), sum(lq), 8, 2, 128, BF16, seed=6, fused=True)
    a = run(q, k, v, do, lq)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        b = run(q, k, v, do, lq)
    st.synchronize()
    for n in a:
        assert torch.equal(a[n], b[n]), n


@gpu
def test_in_a_graph():
    q, k, v, do = inputs(1, 260, 260, 4, 2, 128, BF16, seed=7)
    want = run(q, k, v, do)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        o, lse = gdn.attn_fwd(q, k, v)
        dq, dk, dv = gdn.attn_bwd(q, k, v, o, lse, do)
    for x in (o, lse, dq, dk, dv):
        x.zero_()
    g.replay()
    torch.cuda.synchronize()
    for n, x in (("o", o), ("lse", lse), ("dq", dq), ("dk", dk), ("dv", dv)):
        assert torch.equal(x, want[n]), n


@gpu
def test_autograd_and_differences():
    q, k, v, do = inputs(1, 37, 37, 2, 1, 16, F32, seed=8)
    x = [t.requires_grad_() for t in (q, k, v)]
    (gdn.attention(*x) * do).sum().backward()
    loss = lambda *y: float((np64(gdn.attn_fwd(*y)[0]) * np64(do)).sum())  # noqa: E731
    r = np.random.default_rng(0)
    with torch.no_grad():
        for i, t in enumerate(x):
            d = torch.tensor(r.normal(size=t.shape), dtype=F32, device="cuda")
            h = 1e-2
            y = [u.clone() for u in x]
            y[i] = t + h * d
            up = loss(*y)
            y[i] = t - h * d
            num, ana = (up - loss(*y)) / (2 * h), float((t.grad.double() * d.double()).sum())
            # h^2 / 6 times a third derivative of order |ana| + the fp32 loss's own error / h
            assert abs(num - ana) <= 1e-3 * (abs(ana) + np64(do).std() * np.sqrt(do.numel())), (i, num, ana)


@gpu
def test_bad_offsets_are_reported():
    q, k, v, do = inputs(1, 100, 100, 2, 2, 64, BF16, seed=9)
    for c in ([0, 60, 40, 100], [0, 50, 99], [3, 100], [0, 1000000, 100], [0, -70000, 100]):
        gdn.attn_fwd(q, k, v, cu_seqlens=torch.tensor(c, dtype=torch.int32, device="cuda"))
        assert gdn.device_status() == -8, c
        assert gdn.device_status() == 0


# ------------------------------------------------------------------ decode

def decode_reference(q, k, v, kc, vc, lens, scale, bf16):
    q, k, v, kc, vc = map(np64, (q, k, v, kc, vc))
    B, T, H, D = q.shape
    G = H // k.shape[2]
    ref, bound = np.zeros_like(q), np.zeros_like(q)
    for b, n in enumerate(lens):
        for h in range(H):
            kk = np.concatenate([kc[b, :n, h // G], k[b, :, h // G]])
            vv = np.concatenate([vc[b, :n, h // G], v[b, :, h // G]])
            o, _, a = at.attn_fwd(q[b, :, h], kk, vv, scale)
            ref[b, :, h], bound[b, :, h] = o, ((E if bf16 else 0) + F) * a
    return ref, bound + (E if bf16 else 0) * np.abs(ref) + F * np.sqrt(np.mean(ref * ref))


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("H,Hkv,D", [(8, 2, 128), (4, 4, 64), (6, 1, 80), (2, 1, 33), (32, 1, 128), (2, 2, 8)])
@pytest.mark.parametrize("T", [1, 3])
@pytest.mark.parametrize("S", [8, 129, 2000])
def test_decode(S, T, H, Hkv, D, dtype):
    """Empty and full rows; slots past a row's end hold NaN and are not read."""
    lens = [0, S - T, S // 2, 1]
    q, k, v, _ = inputs(4, T, T, H, Hkv, D, dtype, seed=S + T)
    _, kc, vc, _ = inputs(4, 1, S, H, Hkv, D, dtype, seed=S + T + 1)
    for b, n in enumerate(lens):
        kc[b, n:], vc[b, n:] = float("nan"), float("inf")
    want_k, want_v = kc.clone(), vc.clone()
    for b, n in enumerate(lens):
        want_k[b, n:n + T], want_v[b, n:n + T] = k[b], v[b]
    ref, bound = decode_reference(q, k, v, kc, vc, lens, D ** -0.5, dtype == BF16)
    o = gdn.attn_decode(q, k, v, kc, vc, torch.tensor(lens, dtype=torch.int32, device="cuda"))
    assert gdn.device_status() == 0
    check({"o": o}, {"o": ref}, {"o": bound})
    for got, want in ((kc, want_k), (vc, want_v)):
        assert torch.equal(got.nan_to_num(nan=123.0), want.nan_to_num(nan=123.0))


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_decode_strided_cache_and_long_row(dtype):
    """Caches as views of one [B, Hkv, S, 2 D] buffer; a row of many parts."""
    B, T, S, H, Hkv, D = 1, 2, 20000, 4, 2, 64
    q, k, v, _ = inputs(B, T, T, H, Hkv, D, dtype, seed=21)
    buf = torch.randn(B, Hkv, S, 2 * D, generator=torch.Generator().manual_seed(3)).to(dtype).cuda()
    kc, vc = buf[..., :D].transpose(1, 2), buf[..., D:].transpose(1, 2)
    ref, bound = decode_reference(q, k, v, kc, vc, [19000], 0.1, dtype == BF16)
    lens = torch.tensor([19000], dtype=torch.int32, device="cuda")
    o = gdn.attn_decode(q, k, v, kc, vc, lens, scale=0.1)
    check({"o": o}, {"o": ref}, {"o": bound})
    assert torch.equal(kc[:, 19000:19002], k) and torch.equal(vc[:, 19000:19002], v)
    assert gdn.device_status() == 0


@gpu
def test_decode_continues_a_prompt():
    """Token by token from an empty cache equals the prompt's attention."""
    T, H, Hkv, D = 40, 4, 2, 128
    q, k, v, do = inputs(2, T, T, H, Hkv, D, BF16, seed=31)
    ref, bound = reference(q, k, v, do, [T], [T], D ** -0.5, True)
    kc, vc = (torch.empty(2, 64, Hkv, D, dtype=BF16, device="cuda") for _ in range(2))
    lens = torch.zeros(2, dtype=torch.int32, device="cuda")
    out = []
    for t in range(T):
        sl = slice(t, t + 1)
        out.append(gdn.attn_decode(q[:, sl].contiguous(), k[:, sl].contiguous(), v[:, sl].contiguous(),
                                   kc, vc, lens))
        lens += 1
    check({"o": torch.cat(out, 1)}, ref, bound)


@gpu
def test_decode_bad_lengths_are_reported():
    q, k, v, _ = inputs(3, 2, 2, 2, 1, 64, BF16, seed=41)
    kc, vc = (torch.ones(3, 10, 1, 64, dtype=BF16, device="cuda") for _ in range(2))
    want = kc.clone()
    want[1, 4:6] = k[1]
    o = gdn.attn_decode(q, k, v, kc, vc, torch.tensor([9, 4, -1], dtype=torch.int32, device="cuda"))
    assert gdn.device_status() == -8 and gdn.device_status() == 0
    assert not o[0].any() and not o[2].any() and o[1].any()
    assert torch.equal(kc, want)


# ------------------------------------------------------------------ refusals (host side)

FAKE = ctypes.c_void_p(0x10000)  # never dereferenced


def attn_shape(B=1, Tq=8, Tk=8, H=2, Hkv=1, D=16, dtype=1, qs=(256, 32, 16), ks=(128, 16, 16)):
    return gdn.AttnShape(B, Tq, Tk, H, Hkv, D, dtype, qs, ks, ks)


def call_fwd(s, q=FAKE, k=FAKE, v=FAKE, scale=0.5, cq=None, ck=None, nseq=0, o=FAKE, lse=FAKE):
    return gdn.lib().gdn_attn_fwd(ctypes.byref(s), q, k, v, scale, cq, ck, nseq, o, lse, None, 0, None)


def test_attention_refusals():
    ARG, SHAPE, DTYPE, ALIGN, WS = -1, -2, -3, -4, -5
    for kw in (dict(D=0), dict(D=129), dict(H=3, Hkv=2), dict(Hkv=0), dict(B=-1), dict(Tq=-1),
               dict(H=70000, Hkv=1), dict(qs=(256, -32, 16)), dict(B=1 << 20, Tq=1 << 20)):
        assert call_fwd(attn_shape(**kw)) == SHAPE, kw
    assert call_fwd(attn_shape(dtype=2)) == DTYPE
    for x in (0.0, -1.0, float("nan"), float("inf")):
        assert call_fwd(attn_shape(), scale=x) == ARG
    for n in ("q", "k", "v", "o", "lse"):
        assert call_fwd(attn_shape(), **{n: None}) == ARG
    assert call_fwd(attn_shape(), cq=FAKE) == ARG
    assert call_fwd(attn_shape(B=2), cq=FAKE, ck=FAKE, nseq=1) == SHAPE
    assert call_fwd(attn_shape(), cq=FAKE, ck=FAKE, nseq=0) == SHAPE
    assert call_fwd(attn_shape(), cq=ctypes.c_void_p(0x10002), ck=FAKE, nseq=1) == ALIGN
    assert call_fwd(attn_shape(), q=ctypes.c_void_p(0x10001)) == ALIGN
    assert call_fwd(attn_shape(), o=ctypes.c_void_p(0x10008)) == ALIGN
    assert call_fwd(attn_shape(B=0), q=None, k=None, v=None, o=None, lse=None) == 0
    assert gdn.lib().gdn_attn_fwd(None, FAKE, FAKE, FAKE, 0.5, None, None, 0, FAKE, FAKE, None, 0, None) == ARG
    s = attn_shape()
    need = gdn.lib().gdn_attn_bwd_workspace(ctypes.byref(s), 0)
    assert need >= 8 * 2 * 4
    bwd = lambda ws, n, dk=FAKE: gdn.lib().gdn_attn_bwd(  # noqa: E731
        ctypes.byref(s), FAKE, FAKE, FAKE, 0.5, None, None, 0, FAKE, FAKE, FAKE, FAKE, dk, FAKE, ws, n, None)
    assert bwd(None, 0) == WS and bwd(FAKE, need - 1) == WS and bwd(FAKE, need, None) == ARG


def test_decode_refusals():
    mk = lambda B=1, T=1, S=8, H=2, Hkv=1, D=16, dtype=1, st=(128, 16, 16): gdn.AttnDecodeShape(  # noqa: E731
        B, T, S, H, Hkv, D, dtype, st, st)

    def call(s, q=FAKE, kc=FAKE, lens=FAKE, scale=0.5, o=FAKE):
        return gdn.lib().gdn_attn_decode(ctypes.byref(s), q, FAKE, FAKE, kc, FAKE, lens, scale, o, None, 0, None)
    for kw in (dict(D=0), dict(D=200), dict(H=3, Hkv=2), dict(T=9), dict(T=-1), dict(B=40000, Hkv=2),
               dict(st=(-1, 16, 16)), dict(S=(1 << 30) + 1)):
        assert call(mk(**kw)) == -2, kw
    assert call(mk(dtype=5)) == -3
    assert call(mk(), scale=0.0) == -1 and call(mk(), lens=None) == -1 and call(mk(), o=None) == -1
    assert call(mk(), q=ctypes.c_void_p(0x10008)) == -4 and call(mk(), kc=ctypes.c_void_p(0x10001)) == -4
    assert call(mk(S=100000, D=128)) == -5
    assert call(mk(B=0), q=None) == 0 and call(mk(T=0), q=None) == 0


def test_binding_refuses_cpu_tensors():
    q = torch.zeros(1, 4, 2, 16)
    with pytest.raises(gdn.GdnError):
        gdn.attn_fwd(q, q, q)
    with pytest.raises(gdn.GdnError):
        gdn.attn_decode(q, q, q, q, q, torch.zeros(1, dtype=torch.int32))
    with pytest.raises(gdn.GdnError):
        gdn.attn_fwd(q.long(), q, q)


@gpu
def test_binding_refusals():
    z = lambda *s, dt=BF16: torch.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
    q, k = z(1, 4, 2, 16), z(1, 4, 1, 16)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    for call in (lambda: gdn.attn_fwd(q, k, z(1, 5, 1, 16)),
                 lambda: gdn.attn_fwd(q, k.float(), k),
                 lambda: gdn.attn_fwd(z(1, 4, 3, 16), z(1, 4, 2, 16), z(1, 4, 2, 16)),
                 lambda: gdn.attn_fwd(q, z(1, 4, 1, 8), z(1, 4, 1, 8)),
                 lambda: gdn.attn_fwd(q.transpose(2, 3).contiguous().transpose(2, 3), k, k),
                 lambda: gdn.attn_fwd(q, z(1, 9, 1, 16), z(1, 9, 1, 16), cu_seqlens=i32(0, 4)),
                 lambda: gdn.attn_fwd(q, k, k, cu_seqlens=i32(0, 4).long()),
                 lambda: gdn.attn_fwd(q, k, k, cu_seqlens_k=i32(0, 4)),
                 lambda: gdn.attn_fwd(q, k, k, cu_seqlens=i32(0, 4), cu_seqlens_k=i32(0, 2, 4)),
                 lambda: gdn.attn_fwd(q, k, k, scale=-1.0),
                 lambda: gdn.attn_bwd(q, k, k, q, z(1, 2, 4, dt=F32), z(1, 4, 1, 16)),
                 lambda: gdn.attn_bwd(q, k, k, q, z(1, 2, 3, dt=F32), q),
                 lambda: gdn.attn_decode(q, k, k, z(1, 8, 1, 16), z(1, 9, 1, 16), i32(0)),
                 lambda: gdn.attn_decode(q, k, k, z(1, 8, 1, 16), z(1, 8, 1, 16), i32(0, 0)),
                 lambda: gdn.attn_decode(q, k, k, z(1, 3, 1, 16), z(1, 3, 1, 16), i32(0))):
        with pytest.raises(gdn.GdnError):
            call()
    assert gdn.device_status() == 0
