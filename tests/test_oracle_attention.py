"""Pins of the fp64 attention and layer-norm oracle: closed forms, torch's
autograd in fp64, and central differences.  CPU only."""
import numpy as np
import pytest
import torch

from oracle import attention as at


def rand(*shape, seed=0):
    return np.random.default_rng(seed).normal(size=shape)


@pytest.mark.parametrize("lq,lk", [(1, 1), (5, 5), (3, 7), (6, 2), (4, 0), (0, 3)])
def test_attention_against_autograd(lq, lk):
    D, scale = 6, 0.37
    q, k, v, do = rand(lq, D, seed=1), rand(lk, D, seed=2), rand(lk, D, seed=3), rand(lq, D, seed=4)
    o, lse, _ = at.attn_fwd(q, k, v, scale)
    dq, dk, dv, _ = at.attn_bwd(q, k, v, do, scale)
    tq, tk, tv = (torch.tensor(x, requires_grad=True) for x in (q, k, v))
    rows = []
    for i in range(lq):  # the rows that see a key, one by one
        n = i + lk - lq + 1
        rows.append(torch.softmax(scale * tk[:n] @ tq[i], 0) @ tv[:n] if n > 0
                    else torch.zeros(D, dtype=torch.float64))
        if n > 0:
            z = torch.logsumexp(scale * tk[:n] @ tq[i], 0).item()
            assert abs(lse[i] - z) < 1e-12
        else:
            assert lse[i] == -np.inf and not o[i].any()
    if lq == 0:
        assert not dk.any() and not dv.any()
        return
    y = torch.stack(rows)
    assert np.allclose(y.detach().numpy(), o, atol=1e-12)
    if not y.requires_grad:
        assert not dq.any()
        return
    for g, r in zip(torch.autograd.grad(y, (tq, tk, tv), torch.tensor(do)), (dq, dk, dv)):
        assert np.allclose(g.numpy(), r, atol=1e-12)


def test_attention_gradients_against_differences():
    lq, lk, D, scale, h = 3, 5, 4, 0.5, 1e-5
    x = {"q": rand(lq, D, seed=1), "k": rand(lk, D, seed=2), "v": rand(lk, D, seed=3)}
    do = rand(lq, D, seed=4)
    loss = lambda y: float((at.attn_fwd(y["q"], y["k"], y["v"], scale)[0] * do).sum())  # noqa: E731
    for n, g in zip("qkv", at.attn_bwd(x["q"], x["k"], x["v"], do, scale)[:3]):
        for i in np.ndindex(g.shape):
            up, dn = dict(x), dict(x)
            up[n], dn[n] = x[n].copy(), x[n].copy()
            up[n][i] += h
            dn[n][i] -= h
            assert abs((loss(up) - loss(dn)) / (2 * h) - g[i]) < 1e-8


def test_uniform_scores_average_the_values():
    v = rand(4, 3, seed=5)
    o, lse, _ = at.attn_fwd(np.zeros((4, 3)), rand(4, 3), v, 1.0)
    for i in range(4):
        assert np.allclose(o[i], v[:i + 1].mean(0)) and np.isclose(lse[i], np.log(i + 1))


@pytest.mark.parametrize("n,D", [(1, 1), (3, 7), (5, 16)])
def test_layer_norm_against_torch(n, D):
    x, w, b, dy = rand(n, D, seed=1), 1 + rand(D, seed=2), rand(D, seed=3), rand(n, D, seed=4)
    y, mean, rstd = at.layer_norm_fwd(x, w, b, 1e-3)
    t = [torch.tensor(a, requires_grad=True) for a in (x, w, b)]
    z = torch.nn.functional.layer_norm(t[0], (D,), t[1], t[2], 1e-3)
    assert np.allclose(z.detach().numpy(), y, atol=1e-12)
    assert np.allclose(mean, x.mean(1)) and np.allclose(rstd, (x.var(1) + 1e-3) ** -0.5)
    for g, r in zip(torch.autograd.grad(z, t, torch.tensor(dy)), at.layer_norm_bwd(x, w, dy, 1e-3)):
        assert np.allclose(g.numpy(), r, atol=1e-10)
