"""The oracle of norm, rotation and 4-bit storage, pinned: differences, complex
numbers, hand-made values."""
import numpy as np
import pytest

from oracle import paging as pg


def tables(n, R):
    a = np.arange(n)[:, None] * 100.0 ** (-np.arange(0, R, 2) / max(R, 1))
    return np.cos(a), np.sin(a)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,R", [(8, 8), (9, 4), (6, 6), (3, 2)])
def test_rotation_is_a_complex_product(D, R, interleaved):
    x = np.random.default_rng(0).normal(size=(5, D))
    cos, sin = tables(5, R)
    a, b = pg.pairs(R, interleaved)
    z = (x[:, a] + 1j * x[:, b]) * (cos + 1j * sin)
    y = pg.rotate(x, cos, sin, interleaved)
    assert np.allclose(y[:, a], z.real) and np.allclose(y[:, b], z.imag)
    assert np.array_equal(y[:, R:], x[:, R:])
    assert np.allclose(pg.rotate(y, cos, -sin, interleaved), x)


def test_pairs():
    assert [list(p) for p in pg.pairs(6, False)] == [[0, 1, 2], [3, 4, 5]]
    assert [list(p) for p in pg.pairs(6, True)] == [[0, 2, 4], [1, 3, 5]]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_gradient_against_differences(norm, interleaved):
    r = np.random.default_rng(1)
    x, dy, w = r.normal(size=(4, 3, 10)), r.normal(size=(4, 3, 10)), r.normal(size=10)
    cos, sin = (t[:, None] for t in tables(4, 6))
    f = lambda x, w: np.sum(dy * pg.norm_rope(x, w if norm else None, cos, sin, 1e-3, interleaved))  # noqa: E731
    dx, dw, ax, aw = pg.norm_rope_bwd(x, w if norm else None, cos, sin, dy, 1e-3, interleaved)
    assert np.all(np.abs(dx) <= ax + 1e-12)
    h = 1e-5
    d = r.normal(size=x.shape)
    assert abs((f(x + h * d, w) - f(x - h * d, w)) / (2 * h) - np.sum(dx * d)) < 1e-7
    if norm:
        e = r.normal(size=10)
        assert abs((f(x, w + h * e) - f(x, w - h * e)) / (2 * h) - np.sum(dw * e)) < 1e-7
        assert np.all(np.abs(dw) <= aw + 1e-12)


def test_steps_have_five_bits():
    for a, s in ((7.0, 1.0), (7 * 1.03125, 1.0625), (7 * 1.03, 1.0), (7 * 31 / 16, 31 / 16), (0.0, 0.0),
                 (7 * 31.5 / 16, 2.0)):
        assert pg.step_of(np.array(a)) == s, a
    a = np.exp(np.random.default_rng(2).uniform(-20, 20, 1000))
    s = pg.step_of(a)
    m, _ = np.frexp(s)
    assert np.array_equal(m * 32, np.rint(m * 32))
    assert np.all(np.abs(s - a / 7) <= a / 7 * 2 ** -5)
    assert np.all(a - 7 * s <= 0.5 * s)  # the largest value stays within half a step of code 7


def test_codes():
    x = np.zeros((1, 64))
    x[0, :6] = [7, 0.5, 1.5, -2.5, -7, 3.4999]
    n, s = pg.quantise(x)
    assert list(s[0]) == [1, 0] and list(n[0, :6]) == [7, 0, 2, -2, -7, 3] and not n[0, 6:].any()
    codes = (n.astype(np.uint8) + 8).reshape(1, 32, 2)
    back = pg.values((codes[..., 0] | codes[..., 1] << 4).astype(np.uint8), s)
    assert np.array_equal(back, n * np.repeat(s, 32, -1))
