"""Pins of the float64 oracle of the operators ahead of the head: values by hand, gradients against
central differences, the e4m3 grid against its definition."""
import math

import numpy as np
import pytest

from oracle import layers as L


def _diff(f, x, step=1e-6):
    """Central differences of a scalar function, element by element."""
    g = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        a, b = x.copy(), x.copy()
        a[i] += step
        b[i] -= step
        g[i] = (f(a) - f(b)) / (2 * step)
    return g


def test_rmsnorm_by_hand():
    h, y = L.rmsnorm(np.array([[3.0, 4.0]]), None, np.array([1.0, 2.0]), 0.0)
    rms = math.sqrt(12.5)
    np.testing.assert_allclose(y, [[3.0 / rms, 8.0 / rms]], rtol=1e-15)
    h, y = L.rmsnorm(np.array([[1.0, 1.0]]), np.array([[1.0, -1.0]]), np.ones(2), 1.0)
    np.testing.assert_allclose(h, [[2.0, 0.0]])
    np.testing.assert_allclose(y, [[2.0 / math.sqrt(3.0), 0.0]], rtol=1e-15)


def test_rmsnorm_gradient_against_differences():
    rng = np.random.default_rng(1)
    x, r, g = rng.standard_normal((3, 8)), rng.standard_normal((3, 8)), 1 + 0.3 * rng.standard_normal(8)
    w, wh = rng.standard_normal((3, 8)), rng.standard_normal((3, 8))
    eps = 0.1

    def f(xv, gv):
        h, y = L.rmsnorm(xv, r, gv, eps)
        return (w * y).sum() + (wh * h).sum()
    dx, dg = L.rmsnorm_grad(w, x + r, g, eps, dh=wh)
    np.testing.assert_allclose(dx, _diff(lambda v: f(v, g), x), atol=1e-8)
    np.testing.assert_allclose(dg, _diff(lambda v: f(x, v), g), atol=1e-8)


def test_e4m3_grid():
    v = L.e4m3_values()
    assert v.max() == 448.0 and v.min() == -448.0 and np.abs(v[v != 0]).min() == 2.0 ** -9
    assert len(v) == 2 * 126 + 1
    q, s = L.e4m3_rows(np.array([[448.0, 17.0, 19.0, -0.5, 0.0], [0.0] * 5]))
    assert s.tolist() == [1.0, 0.0]
    # between 16 and 32 the step is 2: 17 and 19 lie half-way and go to the even mantissas 16 and 20
    assert q.tolist() == [[448.0, 16.0, 20.0, -0.5, 0.0], [0.0] * 5]


@pytest.mark.parametrize("kind", L.ACTIVATIONS)
def test_activation_gradient_against_differences(kind):
    z = np.linspace(-6, 6, 101) + 1e-3
    num = (L.act(z + 1e-5, kind) - L.act(z - 1e-5, kind)) / 2e-5
    np.testing.assert_allclose(L.act_grad(z, kind), num, atol=1e-8)


def test_activation_values():
    assert L.act(np.array([-1.0, 0.0, 2.0]), "relu").tolist() == [0.0, 0.0, 2.0]
    np.testing.assert_allclose(L.act(np.array([1.0]), "gelu"), 0.8413447460685429, rtol=1e-12)
    np.testing.assert_allclose(L.act(np.array([1.0]), "silu"), 1 / (1 + math.exp(-1)), rtol=1e-14)
    assert abs(L.act(np.array([1.0]), "gelu_tanh") - 0.8413447460685429) < 1e-3


@pytest.mark.parametrize("kind", L.ACTIVATIONS)
def test_linear_gradient_against_differences(kind):
    rng = np.random.default_rng(2)
    x, W, b = rng.standard_normal((3, 5)), rng.standard_normal((4, 5)), rng.standard_normal(4)
    r, w = rng.standard_normal((3, 4)), rng.standard_normal((3, 4))

    def f(xv, Wv, bv):
        return (w * L.linear(xv, Wv, bv, r, kind)[0]).sum()
    _, z = L.linear(x, W, b, r, kind)
    dx, dW, db, _ = L.linear_grad(w, z, x, W, kind)
    np.testing.assert_allclose(dx, _diff(lambda v: f(v, W, b), x), atol=1e-7)
    np.testing.assert_allclose(dW, _diff(lambda v: f(x, v, b), W), atol=1e-7)
    np.testing.assert_allclose(db, _diff(lambda v: f(x, W, v), b), atol=1e-7)
