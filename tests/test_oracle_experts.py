"""Pins of the expert oracle: every gradient against central differences of its
own forward definition, the gate's order, ties and masks by hand, and the
activations' values at points known in closed form."""

import numpy as np
import pytest

from oracle import experts as OE

H = 1e-6


def _difference(f, x):
    """d f / d x by central differences (f returns a scalar)."""
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        keep = x[i]
        x[i] = keep + H
        hi = f()
        x[i] = keep - H
        lo = f()
        x[i] = keep
        g[i] = (hi - lo) / (2 * H)
    return g


# A difference's error: H^2 times a third derivative of order 10, and 2^-53
# times sums of order 100 over H.
TOL = 100 * 2.0 ** -53 / H * 10


@pytest.mark.parametrize("name", OE.ACTIVATIONS)
def test_activation_slope(name):
    x = np.array([-6.0, -1.3, -0.2, 0.4, 1.0, 5.5])
    want = (OE.act(name, x + H) - OE.act(name, x - H)) / (2 * H)
    assert np.allclose(OE.act_grad(name, x), want, rtol=0, atol=TOL)


def test_activation_values():
    assert OE.act("silu", np.array([0.0]))[0] == 0.0
    assert np.isclose(OE.act("gelu", np.array([1.0]))[0], 0.8413447460685429, rtol=1e-15)
    assert np.isclose(OE.act("silu", np.array([np.log(3.0)]))[0], 0.75 * np.log(3.0), rtol=1e-15)
    t = np.tanh(np.sqrt(2 / np.pi) * 1.044715)
    assert np.isclose(OE.act("gelu_tanh", np.array([1.0]))[0], 0.5 * (1 + t), rtol=1e-15)


@pytest.mark.parametrize("name", ["none", "silu", "gelu", "gelu_tanh"])
def test_product_gradients(name):
    rng = np.random.default_rng(3)
    off = [1, 3, 3, 6]
    x, w, u = rng.standard_normal((7, 4)), rng.standard_normal((3, 5, 4)), rng.standard_normal((3, 5, 4))
    b, d = rng.standard_normal((3, 5)), rng.standard_normal((7, 5))
    at = slice(1, 6)

    def lin():
        return (OE.linear(x, off, w, b, name)[0][at] * d[at]).sum()

    d_x, d_w, d_b = OE.linear_grad(d, x, off, w, OE.linear(x, off, w, b, name)[1], name)
    assert np.allclose(d_x[at], _difference(lin, x)[at], rtol=0, atol=TOL)
    assert np.allclose(d_w, _difference(lin, w), rtol=0, atol=TOL)
    assert np.allclose(d_b, _difference(lin, b), rtol=0, atol=TOL)
    assert not d_w[1].any() and not d_b[1].any()

    def gat():
        return (OE.gated(x, off, w, u, name)[0][at] * d[at]).sum()

    _, g, up = OE.gated(x, off, w, u, name)
    d_x, d_g, d_u = OE.gated_grad(d, x, off, w, u, g, up, name)
    for got, at_ in ((d_g, w), (d_u, u)):
        assert np.allclose(got, _difference(gat, at_), rtol=0, atol=TOL)
    assert np.allclose(d_x[at], _difference(gat, x)[at], rtol=0, atol=TOL)


def test_gate_order_and_masks():
    inf = np.inf
    l = np.array([[1.0, 2.0, 2.0, 0.0], [-inf, 3.0, -inf, 3.0], [-inf] * 4, [-inf, -inf, 5.0, -inf]])
    idx, w = OE.gate(l, 3)
    assert idx.tolist() == [[1, 2, 0], [1, 3, 0], [0, 1, 2], [2, 0, 1]]
    assert w[1].tolist() == [0.5, 0.5, 0.0] and not w[2].any() and w[3].tolist() == [1.0, 0.0, 0.0]
    assert np.isclose(w[0, 0], np.e ** 2 / (1 + np.e + 2 * np.e ** 2))
    _, wr = OE.gate(l, 3, True)
    assert np.isclose(wr[0].sum(), 1.0) and not wr[2].any()


@pytest.mark.parametrize("renorm", [False, True])
def test_gate_gradient(renorm):
    rng = np.random.default_rng(4)
    l = rng.standard_normal((5, 6))
    idx, _ = OE.gate(l, 3)
    d = rng.standard_normal((5, 3))

    def f():
        p = np.take_along_axis(OE.softmax(l), idx, axis=1)
        return ((p / p.sum(axis=1, keepdims=True) if renorm else p) * d).sum()

    assert np.allclose(OE.gate_grad(l, idx, d, renorm), _difference(f, l), rtol=0, atol=TOL)
    l[0] = -np.inf
    l[1, 2:] = -np.inf
    idx, _ = OE.gate(l, 3)
    g = OE.gate_grad(l, idx, d, renorm)
    assert not g[0].any() and not g[1, 2:].any() and np.isfinite(g).all()


def test_combine_gradient():
    rng = np.random.default_rng(5)
    T, k, h = 4, 2, 3
    slot = rng.permutation(T * k).reshape(T, k)
    z, w, d = rng.standard_normal((T * k, h)), rng.standard_normal((T, k)), rng.standard_normal((T, h))

    def f():
        return ((w[:, :, None] * z[slot]).sum(axis=1) * d).sum()

    d_z, d_w = OE.combine_grad(d, z, slot, w)
    assert np.allclose(d_z, _difference(f, z), rtol=0, atol=TOL)
    assert np.allclose(d_w, _difference(f, w), rtol=0, atol=TOL)
