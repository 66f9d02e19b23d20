"""Pins of the float64 oracles of the query / key norm with rotation and of linear attention
(CPU): closed forms, invariances, and every gradient against central differences."""
import numpy as np
import pytest

from oracle import linear as OL
from oracle import qknorm as OQ


def _rng(seed=0):
    return np.random.default_rng(seed)


def test_norm_closed_forms():
    x = np.full((2, 1, 8), 3.0)
    assert np.allclose(OQ.forward(x, eps=0.0), 1.0)
    assert np.allclose(OQ.forward(x, eps=7.0), 3.0 / 4.0)
    assert np.allclose(OQ.forward(np.zeros((1, 1, 8))), 0.0)
    assert np.allclose(OQ.forward(x, norm=False), 3.0)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_keeps_lengths_and_relative_positions(interleaved):
    r = _rng(1)
    inv = 100.0 ** (-np.arange(3) / 3)
    q, k = r.normal(size=(2, 1, 1, 8))
    at = lambda x, p: OQ.rotate(x[None], OQ.angles([[p]], inv, [3]), interleaved)[0]
    assert np.allclose(np.sum(at(q, 5) ** 2), np.sum(q ** 2))
    assert np.allclose(at(q, 5)[..., 6:], q[..., 6:])  # behind the rotated values
    # a product of rotated vectors goes by the distance of their positions
    assert np.allclose(np.sum(at(q, 5) * at(k, 2)), np.sum(at(q, 105) * at(k, 102)))
    assert np.allclose(OQ.rotate(at(q, 9)[None], OQ.angles([[9]], inv, [3]), interleaved, -1.0)[0], q)


def test_rotation_quarter_turn_places():
    x = np.arange(1.0, 9.0)[None, None]
    ang = np.full((1, 2), np.pi / 2)
    assert np.allclose(OQ.rotate(x, ang, False), [[[-3, -4, 1, 2, 5, 6, 7, 8]]])
    assert np.allclose(OQ.rotate(x, ang, True), [[[-2, 1, -4, 3, 5, 6, 7, 8]]])


def test_axes_of_pairs():
    ang = OQ.angles(np.array([[1], [10], [100]]), np.array([1.0, 2.0, 3.0, 4.0]), [1, 2, 1])
    assert np.allclose(ang, [[1, 20, 30, 400]])


@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("interleaved", [False, True])
def test_norm_gradient_against_differences(norm, interleaved):
    r = _rng(2)
    x, dy, w = r.normal(size=(3, 2, 8)), r.normal(size=(3, 2, 8)), r.normal(size=8)
    ang = r.normal(size=(3, 3))
    f = lambda x, w: np.sum(dy * OQ.forward(x, w, 1e-2, ang, interleaved, norm))
    dx, dw = OQ.backward(x, dy, w, 1e-2, ang, interleaved, norm)
    e = 1e-6
    for i in np.ndindex(x.shape):
        d = np.zeros_like(x)
        d[i] = e
        assert abs((f(x + d, w) - f(x - d, w)) / (2 * e) - dx[i]) < 1e-7
    for i in range(8):
        d = np.zeros(8)
        d[i] = e
        assert abs((f(x, w + d) - f(x, w - d)) / (2 * e) - dw[i]) < 1e-7


def test_linear_closed_forms():
    r = _rng(3)
    q, k, v = r.normal(size=(3, 6, 2, 4))
    # lambda = 0: each token sees itself alone
    o, s = OL.forward(q, k, v, [-np.inf, -np.inf], 2.0)
    assert np.allclose(o, 2.0 * np.sum(q * k, -1, keepdims=True) * v)
    assert np.allclose(s, k[-1][:, :, None] * v[-1][:, None, :])
    # lambda = 1: prefix sums; above 0 counts as 0
    o, s = OL.forward(q, k, v, [0.0, 0.7], 1.0)
    a = np.einsum("ihd,jhd->hij", q, k) * np.tril(np.ones((6, 6)))
    assert np.allclose(o, np.einsum("hij,jhd->ihd", a, v))
    assert np.allclose(s, np.einsum("nhi,nhj->hij", k, v))
    # no tokens: the state passes
    s0 = r.normal(size=(2, 4, 4))
    assert np.allclose(OL.forward(q[:0], k[:0], v[:0], [-1.0, -1.0], 1.0, s0)[1], s0)


def test_linear_splits_anywhere():
    r = _rng(4)
    q, k, v = r.normal(size=(3, 9, 2, 4))
    g = [-0.3, -1.0]
    o, s = OL.forward(q, k, v, g, 0.5)
    a, s1 = OL.forward(q[:4], k[:4], v[:4], g, 0.5)
    b, s2 = OL.forward(q[4:], k[4:], v[4:], g, 0.5, s1)
    assert np.allclose(np.concatenate([a, b]), o) and np.allclose(s2, s)


def test_linear_gradient_against_differences():
    r = _rng(5)
    n, H, d = 5, 2, 3
    x = dict(zip("qkv", r.normal(size=(3, n, H, d))))
    x["s"] = r.normal(size=(H, d, d))
    do, e = r.normal(size=(n, H, d)), r.normal(size=(H, d, d))
    g = [-0.2, -1.5]

    def loss(x):
        o, s = OL.forward(x["q"], x["k"], x["v"], g, 0.7, x["s"])
        return np.sum(do * o) + np.sum(e * s)

    grads = dict(zip("qkvs", OL.backward(x["q"], x["k"], x["v"], do, g, 0.7, x["s"], e)))
    for name, grad in grads.items():
        for i in np.ndindex(grad.shape):
            d1, d2 = dict(x), dict(x)
            d1[name], d2[name] = x[name].copy(), x[name].copy()
            d1[name][i] += 1e-6
            d2[name][i] -= 1e-6
            assert abs((loss(d1) - loss(d2)) / 2e-6 - grad[i]) < 1e-6
