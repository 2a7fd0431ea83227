"""Pins of the feed-forward oracle (CPU): the activations against closed
values and their derivatives against differences, the layer's gradient
against differences of a loss, the experts' layer against a dense sum, the
routing's ties, and the clipping rule."""

import math

import numpy as np
import pytest

import oracle

KINDS = ("none", "relu", "gelu", "gelu_tanh", "silu")


def test_activations_at_known_points():
    z = np.array([-1.0, 0.0, 1.0, 2.0])
    assert np.array_equal(oracle.act(z, "relu"), [0, 0, 1, 2])
    phi1 = 0.8413447460685429  # the normal distribution's value at 1
    assert np.allclose(oracle.act(z, "gelu")[[0, 2]], [-(1 - phi1), phi1], atol=1e-15)
    assert np.allclose(oracle.act(z, "silu"), [z_ / (1 + math.exp(-z_)) for z_ in z], atol=1e-15)
    # the tanh form stays within 5e-4 of the error function's
    g = np.linspace(-6, 6, 1001)
    assert np.abs(oracle.act(g, "gelu_tanh") - oracle.act(g, "gelu")).max() < 5e-4


@pytest.mark.parametrize("kind", KINDS)
def test_derivatives_against_differences(kind):
    z = np.linspace(-5.03, 5.03, 400)  # no point within h of 0, where relu has its corner
    h = 1e-5
    d = (oracle.act(z + h, kind) - oracle.act(z - h, kind)) / (2 * h)
    assert np.abs(d - oracle.act_grad(z, kind)).max() < 1e-9


@pytest.mark.parametrize("kind", KINDS)
def test_layer_gradient_against_differences(kind):
    """loss = sum(c * (act(a @ b + bias) + residual)), a = act(z_in)."""
    r = np.random.RandomState(1)
    m, n, k = 5, 7, 6
    z_in, b, bias, res, c = (r.randn(*s) for s in ((m, k), (k, n), (n,), (m, n), (m, n)))

    def loss(z_in, b, bias):
        return float((c * oracle.gemm_epilogue(oracle.act(z_in, kind), b, bias, res, kind)[0]).sum())

    a = oracle.act(z_in, kind)
    _, z = oracle.gemm_epilogue(a, b, bias, res, kind)
    da, db, dbias = oracle.gemm_epilogue_grad(c * oracle.act_grad(z, kind), a, b, z_in, kind)
    h = 1e-6
    for grad, at in ((da, 0), (db, 1), (dbias, 2)):
        d = r.randn(*grad.shape)
        args = [z_in, b, bias]
        up, dn = list(args), list(args)
        up[at], dn[at] = args[at] + h * d, args[at] - h * d
        assert abs((loss(*up) - loss(*dn)) / (2 * h) - float((grad * d).sum())) < 1e-6 * (1 + np.abs(grad).sum())


def test_gradient_accumulates():
    r = np.random.RandomState(2)
    dz, a, b = r.randn(4, 3), r.randn(4, 2), r.randn(2, 3)
    _, db, dbias = oracle.gemm_epilogue_grad(dz, a, b)
    _, db2, dbias2 = oracle.gemm_epilogue_grad(dz, a, b, db_in=db, dbias_in=dbias)
    assert np.allclose(db2, 2 * db) and np.allclose(dbias2, 2 * dbias)


def test_route_ties_and_gates():
    ids, gates = oracle.route(np.array([[1.0, 3.0, 3.0, 0.0]]), 3, True)
    assert ids.tolist() == [[1, 2, 0]]
    assert math.isclose(gates.sum(), 1.0) and gates[0, 0] == gates[0, 1]
    _, full = oracle.route(np.array([[1.0, 3.0, 3.0, 0.0]]), 3, False)
    assert full.sum() < 1.0 and np.allclose(full / full.sum(), gates)


def test_moe_layer_against_a_dense_sum():
    r = np.random.RandomState(3)
    T, H, I, E, K = 4, 6, 5, 3, 2
    x, w1, w2 = r.randn(T, H), r.randn(E, H, 2 * I), r.randn(E, I, H)
    ids, gates = oracle.route(r.randn(T, E), K, True)
    got = oracle.moe_layer(x, ids, gates, w1, w2, "silu", True)
    g = np.zeros((T, E))
    np.put_along_axis(g, ids, gates, axis=1)
    u = np.einsum("th,ehn->ten", x, w1)
    y = np.einsum("tei,eih->teh", oracle.act(u[..., :I], "silu") * u[..., I:], w2)
    assert np.allclose(got, (g[..., None] * y).sum(axis=1))
    # an id that names no expert, and an id that stands twice
    ids2 = np.array(ids)
    ids2[:, 1] = ids2[:, 0]
    twice = oracle.moe_layer(x, ids2, gates, w1, w2)
    ids2[:, 1] = -1
    once = oracle.moe_layer(x, ids2, gates, w1, w2)
    assert np.allclose(twice, once / gates[:, :1])


def test_clip_rule():
    norm, out = oracle.grad_norm_clip([np.array([3.0]), np.array([[4.0]])], 1.0)
    assert norm == 5.0 and abs(out[0][0] - 0.6) < 1e-6
    _, same = oracle.grad_norm_clip([np.array([3.0])], math.inf)
    assert same[0][0] == 3.0
    _, same = oracle.grad_norm_clip([np.array([3.0])], 7.0)
    assert same[0][0] == 3.0


def test_planted_mistakes_are_seen():
    """A derivative taken at the output, a transposed weight gradient and a
    gate left out all move the results."""
    r = np.random.RandomState(4)
    z = r.randn(8)
    assert np.abs(oracle.act_grad(oracle.act(z, "silu"), "silu") - oracle.act_grad(z, "silu")).max() > 1e-2
    dz, a, b = r.randn(4, 3), r.randn(4, 3), r.randn(3, 3)
    assert np.abs(oracle.gemm_epilogue_grad(dz, a, b)[1].T - oracle.gemm_epilogue_grad(dz, a, b)[1]).max() > 1e-2
    x, w1, w2 = r.randn(2, 4), r.randn(2, 4, 3), r.randn(2, 3, 4)
    ids, gates = oracle.route(r.randn(2, 2), 2, True)
    plain = oracle.moe_layer(x, ids, np.ones_like(gates), w1, w2, "relu", False)
    assert np.abs(plain - oracle.moe_layer(x, ids, gates, w1, w2, "relu", False)).max() > 1e-3
