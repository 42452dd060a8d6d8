"""Pins of the fp64 oracle of the layer operators: values worked out by hand."""
import math

import numpy as np

from oracle import layer


def test_norm_by_hand():
    # h = (3, 4): mean of squares 12.5
    y, h = layer.rmsnorm_residual(np.array([[1.0, 5.0]]), np.array([2.0, 1.0]), np.array([[2.0, -1.0]]), eps=0.0)
    assert np.array_equal(h, [[3.0, 4.0]])
    assert np.allclose(y, [[6.0 / math.sqrt(12.5), 4.0 / math.sqrt(12.5)]], rtol=1e-15)
    # eps inside the root: h = (0, 0) gives 0, and eps = 12.5 doubles the mean
    assert np.array_equal(layer.rmsnorm_residual(np.zeros((1, 2)), np.ones(2))[0], [[0.0, 0.0]])
    y, _ = layer.rmsnorm_residual(np.array([[3.0, 4.0]]), np.ones(2), eps=12.5)
    assert np.allclose(y, [[0.6, 0.8]], rtol=1e-15)


def test_row_scale_by_hand():
    assert np.array_equal(layer.row_scale(np.array([[-896.0, 1.0], [0.0, 0.0]])), [2.0, 1e-30 / 448.0])
    assert np.isnan(layer.row_scale(np.array([[np.nan, 1.0]])))[0]


def test_linear_by_hand():
    x, w = np.array([[1.0, 2.0]]), np.array([[3.0, -1.0], [0.5, -4.0]])   # [K, N]
    assert np.array_equal(layer.linear(x, w), [[4.0, -9.0]])
    assert np.array_equal(layer.linear(x, w.T, layout="nk"), [[4.0, -9.0]])
    assert np.array_equal(layer.linear(x, w, bias=[1.0, 1.0], residual=[[10.0, 20.0]], act="relu"), [[15.0, 20.0]])
    assert np.array_equal(layer.linear(x, w, x_scale=[2.0], weight_scale=[0.5, 1.0]), [[4.0, -18.0]])
    assert np.array_equal(layer.linear(x, w, gated=True), [[4.0 * -9.0]])
    a, s = layer.affine(x, w, bias=[-1.0, 0.0])
    assert np.array_equal(a, [[3.0, -9.0]]) and np.array_equal(s, [[5.0, 9.0]])


def test_activations_by_hand():
    v = np.array([-1.0, 0.0, 2.0])
    e = math.e
    assert np.allclose(layer.activation("silu", v), [-1 / (1 + e), 0.0, 2 / (1 + e ** -2)], rtol=1e-15)
    # erf(1 / sqrt 2) = 0.6826894921370859 (the normal distribution within one deviation)
    assert np.allclose(layer.activation("gelu", np.array([-1.0, 1.0])), [-0.5 * (1 - 0.6826894921370859),
                                                                        0.5 * (1 + 0.6826894921370859)], rtol=1e-14)
    assert np.array_equal(layer.activation("relu", v), [0.0, 0.0, 2.0])
    assert np.isnan(layer.activation("relu", np.array([np.nan])))[0]
    assert layer.activation("silu", np.array([-1e4]))[0] == 0.0
