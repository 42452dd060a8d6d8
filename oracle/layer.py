"""fp64 oracle of the layer operators around the decode block: the norm behind the residual's
addition and the matrix product with its epilogue.  Numpy; shares no code with the CUDA library."""
from __future__ import annotations

import numpy as np

from . import _as_f64

E4M3_MAX = 448.0
AMAX_MIN = 1e-30


def rmsnorm_residual(x, weight, residual=None, eps=1e-6):
    """``(y, h)`` over the last dimension: h = x + residual, y = h / sqrt(mean(h^2) + eps) * weight."""
    h = _as_f64(x)
    if residual is not None:
        h = h + _as_f64(residual)
    return h / np.sqrt(np.mean(h * h, axis=-1, keepdims=True) + eps) * _as_f64(weight), h


def row_scale(y):
    """The 8-bit scale of every row: max(max |y|, AMAX_MIN) / 448 (NaN where the row has one)."""
    return np.maximum(np.abs(y).max(axis=-1), AMAX_MIN) / E4M3_MAX


def _erf(v):
    import math
    return np.vectorize(math.erf, otypes=[np.float64])(v)


def activation(name, v):
    if name == "silu":
        with np.errstate(over="ignore"):
            return v / (1.0 + np.exp(-v))
    if name == "gelu":
        return 0.5 * v * (1.0 + _erf(v / np.sqrt(2.0)))
    if name == "relu":
        return np.where(v < 0, 0.0, v)
    return v


def affine(x, weight, bias=None, x_scale=None, weight_scale=None, layout="kn"):
    """``(a, s)``: the scaled and biased products [M, N'], and the sums of their terms' magnitudes
    (what the rounding of a sum is measured by)."""
    x, w = _as_f64(x), _as_f64(weight)
    w = w.T if layout == "nk" else w
    a, s = x @ w, np.abs(x) @ np.abs(w)
    if x_scale is not None:
        f = _as_f64(x_scale)[:, None] * _as_f64(weight_scale)[None, :]
        a, s = a * f, s * np.abs(f)
    if bias is not None:
        b = _as_f64(bias)
        a, s = a + b, s + np.abs(b)
    return a, s


def linear(x, weight, bias=None, residual=None, act="none", x_scale=None, weight_scale=None, layout="kn", gated=False):
    """``act(x W + bias) + residual``, or gated: ``act(first half) * second half + residual``."""
    a, _ = affine(x, weight, bias, x_scale, weight_scale, layout)
    if gated:
        n = a.shape[1] // 2
        y = activation(act, a[:, :n]) * a[:, n:]
    else:
        y = activation(act, a)
    return y if residual is None else y + _as_f64(residual)
