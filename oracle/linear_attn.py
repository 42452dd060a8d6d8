"""fp64 oracle of linear attention with a decay for each head and of rotary positions.  Numpy; shares no code
with the CUDA library."""
from __future__ import annotations

import numpy as np

from . import _as_f64


def recurrence(q, k, v, g_log, scale, state=None, lengths=None):
    """``(out, state, size)`` of S_t = e^{g_t} S_{t-1} + k_t v_t^T, o_t = scale S_t^T q_t, token by token.

    q, k [B, Hk, S, Dk], v [B, Hv, S, Dv], g_log [B, Hv, S] or [Hv]; rows behind a sequence's length are zeros in out.
    ``size`` is what roundings are measured by: ``(out_mag, mag, out_acc, acc)``, with mag the recurrence over the
    magnitudes |state|, |k|, |v| (and |q| for out_mag), and acc that of mag itself, acc_t = e^{g_t} acc_{t-1} + mag_t: a relative
    error of u at every token adds up to u acc."""
    q, k, v, g = (_as_f64(x) for x in (q, k, v, g_log))
    B, Hk, S, Dk = q.shape
    Hv, Dv = v.shape[1], v.shape[3]
    q, k = (np.repeat(x, Hv // Hk, axis=1) for x in (q, k))
    a = np.exp(g) if g.ndim == 3 else np.broadcast_to(np.exp(g)[None, :, None], (B, Hv, S))
    st = np.zeros((B, Hv, Dk, Dv)) if state is None else _as_f64(state).copy()
    mag = np.abs(st)
    acc = np.zeros_like(mag)
    out, out_mag, out_acc = (np.zeros((B, Hv, S, Dv)) for _ in range(3))
    n = np.full(B, S) if lengths is None else np.clip(np.asarray(lengths), 0, S)
    keep = lambda f, x: np.where(f == 0, 0, f * x)  # noqa: E731  (a decay of zero drops infinities too)
    for t in range(S):
        at = n > t
        f = a[at, :, t, None, None]
        kv, qt = k[at, :, t, :, None] * v[at, :, t, None, :], q[at, :, t, None, :]
        st[at] = keep(f, st[at]) + kv
        mag[at] = keep(f, mag[at]) + np.abs(kv)
        acc[at] = keep(f, acc[at]) + mag[at]
        out[at, :, t] = scale * (qt @ st[at])[:, :, 0]
        out_mag[at, :, t] = abs(scale) * (np.abs(qt) @ mag[at])[:, :, 0]
        out_acc[at, :, t] = abs(scale) * (np.abs(qt) @ acc[at])[:, :, 0]
    return out, st, (out_mag, mag, out_acc, acc)


def _inverse_2pi(bits):
    """1 / (2 pi) in units of 2^-bits, from Machin's pi/4 = 4 arctan(1/5) - arctan(1/239) in whole numbers."""
    one = 1 << (bits + 32)

    def arctan_of_inverse(n):
        total, term, k = 0, one // n, 0
        while term:
            total += (-term if k & 1 else term) // (2 * k + 1)
            term //= n * n
            k += 1
        return total
    pi = 4 * (4 * arctan_of_inverse(5) - arctan_of_inverse(239))
    return (one << bits) // (2 * pi)


_BITS = 192
_INV_2PI = _inverse_2pi(_BITS)


def _turned(positions, inv_freq):
    """positions * inv_freq (radians) less its whole turns, in [-pi, pi): the product as whole numbers, exactly."""
    steps = []
    for f in np.asarray(inv_freq, dtype=np.float64).ravel():
        n, d = float(f).as_integer_ratio()
        steps.append((n * _INV_2PI) // d)  # turns a position in units of 2^-192
    half, whole = 1 << (_BITS - 1), 1 << _BITS
    flat = [int(p) for p in np.asarray(positions).ravel()]
    turns = [[((p * s + half) % whole - half) / whole for s in steps] for p in flat]
    return 2 * np.pi * np.array(turns).reshape(np.shape(positions) + (len(steps),))


def rotary(x, inv_freq, positions, layout="half", amplitude=1.0, inverse=False):
    """x [B, H, S, D] with its first 2 len(inv_freq) channels turned; positions [B, S] or [S]."""
    y, R = _as_f64(x).copy(), 2 * len(inv_freq)
    theta = _turned(positions, inv_freq) * (-1 if inverse else 1)
    theta = theta[None, None] if theta.ndim == 2 else theta[:, None]
    c, s = amplitude * np.cos(theta), amplitude * np.sin(theta)
    if layout == "half":
        ia, ib = np.arange(R // 2), np.arange(R // 2) + R // 2
    else:
        ia, ib = np.arange(0, R, 2), np.arange(1, R, 2)
    a, b = y[..., ia].copy(), y[..., ib].copy()
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    return y
