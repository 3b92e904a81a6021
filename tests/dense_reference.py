"""Plain float64 forms of the layer's dense half (projections, RMS norm, gradient
clipping), with how far a float32 computation of them may be off.

Functions take and return numpy arrays; results are (reference, tolerance) pairs of the
same shape, the tolerance derived, not fitted, as in operator_reference.py: with u = 2^-24
a rounding is off by at most u of its result, a sum of n terms added in a chain by n u of
the sum of their magnitudes. The matrix instructions' own additions are counted twice
(2 u each), since their inner order and rounding are not written down.
"""
from __future__ import annotations

import numpy as np

from operator_reference import TINY, U, rounded

C0, C1 = 2 * np.sqrt(2 / np.pi), 0.044715
TOP = 448.0


def half_step(dtype):
    """Largest relative error of a rounding to the type."""
    return {'bf16': 2.0 ** -8, 'f32': U}[dtype]


# ---- activations -------------------------------------------------------------

def sigmoid(z):
    e = np.exp(-np.abs(z))
    return np.where(z < 0, e / (1 + e), 1 / (1 + e))


def sigmoid_slope(z):
    e = np.exp(-np.abs(z))
    return e / (1 + e) ** 2


def gelu_arg(z):
    return C0 * (z + C1 * z ** 3)


def act(name, z):
    if name == 'sigmoid':
        return sigmoid(z)
    if name == 'silu':
        return z * sigmoid(z)
    if name == 'gelu_tanh':
        return z * sigmoid(gelu_arg(z))
    return z


def slope(name, z):
    if name == 'sigmoid':
        return sigmoid_slope(z)
    if name == 'silu':
        return sigmoid(z) + z * sigmoid_slope(z)
    if name == 'gelu_tanh':
        u = gelu_arg(z)
        return sigmoid(u) + z * sigmoid_slope(u) * C0 * (1 + 3 * C1 * z * z)
    return np.ones_like(z)


def act_tol(name, z):
    """A float32 evaluation from an exact z: the exponential is off by one rounding of its argument a (|a| u
    of its value) and a few of its own, the rest by a few roundings of the value. gelu's argument itself
    takes five roundings."""
    if name == 'none':
        return 0.0
    a = np.abs(z) if name != 'gelu_tanh' else 6 * np.abs(gelu_arg(z))
    return np.abs(act(name, z)) * (a + 10) * 2 * U


def slope_tol(name, z):
    """As act_tol, for the magnitudes of the slope's terms (which are added)."""
    if name == 'none':
        return 0.0
    if name == 'sigmoid':
        return sigmoid_slope(z) * (np.abs(z) + 10) * 2 * U
    if name == 'silu':
        return (sigmoid(z) + np.abs(z) * sigmoid_slope(z)) * (np.abs(z) + 12) * 2 * U
    u = gelu_arg(z)
    # (beyond |z| = 16 the library takes 0 or 1: the terms left out are below 1e-60)
    return (sigmoid(u) + np.abs(z) * sigmoid_slope(u) * C0 * (1 + 3 * C1 * z * z)) * (6 * np.abs(u) + 14) * 2 * U


# ---- linear --------------------------------------------------------------------

def _eights(x, w):
    """What the 8-bit matrix instructions leave out. They add aligned eights of products with the bits down to
    2^-13 of the power of two of the largest (beside 2^16 and -2^16 in one of them 2^3 is kept and 2^2 is not;
    from one eight to the next all 24 bits are), so the other seven of an eight are each off by less than 2^-13
    of the largest, and that is at most the largest |x| times the largest |w| there."""
    k = -x.shape[1] % 8
    gx, gw = (np.abs(np.pad(t, ((0, 0), (0, k)))).reshape(len(t), -1, 8).max(-1) for t in (x, w))
    return 7 * 2.0 ** -13 * (gx @ gw.T)


def linear_fwd(x, w, bias=None, residual=None, activation='none', x_scale=None, w_scale=None, out_dtype='f32',
               z_dtype='f32'):
    """(y, tol), (z, tol)."""
    x, w = x.astype(np.float64), w.astype(np.float64)
    z, mag = x @ w.T, np.abs(x) @ np.abs(w).T
    if x_scale is not None:
        s = x_scale.astype(np.float64)[:, None] * w_scale.astype(np.float64)
        z, mag = z * s, mag * np.abs(s)
    tol = (x.shape[1] + 16) * 2 * U * mag
    if x_scale is not None:
        tol = tol + _eights(x, w) * np.abs(s)
    if bias is not None:
        z = z + bias.astype(np.float64)
        tol = tol + U * np.abs(bias)
    y = act(activation, z)
    # no activation here is steeper than 1.2
    ytol = 1.2 * tol + act_tol(activation, z)
    if residual is not None:
        y = y + residual.astype(np.float64)
        ytol = ytol + U * np.abs(residual)
    return (y, rounded(y, ytol, out_dtype)), (z, rounded(z, tol, z_dtype))


def linear_bwd(dy, x, w, z=None, activation='none', dtype='f32'):
    """{'x', 'weight', 'bias'}: (gradient, tol). dz is rounded to the operands' type for the products."""
    dy, x, w = (t.astype(np.float64) for t in (dy, x, w))
    s, st = (1.0, 0.0) if activation == 'none' else (slope(activation, z.astype(np.float64)),
                                                     slope_tol(activation, z.astype(np.float64)))
    dz = dy * s
    tz = np.abs(dy) * st + U * np.abs(dz)
    tr = tz + half_step(dtype) * np.abs(dz) + TINY if activation != 'none' else tz
    ax, aw, az = np.abs(x), np.abs(w), np.abs(dz)
    M, N = dy.shape
    out = {}
    for n, g, t, terms, mag in (('x', dz @ w, tr @ aw, N, az @ aw), ('weight', dz.T @ x, tr.T @ ax, M, az.T @ ax)):
        out[n] = (g, rounded(g, t + (terms + 16) * 2 * U * mag, dtype))
    out['bias'] = (dz.sum(0), tz.sum(0) + (M + 16) * U * az.sum(0) + TINY)
    return out


# ---- RMS norm -------------------------------------------------------------------

def _chain(cols):
    """Additions in a chain within a row: a lane's own elements, then the lanes."""
    return 48 + cols / 1024


def rms_norm_fwd(x, w, residual=None, eps=1e-5, out_dtype='f32', in_dtype='f32'):
    """(y, tol), (h, tol); e4m3: (q, tol), (scale, tol), (h, tol)."""
    h = x.astype(np.float64) + (0 if residual is None else residual.astype(np.float64))
    w = w.astype(np.float64)
    rstd = 1 / np.sqrt((h * h).mean(-1, keepdims=True) + eps)
    y = h * rstd * w
    # h, the mean of its squares (all of one sign), the root and quotient, two products
    rel = (2 + _chain(h.shape[1]) / 2 + 8) * U
    hp = (h, rounded(h, U * np.abs(h), in_dtype))
    if out_dtype != 'e4m3':
        return (y, rounded(y, rel * np.abs(y), out_dtype)), hp
    scale = np.maximum(np.abs(y).max(-1) / TOP, 2.0 ** -126)
    q = y / scale[:, None]
    # half a step: 2^-4 of the value, or of the smallest numbers' step 2^-9
    tol = np.maximum(2.0 ** -4 * np.abs(q), 2.0 ** -10) + (2 * rel + 4 * U) * np.abs(q) * (1 + 2.0 ** -4)
    return (q, tol), (scale, (rel + 2 * U) * scale + TINY), hp


def rms_norm_bwd(dy, h, w, dsum=None, eps=1e-5, dtype='f32'):
    dy, h, w = (t.astype(np.float64) for t in (dy, h, w))
    n = h.shape[1]
    rstd = 1 / np.sqrt((h * h).mean(-1, keepdims=True) + eps)
    xh, g = h * rstd, dy * w
    m = (g * xh).mean(-1, keepdims=True)
    dh = rstd * (g - xh * m)
    rel = (_chain(n) / 2 + 10) * U
    tm = (_chain(n) + 4) * U * np.abs(g * xh).mean(-1, keepdims=True) + rel * np.abs(m)
    tol = rstd * (4 * U * np.abs(g) + np.abs(xh) * (tm + 2 * rel * np.abs(m))) + rel * rstd * (np.abs(g) + np.abs(xh * m))
    if dsum is not None:
        dh = dh + dsum.astype(np.float64)
        tol = tol + U * np.abs(dsum)
    dw = (dy * xh).sum(0)
    return {'x': (dh, rounded(dh, tol, dtype)),
            'weight': (dw, (rel + (h.shape[0] + 32) * U) * np.abs(dy * xh).sum(0) + TINY)}


# ---- norm and clipping -----------------------------------------------------------

def grad_norm(grads):
    n = np.sqrt(sum((g.astype(np.float64) ** 2).sum() for g in grads))
    return n, 2 * U * n + 1e-45    # (a float: infinite where no float is near)


def clip(grads, max_norm, out_dtypes, norm=None):
    """[(out, tol)]: the norm, the quotient, its rounding to fp32 and the product."""
    n = grad_norm(grads)[0] if norm is None else float(norm)
    c = min(1.0, max_norm / (n + 1e-6))
    return [(g.astype(np.float64) * c, rounded(g * c, 6 * U * np.abs(g * c), t)) for g, t in zip(grads, out_dtypes)]
