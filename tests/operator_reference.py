"""Plain float64 forms of the operators around the mixer, with how far a float32
computation of them may be off.

The recurrence runs on the pinned C oracle and the convolution on the pinned
prologue oracle (tests/test_oracle_pins.py); layer norm and the gradients are
written out here and checked against differences in test_operator_reference.py.

Each function returns (reference, tolerance) pairs of the same shape. A
tolerance is derived, not fitted: with u = 2^-24 a rounding is off by at most u
of its result, a sum of n terms added in a chain by n u of the sum of their
magnitudes; an output in bf16 adds 2^-8 of its value (and one step of the
smallest numbers). What the magnitudes are is written at each.
"""
from __future__ import annotations

import numpy as np

import oracle
import oracle.prologue as opro

U = 2.0 ** -24
TINY = 1e-37


def rounded(ref, tol, out_dtype):
    """Add the output's own rounding to a tolerance."""
    half = 2.0 ** -8 if out_dtype == 'bf16' else U
    return tol + half * (np.abs(ref) + tol) + TINY


# ---- recurrence on slots -------------------------------------------------------

def recurrent(q, k, v, log_alpha, b, w, state, lens, slot_in=None, slot_out=None, commit=None, out_dtype='f32'):
    """q, k [tokens, HK, dk]; v, w [tokens, H, dv]; b, log_alpha [tokens, H, dk] (gates given per
    channel); state [slots, H, dk, dv]; all numpy. Returns (o, tol), (state after, tol).

    Tolerance: each token multiplies the state by a decay, subtracts a rank-one term and adds one. The
    dot products over dk channels run as dk/4 steps of four; with |k| <= 1 and gates in [0, 1] no step
    lengthens a state column by more than 5% (the operator norm of I - k (b k)^T is at most about 1.03),
    so errors of the tokens add up:
    dk/4 + 16 roundings a token (dot, exp of the decay, update) of the largest column norm or written
    value, twice that for the block form, whose triangular factor repeats the dots of A and P."""
    tokens, H, dv = v.shape
    HK, dk = q.shape[1:]
    qh, kh = (np.repeat(x, H // HK, axis=1) for x in (q, k))
    N = len(lens)
    first = np.concatenate([[0], np.cumsum(lens)])
    slots = state.shape[0]
    o, otol = np.zeros((tokens, H, dv)), np.zeros((tokens, H, dv))
    after, stol = state.astype(np.float64).copy(), np.zeros(state.shape)
    inside = lambda s: 0 <= s < slots   # noqa: E731
    for i in range(N):
        s = slice(first[i], first[i + 1])
        sin = i if slot_in is None else int(slot_in[i])
        sout = sin if slot_out is None else int(slot_out[i])
        S0 = state[sin:sin + 1].astype(np.float64) if inside(sin) else np.zeros((1, H, dk, dv))
        n = lens[i] if commit is None else min(max(int(commit[i]), 0), lens[i])
        run = lambda a, e, st: oracle.forward(qh[a:e], kh[a:e], v[a:e], log_alpha[a:e], b[a:e], w[a:e], st,   # noqa: E731
                                              cu_seqlens=np.array([0, e - a], np.int32), nthreads=4)
        mid = S0
        if n > 0:
            o[s.start:s.start + n], mid = run(s.start, s.start + n, S0)
        if n < lens[i]:
            o[s.start + n:s.stop], _ = run(s.start + n, s.stop, mid)
        size = np.sqrt((S0 ** 2).sum(2)).max() if lens[i] == 0 else max(
            np.sqrt((S0 ** 2).sum(2)).max(), np.sqrt((mid ** 2).sum(2)).max(), np.abs(w[s] * v[s]).max() * 2)
        per = 2 * 1.05 * (dk / 4 + 16) * U * size
        otol[s] = per * (np.arange(lens[i]) + 1)[:, None, None]
        if inside(sout):
            after[sout] = mid[0]
            stol[sout] = per * n
    return (o, rounded(o, otol, out_dtype)), (after, stol)


# ---- prologue -------------------------------------------------------------------

def _segments(lens):
    first = np.concatenate([[0], np.cumsum(lens)])
    return [(first[i], first[i + 1]) for i in range(len(lens))]


def _history(hist, slot, i, shape):
    """[heads, 3, d] before sequence i, or zeros."""
    if hist is None:
        return np.zeros(shape)
    s = i if slot is None else int(slot[i])
    return hist[s].astype(np.float64) if 0 <= s < hist.shape[0] else np.zeros(shape)


def _histories(hist, slot, N, heads, d):
    return np.stack([_history(hist, slot, i, (heads, 3, d)) for i in range(N)])


def conv(x, weight, bias, lens, hist, slot):
    """y and the same sum of magnitudes |bias| + sum |w x|."""
    heads, d = x.shape[1:]
    cu = np.concatenate([[0], np.cumsum(lens)])
    h = _histories(hist, slot, len(lens), heads, d)
    y, _ = opro.short_conv(x, weight, bias, cu_seqlens=cu, history=h)
    m, _ = opro.short_conv(np.abs(x), np.abs(weight), None if bias is None else np.abs(bias), cu_seqlens=cu,
                           history=np.abs(h))
    return y, m


def sigmoid(x):
    return 1 / (1 + np.exp(-np.asarray(x, np.float64)))


def prologue_fwd(raw, logits, weight, bias, lens, hist=None, slot_in=None, slot_out=None, commit=None, dtype='f32'):
    """Returns five (reference, tolerance) pairs and the three pools after.

    Tolerance: y is five roundings of M = |bias| + sum |w x|. The squared norm adds d/8 + 8 roundings
    and what y is off by, 6 u |M| / |y| of it; the reciprocal root is good to 2 units (2^-22). The
    sigmoid: exp is off by 2^-22 + |x| u of itself, the sum and the reciprocal (2^-23) by 4 u more."""
    out = []
    for z, x in enumerate(raw):
        d = x.shape[-1]
        y, m = conv(x, weight[z], bias[z], lens, hist and hist[z], slot_in)
        tol = 6 * U * m
        if z < 2:
            n = np.sqrt((y ** 2).sum(-1, keepdims=True))
            r = 1 / np.maximum(n, 1e-12)
            y = y * r
            off = (d / 8 + 16) * U + 6 * U * np.sqrt((m ** 2).sum(-1, keepdims=True)) * r
            tol = tol * r + off * np.abs(y)
        out.append((y, rounded(y, tol, dtype)))
    for x in logits:
        s = sigmoid(x)
        out.append((s, rounded(s, s * (8 + 2 * np.abs(x)) * U, dtype)))
    pools = None
    if hist is not None:
        pools = [h.copy() for h in hist]
        for i, (a, e) in enumerate(_segments(lens)):
            s = i if slot_in is None else int(slot_in[i])
            so = s if slot_out is None else int(slot_out[i])
            if not 0 <= so < hist[0].shape[0]:
                continue
            n = e - a if commit is None else min(max(int(commit[i]), 0), e - a)
            for z, x in enumerate(raw):
                before = _history(hist[z], slot_in, i, hist[z].shape[1:])
                rows = np.concatenate([before.transpose(1, 0, 2), x[a:a + n]])
                pools[z][so] = rows[-3:].transpose(1, 0, 2)
    return out, pools


def _shift_back(d, weight, lens):
    """dx_t = sum_j w_j d_{t+3-j} within each sequence."""
    heads, c = d.shape[1:]
    w = weight.reshape(heads, c, 4)
    dx = np.zeros_like(d)
    for a, e in _segments(lens):
        for j in range(4):
            back = 3 - j
            if e - a > back:
                dx[a:e - back] += w[..., j] * d[a + back:e]
    return dx


def prologue_bwd(raw, logits, weight, bias, grads, lens, hist=None, slot_in=None, dtype='f32'):
    """{name: (reference, tolerance)}.

    Tolerance: with r = 1/|y| and kappa = r |M| (M as in the forward: how much the convolution cancels),
    dy = r (dq - q (q.dq)) is off by (d/4 + 40) kappa u of D = r (|dq| + |q| |dq|_2); dx adds four such
    terms with |w|. The taps' sums add at most 256 tokens in a chain, then the partial rows in 16 chains."""
    out = {}
    cu = np.concatenate([[0], np.cumsum(lens)])
    for z, name in enumerate('qkv'):
        x, dq = raw[z].astype(np.float64), grads[z].astype(np.float64)
        tokens, heads, d = x.shape
        y, m = conv(x, weight[z], bias[z], lens, hist and hist[z], slot_in)
        dy, size, off = dq, np.abs(dq), np.full((tokens, 1, 1), 2 * U)
        if z < 2:
            n = np.sqrt((y ** 2).sum(-1, keepdims=True))
            r = 1 / np.maximum(n, 1e-12)
            q = y * r
            along = np.where(n > 1e-12, (q * dq).sum(-1, keepdims=True), 0)
            dy = r * (dq - q * along)
            size = r * (np.abs(dq) + np.abs(q) * np.sqrt((dq ** 2).sum(-1, keepdims=True)))
            kappa = np.maximum(1, r * np.sqrt((m ** 2).sum(-1, keepdims=True)))
            off = (d / 4 + 40) * U * kappa ** 2
        err = off * size
        dx = _shift_back(dy, weight[z], lens)
        tol = _shift_back(err + 4 * U * size, np.abs(weight[z]), lens)
        out[name + '_raw'] = (dx, rounded(dx, tol, dtype))
        h = _histories(hist and hist[z], slot_in, len(lens), heads, d)
        serial = 256 + tokens / 16 / 16 + 32
        dw, dwt = np.zeros((heads, d, 4)), np.zeros((heads, d, 4))
        for i, (a, e) in enumerate(_segments(lens)):
            ext = np.concatenate([h[i].transpose(1, 0, 2), x[a:e]])
            for j in range(4):
                xs = ext[j:j + e - a]
                dw[..., j] += (dy[a:e] * xs).sum(0)
                dwt[..., j] += ((err[a:e] + serial * U * np.abs(dy[a:e])) * np.abs(xs)).sum(0)
        out['weight_' + name] = (dw.reshape(-1, 4), dwt.reshape(-1, 4) + TINY)
        if bias[z] is not None:
            out['bias_' + name] = (dy.sum(0).ravel(), (err + serial * U * np.abs(dy)).sum(0).ravel() + TINY)
    for x, name, dg in zip(logits, ('b_logit', 'w_logit'), grads[3:]):
        s = sigmoid(x)
        g = dg * s * (1 - s)
        # 1 - s of a rounded s: one more unit of s
        tol = np.abs(dg) * s * ((8 + 2 * np.abs(x)) * U * (1 - s) + (10 + 2 * np.abs(x)) * U * s)
        out[name] = (g, rounded(g, tol, dtype))
    assert cu[-1] == raw[0].shape[0]
    return out


# ---- layer norm -------------------------------------------------------------------

def _chain(cols):
    """Terms a thread adds in a row's sums (at most 32 in registers, or every 1024th of a long
    row), the lanes' and waves' sums."""
    return max(32, cols / 1024) + 24


def _normalised(h, eps):
    """xh, rstd and how far float32 statistics leave xh: the mean is off by K u of the mean
    magnitude, the deviations by that and their own rounding, the variance by 2 K u of itself."""
    K = _chain(h.shape[-1])
    mean = h.mean(-1, keepdims=True)
    c = h - mean
    var = (c ** 2).mean(-1, keepdims=True)
    rstd = 1 / np.sqrt(var + eps)
    dc = U * (np.abs(h) + (K + 2) * np.abs(h).mean(-1, keepdims=True))
    # the deviations' errors move the variance by 2 mean(|c| dc), relative to var + eps
    drel = 2 * (np.abs(c) * dc).mean(-1, keepdims=True) * rstd ** 2 + (K + 8) * U
    return c * rstd, rstd, dc * rstd + np.abs(c) * rstd * drel, drel


def layer_norm_fwd(x, weight, bias, residual=None, eps=1e-5, out_dtype='f32', in_dtype='f32'):
    """(y, tol), (h, tol)."""
    h = x.astype(np.float64) + (0 if residual is None else residual.astype(np.float64))
    xh, rstd, dxh, _ = _normalised(h, eps)
    if residual is not None:
        dxh = dxh + 2 * U * rstd * (np.abs(h) + np.abs(h).mean(-1, keepdims=True))
    y = xh * weight + (0 if bias is None else bias)
    tol = np.abs(weight) * (dxh + 2 * U * np.abs(xh)) + 2 * U * np.abs(y)
    return (y, rounded(y, tol, out_dtype)), (h, rounded(h, 0, in_dtype))


def layer_norm_bwd(dy, h, weight, dsum=None, eps=1e-5, dtype='f32'):
    """{name: (reference, tolerance)}. dh = rstd (g - mean(g) - xh mean(g xh)): each sum off by K u of
    its terms' magnitudes and by what xh is off; the weights' sums run over the rows in a chain."""
    h, dy = h.astype(np.float64), dy.astype(np.float64)
    rows, cols = h.shape
    K = _chain(cols)
    xh, rstd, dxh, drel = _normalised(h, eps)
    g = dy * weight
    ag = np.abs(g)
    gm, gx = g.mean(-1, keepdims=True), (g * xh).mean(-1, keepdims=True)
    dh = rstd * (g - gm - xh * gx)
    agx = (ag * np.abs(xh)).mean(-1, keepdims=True)
    parts = (ag + ag.mean(-1, keepdims=True) + np.abs(xh) * agx)
    tol = rstd * ((K + 8) * U * parts + drel * parts + dxh * agx + np.abs(xh) * (ag * dxh).mean(-1, keepdims=True))
    if dsum is not None:
        dh = dh + dsum
        tol = tol + U * (np.abs(dh) + np.abs(dsum))
    chain = rows / 128 + 64
    return {'x': (dh, rounded(dh, tol, dtype)),
            'weight': ((dy * xh).sum(0), (np.abs(dy) * (dxh + chain * U * np.abs(xh))).sum(0) + TINY),
            'bias': (dy.sum(0), chain * U * np.abs(dy).sum(0) + TINY)}


def check(name, got, pair):
    """Assert that ``got`` is within the tolerance everywhere; returns the largest error over it."""
    ref, tol = pair
    got = np.asarray(got, np.float64).reshape(ref.shape)
    if not ref.size:
        return 0.0
    err = np.abs(got - ref)
    over = float(np.max(err / tol)) if np.all(tol > 0) else float(np.max(np.where(err > tol, np.inf, 0)))
    assert np.all(np.isfinite(got)), f'{name}: non-finite values'
    at = np.unravel_index(np.argmax(err - tol), ref.shape)
    assert np.all(err <= tol), f'{name}: {got[at]} for {ref[at]} at {at}, off by {err[at]:.3e}, allowed {tol[at]:.3e}'
    return over
