"""The float64 forms that the operators' GPU tests compare with, against differences
and against torch's own functions in float64 (CPU)."""
import numpy as np
import pytest
import torch

import operator_reference as ref


def _difference(f, x, g, eps=1e-5):
    """Directional derivative of sum(f(x) * g) along each element, by central differences."""
    d = np.zeros(x.size)
    flat = x.reshape(-1)
    for i in range(x.size):
        old = flat[i]
        flat[i] = old + eps
        up = (f() * g).sum()
        flat[i] = old - eps
        down = (f() * g).sum()
        flat[i] = old
        d[i] = (up - down) / (2 * eps)
    return d.reshape(x.shape)


@pytest.mark.parametrize('cols', [1, 2, 5, 16])
def test_layer_norm_against_torch_and_differences(cols):
    rng = np.random.default_rng(cols)
    h, w, b = rng.standard_normal((4, cols)) + 1, 1 + rng.standard_normal(cols) / 4, rng.standard_normal(cols)
    dy = rng.standard_normal((4, cols))
    (y, _), _ = ref.layer_norm_fwd(h, w, b)
    t = [torch.tensor(a, requires_grad=True) for a in (h, w, b)]
    ty = torch.nn.functional.layer_norm(t[0], (cols,), t[1], t[2], 1e-5)
    assert np.allclose(y, ty.detach().numpy(), rtol=1e-12, atol=1e-12)
    g = ref.layer_norm_bwd(dy, h, w)
    fwd = lambda: ref.layer_norm_fwd(h, w, b)[0][0]   # noqa: E731
    for name, x in (('x', h), ('weight', w), ('bias', b)):
        # second-order error eps^2 times a third derivative, at most rstd^3 ~ 3e7 where a row has no spread
        assert np.allclose(g[name][0], _difference(fwd, x, dy), rtol=1e-5, atol=1e-5 if cols > 2 else 1e-2), name


def _prologue_case(seed, lens, HK, H, dk, dv, history):
    rng = np.random.default_rng(seed)
    T = sum(lens)
    shapes = ((HK, dk), (HK, dk), (H, dv))
    raw = [rng.standard_normal((T, *s)) for s in shapes]
    logits = [rng.standard_normal((T, H, dk)), rng.standard_normal((T, H))]
    weight = [rng.uniform(-.5, .5, (s[0] * s[1], 4)) for s in shapes]
    bias = [rng.uniform(-.5, .5, s[0] * s[1]) for s in shapes]
    hist = [rng.standard_normal((len(lens) + 1, s[0], 3, s[1])) for s in shapes] if history else None
    slot = rng.permutation(len(lens) + 1)[:len(lens)] if history else None
    grads = [rng.standard_normal(x.shape) for x in (*raw, *logits)]
    return raw, logits, weight, bias, hist, slot, grads


@pytest.mark.parametrize('history', [False, True])
def test_prologue_gradient_against_differences(history):
    lens = [3, 0, 1, 5]
    raw, logits, weight, bias, hist, slot, grads = _prologue_case(3, lens, 1, 2, 3, 2, history)
    g = ref.prologue_bwd(raw, logits, weight, bias, grads, lens, hist, slot)
    for z, n in enumerate('qkv'):
        fwd = lambda: ref.prologue_fwd(raw, logits, weight, bias, lens, hist, slot)[0][z][0]   # noqa: B023, E731
        for name, x in ((n + '_raw', raw[z]), ('weight_' + n, weight[z]), ('bias_' + n, bias[z])):
            assert np.allclose(g[name][0], _difference(fwd, x, grads[z]), rtol=1e-4, atol=1e-6), name
    for z, n in ((3, 'b_logit'), (4, 'w_logit')):
        fwd = lambda: ref.prologue_fwd(raw, logits, weight, bias, lens, hist, slot)[0][z][0]   # noqa: B023, E731
        assert np.allclose(g[n][0], _difference(fwd, logits[z - 3], grads[z]), rtol=1e-6, atol=1e-8), n


def test_prologue_histories_carry():
    """Two calls with the history carried equal one; commit keeps a prefix."""
    raw, logits, weight, bias, hist, slot, _ = _prologue_case(5, [7, 4], 1, 2, 4, 4, True)
    whole, pools = ref.prologue_fwd(raw, logits, weight, bias, [7, 4], hist, slot)
    cut = [2, 3]
    first = [np.concatenate([x[:2], x[7:10]]) for x in raw]
    rest = [np.concatenate([x[2:7], x[10:]]) for x in raw]
    lg = [x[:5] for x in logits]
    a, mid = ref.prologue_fwd(first, lg, weight, bias, cut, hist, slot)
    b, end = ref.prologue_fwd(rest, [x[:6] for x in logits], weight, bias, [5, 1], mid, slot)
    _, kept = ref.prologue_fwd(raw, logits, weight, bias, [7, 4], hist, slot, commit=cut)
    for z in range(3):
        joined = np.concatenate([a[z][0][:2], b[z][0][:5], a[z][0][2:], b[z][0][5:]])
        assert np.allclose(joined, whole[z][0], rtol=1e-13, atol=1e-13)
        assert np.array_equal(end[z], pools[z]) and np.array_equal(kept[z], mid[z])


def test_recurrent_slots_and_commit():
    rng = np.random.default_rng(0)
    lens, H, HK, dk, dv, slots = [3, 0, 5], 2, 1, 4, 3, 6
    T = sum(lens)
    n = lambda *s: rng.standard_normal(s)   # noqa: E731
    q, k = (x / np.linalg.norm(x, axis=-1, keepdims=True) for x in (n(T, HK, dk), n(T, HK, dk)))
    v, b, w, la = n(T, H, dv), rng.random((T, H, dk)), rng.random((T, H, dv)), -rng.random((T, H, dk))
    state = n(slots, H, dk, dv)
    (o, _), (after, _) = ref.recurrent(q, k, v, la, b, w, state, lens, [4, 1, -1], [0, 3, 2], [2, 0, 9])
    # token by token, in the printed matrix form
    for i, (a, e) in enumerate(ref._segments(lens)):
        sin, sout, c = [4, 1, -1][i], [0, 3, 2][i], [2, 0, 9][i]
        for h in range(H):
            S = state[sin, h].copy() if sin >= 0 else np.zeros((dk, dv))
            kept = S
            for t in range(a, e):
                kt, qt = k[t, 0], q[t, 0]
                S = (np.eye(dk) - np.outer(kt, b[t, h] * kt)) @ (np.exp(la[t, h])[:, None] * S) + np.outer(
                    kt, w[t, h] * v[t, h])
                assert np.allclose(o[t, h], qt @ S, rtol=1e-12, atol=1e-12)
                if t - a + 1 == c or (t == e - 1 and c > e - a):
                    kept = S
            assert np.allclose(after[sout, h], kept, rtol=1e-12, atol=1e-12)
    untouched = [s for s in range(slots) if s not in (0, 3, 2)]
    assert np.array_equal(after[untouched], state[untouched])
