"""The float64 references of the dense operators against direct loops, differences and torch's
own functions, on the CPU."""
import numpy as np
import pytest
import torch

import dense_reference as ref

ACTS = ['none', 'sigmoid', 'silu', 'gelu_tanh']


def f(rng, *s):
    return rng.standard_normal(s)


@pytest.mark.parametrize('name', ACTS)
def test_activation_is_torchs(name):
    z = torch.linspace(-40, 40, 4001, dtype=torch.float64)
    want = {'none': lambda t: t, 'sigmoid': torch.sigmoid, 'silu': torch.nn.functional.silu,
            'gelu_tanh': lambda t: torch.nn.functional.gelu(t, approximate='tanh')}[name](z)
    assert np.allclose(ref.act(name, z.numpy()), want.numpy(), rtol=1e-12, atol=1e-14)


@pytest.mark.parametrize('name', ACTS)
def test_slope_by_differences(name):
    z = np.linspace(-12, 12, 997)
    d = 1e-5
    num = (ref.act(name, z + d) - ref.act(name, z - d)) / (2 * d)
    assert np.abs(ref.slope(name, z) - num).max() < 1e-9


@pytest.mark.parametrize('name', ['sigmoid', 'silu', 'gelu_tanh'])
def test_no_activation_is_steeper_than_allowed_for(name):
    assert np.abs(ref.slope(name, np.linspace(-50, 50, 100001))).max() < 1.2


def test_linear_by_loops():
    rng = np.random.default_rng(1)
    M, N, K = 3, 4, 5
    x, w, b, r, sx, sw = f(rng, M, K), f(rng, N, K), f(rng, N), f(rng, M, N), f(rng, M) ** 2, f(rng, N) ** 2
    (y, _), (z, _) = ref.linear_fwd(x, w, b, r, 'silu', sx, sw)
    for m in range(M):
        for n in range(N):
            s = sum(x[m, k] * w[n, k] for k in range(K)) * sx[m] * sw[n] + b[n]
            assert np.isclose(z[m, n], s) and np.isclose(y[m, n], s / (1 + np.exp(-s)) + r[m, n])


@pytest.mark.parametrize('name', ACTS)
def test_linear_bwd_by_differences(name):
    rng = np.random.default_rng(2)
    M, N, K = 3, 4, 5
    x, w, b, dy = f(rng, M, K), f(rng, N, K), f(rng, N), f(rng, M, N)
    z = x @ w.T + b
    g = ref.linear_bwd(dy, x, w, z, name)
    loss = lambda: (ref.act(name, x @ w.T + b) * dy).sum()   # noqa: E731
    for n, t in (('x', x), ('weight', w), ('bias', b)):
        for i in np.ndindex(t.shape):
            old, d = t[i], 1e-6
            t[i] = old + d
            up = loss()
            t[i] = old - d
            num = (up - loss()) / (2 * d)
            t[i] = old
            assert abs(g[n][0][i] - num) < 1e-7, (n, i)


def test_rms_norm_by_loops_and_differences():
    rng = np.random.default_rng(3)
    R, C = 3, 6
    x, r, w, dy, ds = f(rng, R, C), f(rng, R, C), f(rng, C), f(rng, R, C), f(rng, R, C)
    (y, _), (h, _) = ref.rms_norm_fwd(x, w, r)
    for i in range(R):
        ms = sum(v * v for v in x[i] + r[i]) / C
        assert np.allclose(y[i], (x[i] + r[i]) / np.sqrt(ms + 1e-5) * w)
    (q, _), (s, _), _ = ref.rms_norm_fwd(x, w, r, out_dtype='e4m3')
    assert np.allclose(q * s[:, None], y) and np.allclose(np.abs(q).max(-1), 448)
    g = ref.rms_norm_bwd(dy, h, w, ds)
    h = h.copy()
    loss = lambda: (ref.rms_norm_fwd(h, w)[0][0] * dy + h * ds).sum()   # noqa: E731
    for n, t in (('x', h), ('weight', w)):
        for i in np.ndindex(t.shape):
            old, d = t[i], 1e-6
            t[i] = old + d
            up = loss()
            t[i] = old - d
            num = (up - loss()) / (2 * d)
            t[i] = old
            assert abs(g[n][0][i] - num) < 1e-7, (n, i)


def test_clip():
    rng = np.random.default_rng(4)
    gs = [f(rng, 5), f(rng, 2, 3), f(rng, 0)]
    n, _ = ref.grad_norm(gs)
    assert np.isclose(n, np.sqrt(sum(v * v for g in gs for v in g.ravel())))
    out = ref.clip(gs, 0.5, ['f32'] * 3)
    assert np.isclose(ref.grad_norm([o for o, _ in out])[0], 0.5, rtol=1e-5)
    assert all(np.array_equal(o, g) for (o, _), g in zip(ref.clip(gs, 100.0, ['f32'] * 3), gs))
