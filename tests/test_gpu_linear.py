"""gdn2_linear_fwd / gdn2_linear_bwd against float64: every form of the product (waves that share
the contraction, tiles, rows that are no whole chunks, parts that are joined), every type,
activation and epilogue."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip('torch')
if not torch.cuda.is_available():
    pytest.skip('no GPU', allow_module_level=True)

import dense_reference as ref  # noqa: E402
import gated_delta_rule_wy_amd as gdn2  # noqa: E402
import operator_reference as oref  # noqa: E402
from gpu_util import DEV  # noqa: E402

DT = {'bf16': torch.bfloat16, 'f32': torch.float32, 'e4m3': torch.float8_e4m3fn}
ACTS = ['none', 'sigmoid', 'silu', 'gelu_tanh']
SIZES = [(1, 1, 1), (1, 16, 16), (2, 7, 33), (3, 8, 128), (15, 100, 129), (16, 257, 64), (17, 33, 70), (32, 96, 1000), (33, 100, 129),
         (64, 64, 64), (64, 2048, 520), (65, 130, 200), (256, 512, 2048), (300, 257, 1000), (1000, 2056, 520), (130, 8200, 40),
         (2500, 1000, 777), (5000, 2048, 264)]


def back(t):
    return t.float().cpu().numpy()


class Case:
    """Inputs made on the device (their float values are exact in the type)."""
    def __init__(self, seed, M, N, K, dtype, bias=True, residual=True, out=None, scale=1.0):
        g = torch.Generator().manual_seed(seed)
        n = lambda *s: torch.randn(s, generator=g)   # noqa: E731
        self.dtype, self.out = dtype, out or ('bf16' if dtype == 'e4m3' else dtype)
        x, w = n(M, K) * scale, n(N, K) * (scale / K ** 0.5)
        self.sx = self.sw = None
        if dtype == 'e4m3':
            self.sx, self.sw = 0.5 + torch.rand(M, generator=g), 0.5 + torch.rand(N, generator=g)
        self.x, self.w = x.to(DT[dtype]), w.to(DT[dtype])
        self.b = n(N) if bias else None
        self.r = n(M, N).to(DT[self.out]) if residual else None

    def run(self, act, **kw):
        d = lambda t: None if t is None else t.to(DEV)   # noqa: E731
        return gdn2.linear_fwd(d(self.x), d(self.w), d(self.b), d(self.r), activation=act, x_scale=d(self.sx),
                               weight_scale=d(self.sw), out_dtype=DT[self.out], **kw)

    def want(self, act):
        f = lambda t: None if t is None else t.float().numpy()   # noqa: E731
        return ref.linear_fwd(f(self.x), f(self.w), f(self.b), f(self.r), act, f(self.sx), f(self.sw), self.out,
                              'bf16' if self.dtype == 'bf16' else 'f32')


@pytest.mark.parametrize('dtype', ['bf16', 'f32', 'e4m3'])
@pytest.mark.parametrize('M,N,K', SIZES)
def test_sizes(M, N, K, dtype):
    print(f'[sizes] {M}x{N}x{K} {dtype}', flush=True)
    c = Case(M + N + K, M, N, K, dtype)
    act = ACTS[(M + N) % 4]
    y, z = c.run(act, output_preact=dtype != 'e4m3')
    wy, wz = c.want(act)
    oref.check('y', back(y), wy)
    if z is not None:
        oref.check('z', back(z), wz)
    p = Case(M + N, M, N, K, dtype, bias=False, residual=False)
    oref.check('product', back(p.run(None)[0]), p.want('none')[0])


# 256 x 256 tiles, more than the workgroups that stay, with parts of tiles at both edges and of a
# step at the rows' end; 128 x 128 tiles
@pytest.mark.parametrize('dtype', ['bf16', 'f32', 'e4m3'])
@pytest.mark.parametrize('M,N,K', [(3100, 4104, 272), (4352, 4352, 144), (5000, 520, 1104)])
@pytest.mark.parametrize('act', ['none', 'silu'])
def test_tiles(M, N, K, dtype, act):
    print(f'[tiles] {M}x{N}x{K} {dtype} {act}', flush=True)
    c = Case(M, M, N, K, dtype)
    y, z = c.run(act, output_preact=dtype != 'e4m3')
    wy, wz = c.want(act)
    oref.check('y', back(y), wy)
    if z is not None:
        oref.check('z', back(z), wz)


@pytest.mark.parametrize('act', ACTS)
@pytest.mark.parametrize('dtype,out', [('bf16', 'f32'), ('f32', 'bf16'), ('e4m3', 'f32'), ('e4m3', 'bf16'), ('bf16', 'bf16')])
def test_types_and_activations(dtype, out, act):
    for M, N, K in ((20, 48, 96), (700, 4096, 64)):
        print(f'[types] {M}x{N}x{K} {dtype} -> {out} {act}', flush=True)
        c = Case(7, M, N, K, dtype, out=out, scale=3.0)
        y, _ = c.run(act)
        assert y.dtype == DT[out]
        oref.check('y', back(y), c.want(act)[0])


@pytest.mark.parametrize('act', ['sigmoid', 'silu', 'gelu_tanh'])
def test_far_arguments(act):
    """Where exp overflows or vanishes: z from the bias alone."""
    z = np.array([-1e30, -1e5, -200, -104, -88, -50, -17, -16, -15, -1e-30, 0, 1e-30, 15, 17, 50, 88, 104, 200, 1e5, 1e30], np.float32)
    if act == 'gelu_tanh':
        z = z[np.abs(z) < 1e6]    # (z^3 is finite)
    N = len(z)
    x, w = torch.zeros(2, 8, device=DEV), torch.zeros(N, 8, device=DEV)
    y, _ = gdn2.linear_fwd(x, w, torch.from_numpy(z).to(DEV), activation=act)
    want, _ = ref.linear_fwd(np.zeros((2, 8)), np.zeros((N, 8)), z, None, act)
    oref.check('y', back(y), want)
    zs = torch.from_numpy(np.tile(z, (2, 1))).to(DEV)
    dy = torch.full_like(zs, 1.5)
    g = gdn2.linear_bwd(dy, x, w, zs, activation=act, output_x=False, output_weight=False)
    oref.check('bias', back(g['bias']), ref.linear_bwd(np.full((2, N), 1.5), np.zeros((2, 8)), np.zeros((N, 8)), np.tile(z, (2, 1)),
                                                       act)['bias'])


@pytest.mark.parametrize('dtype', ['bf16', 'f32', 'e4m3'])
@pytest.mark.parametrize('M,N,K', [(5, 24, 40), (70, 100, 300), (700, 2000, 208), (3100, 4104, 272), (333, 4001, 131)])
def test_nothing_is_read_or_written_beyond_the_tensors(M, N, K, dtype):
    """Operands that are followed by NaN; an output that is followed by numbers that stay."""
    print(f'[beyond] {M}x{N}x{K} {dtype}', flush=True)
    c = Case(3, M, N, K, dtype, bias=False, residual=False)

    def inside(t):
        flat = torch.full((t.numel() + 4096,), float('nan'), device=DEV).to(t.dtype)
        flat[:t.numel()] = t.flatten().to(DEV)
        return flat[:t.numel()].view(t.shape)

    buf = torch.full((M * N + 4096,), 7.0, device=DEV, dtype=DT[c.out])
    d = lambda t: None if t is None else inside(t)   # noqa: E731
    y, _ = gdn2.linear_fwd(inside(c.x), inside(c.w), x_scale=d(c.sx), weight_scale=d(c.sw), out=buf[:M * N].view(M, N))
    oref.check('y', back(y), c.want('none')[0])
    assert torch.all(buf[M * N:] == 7.0)


@pytest.mark.parametrize('dtype', ['bf16', 'f32', 'e4m3'])
@pytest.mark.parametrize('M,N,K', [(20, 40, 64), (300, 600, 100), (3100, 4104, 272)])
def test_not_finite_stays_in_its_row_and_column(M, N, K, dtype):
    c = Case(4, M, N, K, dtype, residual=False)
    bad = torch.tensor(float('nan')).to(DT[dtype])
    clean = c.want('none')[0]
    c.x[M // 2, K - 1] = bad
    c.w[N - 1, 0] = bad
    y = back(c.run(None)[0])
    rows, cols = np.arange(M) != M // 2, np.arange(N) != N - 1
    assert np.all(np.isnan(y[M // 2])) and np.all(np.isnan(y[:, N - 1]))
    oref.check('y', y[rows][:, cols], (clean[0][rows][:, cols], clean[1][rows][:, cols]))


def test_leading_axes_and_no_rows():
    c = Case(5, 24, 40, 48, 'bf16')
    want = back(c.run('silu')[0])
    c.x, c.r = c.x.view(2, 3, 4, 48), c.r.view(2, 3, 4, 40)
    y, z = c.run('silu', output_preact=True)
    assert y.shape == z.shape == (2, 3, 4, 40) and np.array_equal(back(y).reshape(24, 40), want)
    one = gdn2.linear_fwd(c.x[0, 0, 0].to(DEV), c.w.to(DEV))[0]
    assert one.shape == (40,)
    e = torch.empty(0, 48, device=DEV, dtype=torch.bfloat16)
    y, _ = gdn2.linear_fwd(e, c.w.to(DEV))
    assert y.shape == (0, 40)
    g = gdn2.linear_bwd(y, e, c.w.to(DEV))
    assert g['x'].shape == (0, 48) and torch.all(g['weight'] == 0) and torch.all(g['bias'] == 0)


@pytest.mark.parametrize('M,N,K', [(9, 40, 64), (700, 2048, 64), (3100, 4104, 64)])
@pytest.mark.parametrize('dtype', ['bf16', 'f32'])
def test_onto_the_residual(M, N, K, dtype):
    c = Case(6, M, N, K, dtype)
    want = c.run('sigmoid')[0]
    r = c.r.to(DEV)
    y, _ = gdn2.linear_fwd(c.x.to(DEV), c.w.to(DEV), c.b.to(DEV), r, activation='sigmoid', out=r)
    assert y is r and torch.equal(y, want)


@pytest.mark.parametrize('M,N,K', [(70000, 32768, 64), (70000, 64, 32768)])
def test_offsets_beyond_32_bits(M, N, K):
    """An output, or an operand, of more than 2^31 elements."""
    print(f'[large] {M}x{N}x{K}', flush=True)
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randn(M, K, generator=g, device=DEV, dtype=torch.bfloat16)
    w = torch.randn(N, K, generator=g, device=DEV, dtype=torch.bfloat16)
    y, _ = gdn2.linear_fwd(x, w)
    rows = [0, 1, 255, 256, 32767, 32768, 65535, 65536, 65537, 69887, 69888, M - 1]
    want, _ = ref.linear_fwd(back(x[rows]), back(w), out_dtype='bf16')
    oref.check('y', back(y[rows]), want)


# ---- gradient ------------------------------------------------------------------

def grad_case(seed, M, N, K, dtype, ddtype, act, **kw):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g)   # noqa: E731
    x, w, dy = n(M, K).to(DT[dtype]), (n(N, K) / K ** 0.5).to(DT[dtype]), n(M, N).to(DT[ddtype])
    z = n(M, N).to(DT[dtype]) * 2 if act != 'none' else None
    got = gdn2.linear_bwd(dy.to(DEV), x.to(DEV), w.to(DEV), None if z is None else z.to(DEV), activation=act, **kw)
    f = lambda t: None if t is None else t.float().numpy()   # noqa: E731
    want = ref.linear_bwd(f(dy), f(x), f(w), f(z), act, dtype)
    if act == 'none' and dtype == 'bf16' and ddtype == 'f32':
        # dy itself is rounded for the products
        half = ref.half_step('bf16')
        a = np.abs(f(dy))
        want['x'] = (want['x'][0], want['x'][1] + half * a @ np.abs(f(w)))
        want['weight'] = (want['weight'][0], want['weight'][1] + half * a.T @ np.abs(f(x)))
    return got, want


@pytest.mark.parametrize('dtype', ['bf16', 'f32'])
@pytest.mark.parametrize('M,N,K', [(1, 1, 1), (1, 16, 16), (5, 7, 9), (64, 64, 64), (65, 130, 200), (300, 257, 1000), (777, 96, 40),
                                   (2500, 1000, 777), (5000, 512, 264), (9000, 40, 72), (3000, 3101, 260), (20000, 300, 300)])
def test_gradient_sizes(M, N, K, dtype):
    act = ACTS[(M + K) % 4]
    print(f'[gradient] {M}x{N}x{K} {dtype} {act}', flush=True)
    got, want = grad_case(M + N, M, N, K, dtype, dtype, act)
    for n in want:
        oref.check(n, back(got[n]), want[n])


@pytest.mark.parametrize('act', ACTS)
@pytest.mark.parametrize('dtype,ddtype', [('bf16', 'bf16'), ('bf16', 'f32'), ('f32', 'bf16'), ('f32', 'f32')])
def test_gradient_types(dtype, ddtype, act):
    got, want = grad_case(11, 500, 168, 200, dtype, ddtype, act)
    for n in want:
        assert got[n].dtype == (torch.float32 if n == 'bias' else DT[dtype])
        oref.check(n, back(got[n]), want[n])


def test_only_the_gradients_that_are_asked_for():
    whole, _ = grad_case(12, 300, 130, 96, 'bf16', 'bf16', 'silu')
    for flags in ((1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 0, 1)):
        names = [n for n, f in zip(('x', 'weight', 'bias'), flags) if f]
        g, _ = grad_case(12, 300, 130, 96, 'bf16', 'bf16', 'silu', output_x=bool(flags[0]), output_weight=bool(flags[1]),
                         output_bias=bool(flags[2]))
        assert sorted(g) == sorted(names) and all(torch.equal(g[n], whole[n]) for n in names)


def test_gradient_by_differences():
    """Central differences of the forward itself, in fp32 on a problem small enough for them."""
    g = torch.Generator().manual_seed(13)
    M, N, K = 4, 6, 5
    x, w, b, dy = (torch.randn(*s, generator=g).to(DEV) for s in ((M, K), (N, K), (N,), (M, N)))
    _, z = gdn2.linear_fwd(x, w, b, activation='gelu_tanh', output_preact=True)
    grads = gdn2.linear_bwd(dy, x, w, z, activation='gelu_tanh')
    loss = lambda: float((gdn2.linear_fwd(x, w, b, activation='gelu_tanh')[0].double() * dy.double()).sum())   # noqa: E731
    for n, t in (('x', x), ('weight', w), ('bias', b)):
        flat = t.view(-1)
        for i in range(flat.numel()):
            old, d = float(flat[i]), 2.0 ** -7
            flat[i] = old + d
            up = loss()
            flat[i] = old - d
            num = (up - loss()) / (2 * d)
            flat[i] = old
            # the differences' own error: d^2 / 6 of the third derivative (below 4 times the magnitudes here,
            # each at most 4), and roundings of the two losses over 2 d
            assert abs(float(grads[n].view(-1)[i]) - num) < 2e-2, (n, i)


# ---- as a program runs them ------------------------------------------------------

@pytest.mark.parametrize('M,N,K', [(7, 200, 136), (400, 2048, 256), (3100, 4104, 272)])
def test_same_bits_and_captured(M, N, K):
    """Two eager calls agree bit for bit, and so does every replay of a captured pass, forward and backward,
    with new values in the same memory."""
    c = Case(14, M, N, K, 'bf16')
    x, w, b, r = (t.to(DEV) for t in (c.x, c.w, c.b, c.r))
    dy = torch.randn_like(r)
    need = gdn2.lib().gdn2_linear_bwd_workspace_bytes(M, K, N, 2, gdn2.GDN2_BF16, gdn2.GDN2_BF16, 1, 1, 1)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)

    def step():
        y, z = gdn2.linear_fwd(x, w, b, r, activation='silu', output_preact=True)
        return [y, z, *gdn2.linear_bwd(dy, x, w, z, activation='silu', workspace=ws).values()]

    first, second = step(), step()
    assert all(torch.equal(p, q) for p, q in zip(first, second))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(4):
        x.copy_(torch.randn_like(x))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        assert all(torch.equal(p, q) for p, q in zip(got, step())), i


def test_two_streams():
    """Calls on two streams at once, each with what the other must not touch."""
    cases = [Case(15 + i, 600, 2048, 256, 'bf16') for i in range(2)]
    dev = [[t.to(DEV) for t in (c.x, c.w, c.b, c.r)] for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    outs = [[], []]
    for _ in range(5):
        for i, (s, d) in enumerate(zip(streams, dev)):
            with torch.cuda.stream(s):
                y, z = gdn2.linear_fwd(*d, activation='silu', output_preact=True)
                outs[i].append((y, gdn2.linear_bwd(y, d[0], d[1], z, activation='silu')))
    torch.cuda.synchronize()
    for i, c in enumerate(cases):
        oref.check('y', back(outs[i][0][0]), c.want('silu')[0])
        for y, g in outs[i][1:]:
            assert torch.equal(y, outs[i][0][0]) and all(torch.equal(g[n], outs[i][0][1][n]) for n in g)


def test_binding_refuses():
    x, w = torch.zeros(4, 8, device=DEV), torch.zeros(5, 8, device=DEV)
    y = torch.zeros(4, 5, device=DEV)
    e = lambda t: t.to(torch.float8_e4m3fn)   # noqa: E731
    one = torch.ones(4, device=DEV)
    for err, args, kw in [
            (ValueError, (x.t(), w), {}), (ValueError, (torch.zeros(4, 16, device=DEV)[:, ::2], w), {}), (ValueError, (x, w.t()), {}),
            (TypeError, (x, w.bfloat16()), {}), (TypeError, (x.half(), w.half()), {}), (ValueError, (x, w, torch.zeros(4, device=DEV)), {}),
            (TypeError, (x, w, torch.zeros(5, device=DEV).bfloat16()), {}), (ValueError, (x, w, None, y[:2]), {}),
            (TypeError, (x, w, None, y.bfloat16()), {}), (ValueError, (x, w), dict(activation='relu')),
            (ValueError, (x, w), dict(x_scale=one)), (ValueError, (e(x), e(w)), {}), (ValueError, (e(x), e(w)), dict(x_scale=one)),
            (ValueError, (e(x), e(w)), dict(x_scale=one[:3], weight_scale=torch.ones(5, device=DEV))),
            (ValueError, (e(x), e(w)), dict(x_scale=one, weight_scale=torch.ones(5, device=DEV), output_preact=True)),
            (TypeError, (x, w), dict(out_dtype=torch.float16)), (ValueError, (x, w.cpu()), {}), (ValueError, (x, w), dict(out=y[:3]))]:
        with pytest.raises(err):
            gdn2.linear_fwd(*args, **kw)
    for err, args, kw in [
            (ValueError, (y, x, w), dict(activation='silu')), (ValueError, (y[:3], x, w), {}), (TypeError, (y.half(), x, w), {}),
            (TypeError, (y, e(x), e(w)), {}), (ValueError, (y, x, w), dict(output_x=False, output_weight=False, output_bias=False)),
            (ValueError, (y, x, w, y.t()), dict(activation='silu')),
            (ValueError, (y, x, w), dict(workspace=torch.empty(1 << 20, dtype=torch.uint8)))]:
        with pytest.raises(err):
            gdn2.linear_bwd(*args, **kw)


@pytest.mark.parametrize('dtype', ['bf16', 'f32', 'e4m3'])
def test_more_rows_than_a_grid_has_blocks(dtype):
    """2^22 rows and a few: 64 at a time are more than a launch's second axis holds."""
    M, N, K = 2 ** 22 + 77, 3, 2
    print(f'[many rows] {M}x{N}x{K} {dtype}', flush=True)
    c = Case(5, M, N, K, dtype)
    oref.check('y', back(c.run('silu')[0]), c.want('silu')[0])


def test_gradient_of_the_most_rows():
    M, N, K = 2 ** 22, 2, 3
    print(f'[most rows] {M}x{N}x{K}', flush=True)
    g = torch.Generator().manual_seed(6)
    dy, x, w = (torch.randn(s, generator=g) for s in ((M, N), (M, K), (N, K)))
    out = gdn2.linear_bwd(dy.to(DEV), x.to(DEV), w.to(DEV))
    want = ref.linear_bwd(dy.numpy(), x.numpy(), w.numpy(), None, 'none')
    for k in ('x', 'weight', 'bias'):
        oref.check(k, back(out[k]), want[k])


# fp32 whose operands are read down their columns: dx alone, dw alone, both; sums of one to many terms
@pytest.mark.parametrize('M,N,K', [(1100, 333, 777), (333, 1100, 777), (1000, 1001, 1003), (1554, 777, 1001), (2000, 1, 300),
                                   (2000, 5, 300), (1, 1500, 400), (17, 1500, 401), (700, 8, 4000), (600, 2000, 2040), (8000, 64, 200)])
@pytest.mark.parametrize('act,ddtype', [('none', 'f32'), ('silu', 'bf16')])
def test_gradient_columns_fp32(M, N, K, act, ddtype):
    print(f'[columns] {M}x{N}x{K} {act} {ddtype}', flush=True)
    got, want = grad_case(M + K, M, N, K, 'f32', ddtype, act)
    for n in want:
        oref.check(n, back(got[n]), want[n])


@pytest.mark.parametrize('M,N,K', [(1000, 1001, 1003), (1100, 336, 777), (333, 1104, 779), (64, 2000, 1040)])
def test_gradient_reads_nothing_beyond_the_tensors(M, N, K):
    """fp32 operands that are followed by NaN; outputs that are followed by numbers that stay."""
    print(f'[beyond] {M}x{N}x{K}', flush=True)
    g = torch.Generator().manual_seed(M)
    dy, x, w = (torch.randn(s, generator=g) for s in ((M, N), (M, K), (N, K)))

    def inside(t):
        flat = torch.full((t.numel() + 4096,), float('nan'), device=DEV)
        flat[:t.numel()] = t.flatten().to(DEV)
        return flat[:t.numel()].view(t.shape)

    dx, dw = (torch.full((n + 4096,), 7.0, device=DEV) for n in (M * K, N * K))
    lib, p = gdn2.lib(), lambda t: t.data_ptr()   # noqa: E731
    need = lib.gdn2_linear_bwd_workspace_bytes(M, K, N, 0, gdn2.GDN2_F32, gdn2.GDN2_F32, 1, 1, 0)
    ws = torch.full((need + 4096,), 0xff, dtype=torch.uint8, device=DEV)   # (NaN as well)
    args = [inside(t) for t in (dy, x, w)]
    lib.gdn2_set_stream(torch.cuda.current_stream().cuda_stream)
    assert lib.gdn2_linear_bwd(*map(p, args), None, p(dx), p(dw), None, M, K, N, 0, gdn2.GDN2_F32, gdn2.GDN2_F32, p(ws), need) == 0
    want = ref.linear_bwd(dy.numpy(), x.numpy(), w.numpy(), None, 'none')
    oref.check('x', back(dx[:M * K].view(M, K)), want['x'])
    oref.check('weight', back(dw[:N * K].view(N, K)), want['weight'])
    assert torch.all(dx[M * K:] == 7.0) and torch.all(dw[N * K:] == 7.0) and torch.all(ws[need:] == 0xff)


def test_only_the_fp32_gradients_that_are_asked_for():
    whole, _ = grad_case(12, 1000, 1001, 1003, 'f32', 'f32', 'silu')
    for flags in ((1, 0, 0), (0, 1, 0), (0, 1, 1)):
        names = [n for n, f in zip(('x', 'weight', 'bias'), flags) if f]
        g, _ = grad_case(12, 1000, 1001, 1003, 'f32', 'f32', 'silu', output_x=bool(flags[0]), output_weight=bool(flags[1]),
                         output_bias=bool(flags[2]))
        assert sorted(g) == sorted(names) and all(torch.equal(g[n], whole[n]) for n in names)


@pytest.mark.parametrize('M,N,K', [(64, 2048, 256), (1000, 1001, 1003), (4999, 500, 255)])
def test_fp32_captured_twice(M, N, K):
    """Two captured passes over the same tensors, replayed in turn on another stream than they were captured
    on, give the eager pass's bits."""
    c = Case(15, M, N, K, 'f32')
    x, w, b, r = (t.to(DEV) for t in (c.x, c.w, c.b, c.r))
    dy = torch.randn_like(r)

    def step():
        y, z = gdn2.linear_fwd(x, w, b, r, activation='gelu_tanh', output_preact=True)
        return [y, z, *gdn2.linear_bwd(dy, x, w, z, activation='gelu_tanh').values()]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    outs = []
    for g in graphs:
        with torch.cuda.graph(g):
            outs.append(step())
    for i in range(3):
        x.copy_(torch.randn_like(x))
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for g in graphs:
                g.replay()
        side.synchronize()
        want = step()
        for out in outs:
            assert all(torch.equal(p, q) for p, q in zip(out, want)), i


def test_weight_gradient_of_more_than_2_to_the_35_elements():
    """64 GiB of dweight from a few rows: whole numbers, so every element has to be the exact one."""
    M, N, K = 16, 2 ** 18, 2 ** 17 + 8
    print(f'[weight] {M}x{N}x{K}', flush=True)
    torch.cuda.empty_cache()
    g = torch.Generator(device=DEV).manual_seed(16)
    dy = torch.randint(-1, 2, (M, N), generator=g, device=DEV).bfloat16()
    x = torch.randint(-8, 9, (M, K), generator=g, device=DEV).bfloat16()
    # (sums of at most 128: whole numbers that bf16 holds)
    dw = torch.empty(N, K, dtype=torch.bfloat16, device=DEV)
    lib, code = gdn2.lib(), gdn2.GDN2_BF16
    need = lib.gdn2_linear_bwd_workspace_bytes(M, K, N, 0, code, code, 0, 1, 0)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    lib.gdn2_set_stream(torch.cuda.current_stream().cuda_stream)
    assert lib.gdn2_linear_bwd(dy.data_ptr(), x.data_ptr(), None, None, None, dw.data_ptr(), None, M, K, N, 0, code, code, ws.data_ptr(),
                               need) == gdn2.GDN2_OK
    xf = x.float()
    for n in range(0, N, 8192):
        assert torch.equal(dw[n:n + 8192], (dy[:, n:n + 8192].float().t().contiguous() @ xf).bfloat16()), n
    del dw
    torch.cuda.empty_cache()


# blocks of the waves that share the contraction, tiles, rows that are no whole chunks
@pytest.mark.parametrize('M,N,K', [(24, 48, 96), (700, 4096, 64), (2000, 1001, 33)])
def test_scales_whose_product_leaves_the_range(M, N, K):
    """x has one element a row, so z is one exact product v times two scales; each of the scales' products
    overflows or vanishes somewhere while v times both does not."""
    g = torch.Generator().manual_seed(17)
    x = torch.zeros(M, K)
    x[torch.arange(M), torch.arange(M) % K] = torch.randint(-8, 9, (M,), generator=g).float() * 2.0 ** torch.randint(-6, 5, (M,), generator=g)
    w = torch.randint(-8, 9, (N, K), generator=g).float() * 2.0 ** -6
    far = torch.tensor([1.0, 1e25, 1e-25, 1e30, 1e-30, 3e38, 1e-38, 1e-42, 0.0])
    mant = lambda n: 1 + torch.rand(n, generator=g) / 9   # noqa: E731
    sx, sw = far[torch.randint(0, 9, (M,), generator=g)] * mant(M), far[torch.randint(0, 9, (N,), generator=g)] * mant(N)
    e, d = lambda t: t.to(DT['e4m3']).to(DEV), lambda t: t.to(DEV)   # noqa: E731
    assert np.array_equal(back(e(x)), x.numpy()) and np.array_equal(back(e(w)), w.numpy())
    y, _ = gdn2.linear_fwd(e(x), e(w), x_scale=d(sx), weight_scale=d(sw), out_dtype=torch.float32)
    v = x.double() @ w.double().t()
    want = (v * sx.double()[:, None] * sw.double()).numpy()
    got = back(y).astype(np.float64)
    # (v, both mantissas' product and v's with it are rounded, and the result; its exponent may leave the range itself)
    inside = np.abs(want) < 3.4e38
    assert np.all(np.abs(got - want)[inside] <= 4 * oref.U * np.abs(want)[inside] + 2.0 ** -149)
    assert np.all(np.isinf(got[np.abs(want) > 3.41e38]))
    assert inside.mean() > 0.5 and np.any((want != 0) & inside & ~np.isfinite((sx[:, None] * sw).numpy()))


# e4m3 sums: one form of the blocks of waves that share the contraction each (16 x 16 to 32 x 64), tiles of each
# size, rows that are no whole chunks in both kinds
SUMS = [(20, 48, 96), (20, 4096, 300 * 16), (60, 4096, 2048), (100, 2048, 512), (256, 2048, 1040), (300, 257, 1000), (1000, 2056, 528),
        (4000, 1024, 272), (5000, 2048, 272), (2000, 1001, 333)]


def check_sums(M, N, K, out):
    """Whole numbers whose every sum, in whatever order, is one below 2^24: 2^16 twice in an aligned eight, which
    cancel, beside products of at most 9. fp32 holds all of it, so the result has to be exact."""
    g = torch.Generator().manual_seed(18)
    x, w = torch.randint(-3, 4, (M, K), generator=g).float(), torch.randint(-3, 4, (N, K), generator=g).float()
    at = torch.arange(0, K - 1, 8)
    at = at[torch.randperm(len(at), generator=g)[:96]]
    x[:, at], x[:, at + 1] = 256.0, 256.0
    w[:, at], w[:, at + 1] = 256.0, -256.0
    want = (x.double() @ w.double().t()).float()
    d, one = lambda t: t.to(DT['e4m3']).to(DEV), lambda n: torch.ones(n, device=DEV)   # noqa: E731
    y, _ = gdn2.linear_fwd(d(x), d(w), x_scale=one(M), weight_scale=one(N), out_dtype=DT[out])
    assert torch.equal(y.cpu(), want.to(DT[out]))


@pytest.mark.parametrize('M,N,K', SUMS)
def test_sums_of_8_bit_products(M, N, K):
    print(f'[sums] {M}x{N}x{K}', flush=True)
    check_sums(M, N, K, 'f32')


# (those that are no tiles)
@pytest.mark.parametrize('M,N,K', [s for s in SUMS if s[0] <= 300 or s[1] % 8])
def test_sums_of_8_bit_products_in_blocks(M, N, K):
    """Where the matrix instructions' rate is no bound the bf16 output has them too."""
    print(f'[sums] {M}x{N}x{K}', flush=True)
    check_sums(M, N, K, 'bf16')


@pytest.mark.parametrize('rows', [3, 5000])
@pytest.mark.parametrize('N,K', [(256, 256), (257, 256)])
def test_every_8_bit_number(rows, N, K):
    """Each of the 256 codes on either side of a one."""
    codes = torch.arange(256, dtype=torch.uint8).view(DT['e4m3'])
    want = codes.float()
    hot = torch.zeros(rows, K)
    hot[:, 0] = 1
    w = torch.zeros(N, K, dtype=torch.uint8)
    w[:256, 0] = torch.arange(256, dtype=torch.uint8)
    one = lambda n: torch.ones(n, device=DEV)   # noqa: E731
    run = lambda x, w: gdn2.linear_fwd(x, w, x_scale=one(len(x)), weight_scale=one(len(w)), out_dtype=torch.float32)[0]   # noqa: E731
    y = run(hot.to(DT['e4m3']).to(DEV), w.view(DT['e4m3']).to(DEV)).cpu()
    assert torch.equal(torch.nan_to_num(y[:, :256], 999.0), torch.nan_to_num(want, 999.0).expand(rows, 256))
    x = torch.zeros(rows, K, dtype=torch.uint8)
    at = torch.arange(rows) % 256
    x[:, 0] = at.to(torch.uint8)
    hot = torch.zeros(N, K)
    hot[:, 0] = 1
    y = run(x.view(DT['e4m3']).to(DEV), hot.to(DT['e4m3']).to(DEV)).cpu()
    assert torch.equal(torch.nan_to_num(y, 999.0), torch.nan_to_num(want[at], 999.0)[:, None].expand(rows, N))
