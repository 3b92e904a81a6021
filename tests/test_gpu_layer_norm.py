"""gdn2_layer_norm_fwd / gdn2_layer_norm_bwd against float64: every way a row is
held (part of a wave, a wave, a workgroup, read again), odd widths, types, and
rows that are hard on the statistics."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip('torch')
if not torch.cuda.is_available():
    pytest.skip('no GPU', allow_module_level=True)

import gated_delta_rule_wy_amd as gdn2  # noqa: E402
import gdn2_inputs as gi  # noqa: E402
import operator_reference as ref  # noqa: E402
from gpu_util import DEV  # noqa: E402

DT = {'bf16': torch.bfloat16, 'f32': torch.float32}
WIDTHS = [1, 2, 7, 8, 16, 17, 63, 64, 65, 120, 128, 250, 256, 257, 512, 1000, 1001, 1024, 1025, 2048, 2056, 4096, 4100,
          8192, 8200, 16384, 16385, 16392, 20000]


def make(seed, rows, cols, dtype, scale=None, offset=None):
    rng = np.random.default_rng(seed)
    rnd = gi.bf16_round if dtype == 'bf16' else (lambda x: np.asarray(x, np.float32))
    s = 0.5 + 2 * rng.random((rows, 1)) if scale is None else scale
    m = rng.standard_normal((rows, 1)) if offset is None else offset
    x = rnd((rng.standard_normal((rows, cols)) * s + m).astype(np.float32))
    r = rnd(rng.standard_normal((rows, cols)).astype(np.float32))
    dy = rnd(rng.standard_normal((rows, cols)).astype(np.float32))
    w = (1 + 0.2 * rng.standard_normal(cols)).astype(np.float32)
    b = (0.2 * rng.standard_normal(cols)).astype(np.float32)
    return x, r, dy, w, b


def gpu(x, dtype='f32'):
    return torch.from_numpy(x).to(DEV).to(DT[dtype])


def back(t):
    return t.float().cpu().numpy()


def fwd(x, w, b, r, dtype, out='f32', **kw):
    return gdn2.layer_norm_fwd(gpu(x, dtype), gpu(w), None if b is None else gpu(b), None if r is None else gpu(r, dtype),
                               out_dtype=DT[out], **kw)


@pytest.mark.parametrize('dtype', ['bf16', 'f32'])
@pytest.mark.parametrize('cols', WIDTHS)
def test_forward_widths(cols, dtype):
    print(f'[forward] cols={cols} {dtype}', flush=True)
    x, r, _, w, b = make(cols, 5, cols, dtype)
    for res, bias in ((r, b), (None, None)):
        y, h = fwd(x, w, bias, res, dtype, output_sum=True)
        ry, rh = ref.layer_norm_fwd(x, w, bias, res, in_dtype=dtype)
        ref.check('y', back(y), ry)
        ref.check('h', back(h), rh)


@pytest.mark.parametrize('dtype', ['bf16', 'f32'])
@pytest.mark.parametrize('cols', WIDTHS)
def test_backward_widths(cols, dtype):
    print(f'[backward] cols={cols} {dtype}', flush=True)
    h, s, dy, w, _ = make(cols + 1, 9, cols, dtype)
    for dsum in (None, s):
        g = gdn2.layer_norm_bwd(gpu(dy, dtype), gpu(h, dtype), gpu(w), dsum=None if dsum is None else gpu(dsum, dtype))
        want = ref.layer_norm_bwd(dy, h, w, dsum, dtype=dtype)
        for n in want:
            ref.check(n, back(g[n]), want[n])


@pytest.mark.parametrize('rows', [1, 2, 3, 4, 31, 33, 257, 2500, 9000])
@pytest.mark.parametrize('cols', [24, 256, 2048, 999])
def test_row_counts(rows, cols):
    """Fewer rows than a workgroup takes, and more than all workgroups take at once."""
    print(f'[rows] {rows}x{cols}', flush=True)
    x, r, dy, w, b = make(rows, rows, cols, 'bf16')
    y, h = fwd(x, w, b, r, 'bf16', 'bf16', output_sum=True)
    ry, rh = ref.layer_norm_fwd(x, w, b, r, out_dtype='bf16', in_dtype='bf16')
    ref.check('y', back(y), ry)
    ref.check('h', back(h), rh)
    g = gdn2.layer_norm_bwd(gpu(dy, 'bf16'), gpu(x, 'bf16'), gpu(w))
    want = ref.layer_norm_bwd(dy, x, w, dtype='bf16')
    for n in want:
        ref.check(n, back(g[n]), want[n])


@pytest.mark.parametrize('din,dout', [('bf16', 'f32'), ('f32', 'bf16')])
def test_mixed_types(din, dout):
    x, r, _, w, b = make(1, 6, 384, din)
    dy = make(2, 6, 384, dout)[2]
    y, _ = fwd(x, w, b, r, din, dout)
    assert y.dtype == DT[dout]
    ref.check('y', back(y), ref.layer_norm_fwd(x, w, b, r, out_dtype=dout)[0])
    g = gdn2.layer_norm_bwd(gpu(dy, dout), gpu(x, din), gpu(w))
    assert g['x'].dtype == DT[din]
    want = ref.layer_norm_bwd(dy, x, w, dtype=din)
    for n in want:
        ref.check(n, back(g[n]), want[n])


@pytest.mark.parametrize('cols', [64, 2048, 1001])
@pytest.mark.parametrize('scale,offset', [(1e-3, 1000.0), (0.0, 3.0), (1e15, 0.0), (1e-15, 0.0)])
def test_hard_rows(cols, scale, offset):
    """A mean far larger than the spread, constant rows, very large and very small values."""
    x, _, dy, w, b = make(3, 4, cols, 'f32', scale, offset)
    y, _ = fwd(x, w, b, None, 'f32')
    ref.check('y', back(y), ref.layer_norm_fwd(x, w, b)[0])
    g = gdn2.layer_norm_bwd(gpu(dy), gpu(x), gpu(w))
    want = ref.layer_norm_bwd(dy, x, w)
    for n in want:
        ref.check(n, back(g[n]), want[n])


def test_not_finite_stays_in_its_row():
    x, _, dy, w, b = make(4, 40, 96, 'f32')
    bad = x.copy()
    bad[7, 5], bad[20, 0] = np.nan, np.inf
    keep = [i for i in range(40) if i not in (7, 20)]
    y, _ = fwd(bad, w, b, None, 'f32')
    ry, tol = ref.layer_norm_fwd(x, w, b)[0]
    ref.check('y', back(y)[keep], (ry[keep], tol[keep]))
    assert np.all(np.isnan(back(y)[[7, 20]]))
    g = gdn2.layer_norm_bwd(gpu(dy), gpu(bad), gpu(w))
    rx, tol = ref.layer_norm_bwd(dy, x, w)['x']
    ref.check('dh', back(g['x'])[keep], (rx[keep], tol[keep]))


def test_no_rows():
    w = torch.ones(48, device=DEV)
    x = torch.empty((0, 48), device=DEV)
    y, _ = gdn2.layer_norm_fwd(x, w)
    g = gdn2.layer_norm_bwd(x, x, w)
    assert y.shape == (0, 48) and g['x'].shape == (0, 48)
    assert torch.all(g['weight'] == 0) and torch.all(g['bias'] == 0)


@pytest.mark.parametrize('cols', [2048, 1001, 20000])
def test_in_place(cols):
    """y over x and the sum over the residual; the gradient over dy."""
    x, r, dy, w, b = make(5, 7, cols, 'bf16')
    gx, gr = gpu(x, 'bf16'), gpu(r, 'bf16')
    y, h = gdn2.layer_norm_fwd(gx.clone(), gpu(w), gpu(b), gr, output_sum=True)
    x2, r2 = gx.clone(), gr.clone()
    y2, h2 = gdn2.layer_norm_fwd(x2, gpu(w), gpu(b), r2, out=x2, sum_out=r2)
    assert y2 is x2 and h2 is r2 and torch.equal(y, y2) and torch.equal(h, h2)
    d = gpu(dy, 'bf16')
    g = gdn2.layer_norm_bwd(d, gx, gpu(w))
    d2 = d.clone()
    g2 = gdn2.layer_norm_bwd(d2, gx, gpu(w), out=d2)
    assert all(torch.equal(g[n], g2[n]) for n in g)


@pytest.mark.parametrize('dtype', ['bf16', 'f32'])
@pytest.mark.parametrize('cols', [1, 3, 9, 15, 65, 127, 129, 257, 521, 1025, 2049, 4097, 8191, 16383, 16385])
def test_in_place_odd_widths(cols, dtype):
    """Rows that do not fall into whole packs: what lanes hold twice is written as it is read, the rows around
    stay whole, and a row of NaN stays one row."""
    print(f'[in place] cols={cols} {dtype}', flush=True)
    x, r, dy, w, b = make(cols + 3, 37, cols, dtype)
    x[17] = np.nan
    gx, gr = gpu(x, dtype), gpu(r, dtype)
    y, h = gdn2.layer_norm_fwd(gx, gpu(w), gpu(b), gr, output_sum=True)
    bad = torch.isnan(y).any(1)
    assert bad[17] and int(bad.sum()) == 1 and bool(torch.isnan(y[17]).all())
    x2, r2 = gx.clone(), gr.clone()
    gdn2.layer_norm_fwd(x2, gpu(w), gpu(b), r2, out=x2, sum_out=r2)
    assert torch.equal(y.nan_to_num(7.), x2.nan_to_num(7.)) and torch.equal(h.nan_to_num(7.), r2.nan_to_num(7.))
    d, hr = gpu(dy, dtype), gr
    g = gdn2.layer_norm_bwd(d, hr, gpu(w))
    d2 = d.clone()
    g2 = gdn2.layer_norm_bwd(d2, hr, gpu(w), out=d2)
    assert all(torch.equal(g[n], g2[n]) for n in g)


def test_leading_axes_and_determinism():
    x, r, dy, w, b = make(6, 4 * 5 * 60, 136, 'bf16')
    sh = (4, 5, 60, 136)
    y, h = gdn2.layer_norm_fwd(gpu(x, 'bf16').view(sh), gpu(w), gpu(b), gpu(r, 'bf16').view(sh), output_sum=True)
    assert y.shape == h.shape == sh
    a = gdn2.layer_norm_bwd(gpu(dy, 'bf16').view(sh), h, gpu(w))
    c = gdn2.layer_norm_bwd(gpu(dy, 'bf16').view(sh), h, gpu(w))
    assert a['x'].shape == sh and all(torch.equal(a[n], c[n]) for n in a)


def test_gradient_is_that_of_the_forward():
    """Differences of the forward itself: sum(dy * y) along random directions."""
    rng = np.random.default_rng(8)
    x, r, dy, w, b = (a.astype(np.float64) for a in make(8, 6, 40, 'f32'))
    g = gdn2.layer_norm_bwd(gpu(dy.astype(np.float32)), gpu((x + r).astype(np.float32)), gpu(w.astype(np.float32)))
    step = 1e-2
    for name, at in (('x', x), ('weight', w), ('bias', b)):
        for _ in range(4):
            u = rng.standard_normal(at.shape)
            val = []
            for s in (step, -step):
                p = {'x': x, 'weight': w, 'bias': b}
                p[name] = at + s * u
                y, _ = fwd(p['x'].astype(np.float32), p['weight'].astype(np.float32), p['bias'].astype(np.float32),
                           r.astype(np.float32), 'f32')
                val.append((back(y).astype(np.float64) * dy).sum())
            slope = (val[0] - val[1]) / (2 * step)
            want = (back(g[name]).astype(np.float64) * u).sum()
            # second order in the step (third derivatives of order |u|^3 rstd^3 |dy|), and the forward's
            # rounding of about 1e-6 of each of 240 terms over the step
            size = np.abs(back(g[name]) * u).sum()
            assert abs(slope - want) <= 5e-3 * size + 240 * 1e-6 / step, (name, slope, want)


@pytest.mark.parametrize('cols', [2048, 1001])
def test_captured_and_replayed(cols):
    x, r, dy, w, b = (gpu(a, d) for a, d in zip(make(9, 300, cols, 'bf16'), ('bf16', 'bf16', 'bf16', 'f32', 'f32')))
    need = gdn2.lib().gdn2_layer_norm_bwd_workspace_bytes(300, cols)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)

    def step():
        y, h = gdn2.layer_norm_fwd(x, w, b, r, output_sum=True)
        return y, h, gdn2.layer_norm_bwd(dy, h, w, workspace=ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, h, g = step()
    for i in range(4):
        nx, nr, nd, _, _ = make(50 + i, 300, cols, 'bf16')
        for t, a in ((x, nx), (r, nr), (dy, nd)):
            t.copy_(gpu(a, 'bf16'))
        ey, eh = gdn2.layer_norm_fwd(x, w, b, r, output_sum=True)
        eg = gdn2.layer_norm_bwd(dy, eh, w)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, ey) and torch.equal(h, eh) and all(torch.equal(g[n], eg[n]) for n in g)


def test_other_stream():
    x, r, _, w, b = make(10, 64, 512, 'bf16')
    gx, gr, gw, gb = gpu(x, 'bf16'), gpu(r, 'bf16'), gpu(w), gpu(b)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        y, _ = gdn2.layer_norm_fwd(gx * 1, gw, gb, gr)
    side.synchronize()
    ref.check('y', back(y), ref.layer_norm_fwd(x, w, b, r, out_dtype='bf16')[0])


def test_past_32_bit_offsets():
    """More than 2^31 elements: the last rows against the same rows alone."""
    rows, cols = (1 << 31) // 2048 + 40, 2048
    x = torch.empty((rows, cols), dtype=torch.bfloat16, device=DEV)
    x[-64:] = gpu(make(11, 64, cols, 'bf16')[0], 'bf16')
    w = torch.ones(cols, device=DEV)
    y, _ = gdn2.layer_norm_fwd(x, w)
    few, _ = gdn2.layer_norm_fwd(x[-64:].contiguous(), w)
    assert torch.equal(y[-64:], few)
