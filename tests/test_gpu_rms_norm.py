"""gdn2_rms_norm_fwd / gdn2_rms_norm_bwd against float64: every way a row is held, odd widths,
types, the 8-bit output with its scales, and rows that are hard on them."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip('torch')
if not torch.cuda.is_available():
    pytest.skip('no GPU', allow_module_level=True)

import dense_reference as ref  # noqa: E402
import gated_delta_rule_wy_amd as gdn2  # noqa: E402
import gdn2_inputs as gi  # noqa: E402
import operator_reference as oref  # noqa: E402
from gpu_util import DEV  # noqa: E402

E4M3 = torch.float8_e4m3fn
DT = {'bf16': torch.bfloat16, 'f32': torch.float32, 'e4m3': E4M3}
WIDTHS = [1, 2, 7, 8, 16, 17, 63, 64, 65, 120, 128, 250, 256, 257, 512, 1000, 1001, 1024, 1025, 2048, 2056, 4096, 4100,
          8192, 8200, 16384, 16385, 16392, 20000]


def make(seed, rows, cols, dtype, scale=None):
    rng = np.random.default_rng(seed)
    rnd = gi.bf16_round if dtype == 'bf16' else (lambda x: np.asarray(x, np.float32))
    s = 0.5 + 2 * rng.random((rows, 1)) if scale is None else scale
    x = rnd((rng.standard_normal((rows, cols)) * s).astype(np.float32))
    r = rnd((rng.standard_normal((rows, cols)) * s).astype(np.float32))
    dy = rnd(rng.standard_normal((rows, cols)).astype(np.float32))
    w = (1 + 0.2 * rng.standard_normal(cols)).astype(np.float32)
    return x, r, dy, w


def gpu(x, dtype='f32'):
    return torch.from_numpy(x).to(DEV).to(DT[dtype])


def back(t):
    return t.float().cpu().numpy()


def check8(y, scale, h, want):
    wq, ws, wh = want
    assert y.dtype == E4M3 and scale.dtype == torch.float32
    oref.check('q', back(y), wq)
    oref.check('scale', back(scale), ws)
    if h is not None:
        oref.check('h', back(h), wh)


@pytest.mark.parametrize('dtype', ['bf16', 'f32'])
@pytest.mark.parametrize('cols', WIDTHS)
def test_forward_widths(cols, dtype):
    print(f'[forward] cols={cols} {dtype}', flush=True)
    x, r, _, w = make(cols, 5, cols, dtype)
    for res in (r, None):
        gr = None if res is None else gpu(res, dtype)
        y, h, s = gdn2.rms_norm_fwd(gpu(x, dtype), gpu(w), gr, output_sum=True, out_dtype=torch.float32)
        assert s is None
        wy, wh = ref.rms_norm_fwd(x, w, res, in_dtype=dtype)
        oref.check('y', back(y), wy)
        oref.check('h', back(h), wh)
        y, h, s = gdn2.rms_norm_fwd(gpu(x, dtype), gpu(w), gr, output_sum=True, out_dtype=E4M3)
        check8(y, s, h, ref.rms_norm_fwd(x, w, res, out_dtype='e4m3', in_dtype=dtype))


@pytest.mark.parametrize('dtype', ['bf16', 'f32'])
@pytest.mark.parametrize('cols', WIDTHS)
def test_backward_widths(cols, dtype):
    print(f'[backward] cols={cols} {dtype}', flush=True)
    h, s, dy, w = make(cols + 1, 9, cols, dtype)
    for dsum in (None, s):
        g = gdn2.rms_norm_bwd(gpu(dy, dtype), gpu(h, dtype), gpu(w), dsum=None if dsum is None else gpu(dsum, dtype))
        want = ref.rms_norm_bwd(dy, h, w, dsum, dtype=dtype)
        for n in want:
            oref.check(n, back(g[n]), want[n])


@pytest.mark.parametrize('rows', [1, 2, 3, 4, 31, 33, 257, 2500, 9000])
@pytest.mark.parametrize('cols', [24, 256, 2048, 999])
def test_row_counts(rows, cols):
    """Fewer rows than a workgroup takes, and more than all workgroups take at once."""
    print(f'[rows] {rows}x{cols}', flush=True)
    x, r, dy, w = make(rows, rows, cols, 'bf16')
    y, h, s = gdn2.rms_norm_fwd(gpu(x, 'bf16'), gpu(w), gpu(r, 'bf16'), output_sum=True, out_dtype=E4M3)
    check8(y, s, h, ref.rms_norm_fwd(x, w, r, out_dtype='e4m3', in_dtype='bf16'))
    y, _, _ = gdn2.rms_norm_fwd(gpu(x, 'bf16'), gpu(w), gpu(r, 'bf16'))
    oref.check('y', back(y), ref.rms_norm_fwd(x, w, r, out_dtype='bf16')[0])
    g = gdn2.rms_norm_bwd(gpu(dy, 'bf16'), gpu(x, 'bf16'), gpu(w))
    want = ref.rms_norm_bwd(dy, x, w, dtype='bf16')
    for n in want:
        oref.check(n, back(g[n]), want[n])


@pytest.mark.parametrize('din,dout', [('bf16', 'f32'), ('f32', 'bf16'), ('f32', 'e4m3')])
def test_mixed_types(din, dout):
    x, r, _, w = make(1, 6, 384, din)
    y, h, s = gdn2.rms_norm_fwd(gpu(x, din), gpu(w), gpu(r, din), out_dtype=DT[dout], output_sum=True)
    if dout == 'e4m3':
        check8(y, s, h, ref.rms_norm_fwd(x, w, r, out_dtype='e4m3', in_dtype=din))
        return
    oref.check('y', back(y), ref.rms_norm_fwd(x, w, r, out_dtype=dout)[0])
    dy = make(2, 6, 384, dout)[2]
    g = gdn2.rms_norm_bwd(gpu(dy, dout), gpu(x, din), gpu(w))
    assert g['x'].dtype == DT[din]
    want = ref.rms_norm_bwd(dy, x, w, dtype=din)
    for n in want:
        oref.check(n, back(g[n]), want[n])


@pytest.mark.parametrize('cols', [64, 2048, 1001, 20000])
@pytest.mark.parametrize('scale', [1e15, 1e-3, 1e-15, 1e-30])
def test_hard_rows(cols, scale):
    """Very large values, and very small ones (down to where eps is all of the mean)."""
    x, _, dy, w = make(3, 4, cols, 'f32', scale)
    oref.check('y', back(gdn2.rms_norm_fwd(gpu(x), gpu(w))[0]), ref.rms_norm_fwd(x, w)[0])
    y, _, s = gdn2.rms_norm_fwd(gpu(x), gpu(w), out_dtype=E4M3)
    check8(y, s, None, ref.rms_norm_fwd(x, w, out_dtype='e4m3'))
    g = gdn2.rms_norm_bwd(gpu(dy), gpu(x), gpu(w))
    want = ref.rms_norm_bwd(dy, x, w)
    for n in want:
        oref.check(n, back(g[n]), want[n])


def test_rows_of_zeros_and_one_large_element():
    x = np.zeros((3, 96), np.float32)
    x[1, 40] = 5.0
    x[2] = 1e-40
    w = np.ones(96, np.float32)
    y, _, s = gdn2.rms_norm_fwd(gpu(x), gpu(w), out_dtype=E4M3)
    y, s = back(y), back(s)
    assert np.all(y[0] == 0) and s[0] == np.float32(2.0 ** -126)
    assert y[1, 40] == 448 and np.count_nonzero(y[1]) == 1
    assert np.all(np.isfinite(y)) and np.all(np.isfinite(s))


def test_not_finite_stays_in_its_row():
    x, _, dy, w = make(4, 40, 96, 'f32')
    bad = x.copy()
    bad[7, 5], bad[20, 0] = np.nan, np.inf
    keep = [i for i in range(40) if i not in (7, 20)]
    y = back(gdn2.rms_norm_fwd(gpu(bad), gpu(w))[0])
    ry, tol = ref.rms_norm_fwd(x, w)[0]
    oref.check('y', y[keep], (ry[keep], tol[keep]))
    assert np.all(np.isnan(y[7])) and np.isnan(y[20, 0])
    q, _, s = gdn2.rms_norm_fwd(gpu(bad), gpu(w), out_dtype=E4M3)
    (rq, tq), (rs, ts), _ = ref.rms_norm_fwd(x, w, out_dtype='e4m3')
    oref.check('q', back(q)[keep], (rq[keep], tq[keep]))
    oref.check('scale', back(s)[keep], (rs[keep], ts[keep]))
    assert np.all(np.isnan(back(q)[7]))
    g = gdn2.rms_norm_bwd(gpu(dy), gpu(bad), gpu(w))
    rx, tol = ref.rms_norm_bwd(dy, x, w)['x']
    oref.check('dh', back(g['x'])[keep], (rx[keep], tol[keep]))


def test_no_rows_and_one_axis():
    w = torch.ones(48, device=DEV)
    x = torch.empty((0, 48), device=DEV)
    y, _, s = gdn2.rms_norm_fwd(x, w, out_dtype=E4M3)
    assert y.shape == (0, 48) and s.shape == (0,)
    g = gdn2.rms_norm_bwd(x, x, w)
    assert g['x'].shape == (0, 48) and torch.all(g['weight'] == 0)
    v = torch.randn(48, device=DEV)
    y, _, s = gdn2.rms_norm_fwd(v, w, out_dtype=E4M3)
    assert y.shape == (48,) and s.shape == ()


@pytest.mark.parametrize('cols', [2048, 1001, 20000])
def test_in_place(cols):
    x, r, dy, w = make(5, 70, cols, 'bf16')
    gx, gr, gw = gpu(x, 'bf16'), gpu(r, 'bf16'), gpu(w)
    y, h, _ = gdn2.rms_norm_fwd(gx.clone(), gw, gr, output_sum=True)
    x2, r2 = gx.clone(), gr.clone()
    y2, h2, _ = gdn2.rms_norm_fwd(x2, gw, r2, out=x2, sum_out=r2)
    assert y2 is x2 and h2 is r2 and torch.equal(y, y2) and torch.equal(h, h2)
    x3 = gx.clone()
    y3, h3, _ = gdn2.rms_norm_fwd(x3, gw, gr, sum_out=x3, out_dtype=E4M3)
    assert torch.equal(h3, h)
    d = gpu(dy, 'bf16')
    g = gdn2.rms_norm_bwd(d, gx, gw)
    for over in range(2):
        a, b = d.clone(), gx.clone()
        g2 = gdn2.rms_norm_bwd(a, b, gw, out=(a, b)[over])
        assert torch.equal(g2['x'], g['x']) and torch.equal(g2['weight'], g['weight'])


def test_nothing_is_written_beyond_the_tensors():
    for cols in (7, 64, 999, 2048, 20000):
        x, r, _, w = make(6, 3, cols, 'bf16')
        ybuf = torch.full((3 * cols + 64,), 1.0, device=DEV).to(E4M3)
        sbuf, hbuf = torch.full((3 + 16,), 2.0, device=DEV), torch.full((3 * cols + 64,), 3.0, device=DEV, dtype=torch.bfloat16)
        gdn2.rms_norm_fwd(gpu(x, 'bf16'), gpu(w), gpu(r, 'bf16'), out=ybuf[:3 * cols].view(3, cols), scale_out=sbuf[:3],
                          sum_out=hbuf[:3 * cols].view(3, cols))
        assert torch.all(ybuf[3 * cols:].float() == 1) and torch.all(sbuf[3:] == 2) and torch.all(hbuf[3 * cols:] == 3)


@pytest.mark.parametrize('cols', [2048, 1001])
def test_captured_with_its_gradient(cols):
    torch.manual_seed(1)
    x, r, dy = (torch.randn(300, cols, device=DEV, dtype=torch.bfloat16) for _ in range(3))
    w = 1 + 0.1 * torch.randn(cols, device=DEV)
    ws = torch.empty(gdn2.lib().gdn2_rms_norm_bwd_workspace_bytes(300, cols), dtype=torch.uint8, device=DEV)

    def step():
        y, h, s = gdn2.rms_norm_fwd(x, w, r, output_sum=True, out_dtype=E4M3)
        return [y.view(torch.uint8), h, s, *gdn2.rms_norm_bwd(dy, h, w, workspace=ws).values()]

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


def test_binding_refuses():
    x, w = torch.zeros(4, 8, device=DEV), torch.ones(8, device=DEV)
    for err, args, kw in [
            (ValueError, (torch.zeros(8, 4, device=DEV).t(), w), {}), (TypeError, (x.half(), w), {}), (ValueError, (x, w[:4]), {}),
            (TypeError, (x, w.bfloat16()), {}), (TypeError, (x, w, x.bfloat16()), {}), (TypeError, (x, w), dict(out_dtype=torch.float16)),
            (ValueError, (x, w), dict(scale_out=torch.ones(4, device=DEV))),
            (ValueError, (x, w), dict(out_dtype=E4M3, scale_out=torch.ones(3, device=DEV))), (gdn2.Gdn2Error, (x, w), dict(eps=0.0)),
            (ValueError, (x, w), dict(out=x[:2])), (gdn2.Gdn2Error, (x, w), dict(out=x, sum_out=x))]:
        with pytest.raises(err):
            gdn2.rms_norm_fwd(*args, **kw)
    for err, args, kw in [(TypeError, (x.half(), x, w), {}), (ValueError, (x[:2], x, w), {}), (ValueError, (x, x, w), dict(dsum=x[:2])),
                          (ValueError, (x, x, w), dict(workspace=torch.empty(1 << 20, dtype=torch.uint8)))]:
        with pytest.raises(err):
            gdn2.rms_norm_bwd(*args, **kw)


@pytest.mark.parametrize('cols', [5, 64, 2048, 2049, 5000, 20000])
@pytest.mark.parametrize('dtype', [torch.bfloat16, torch.float32])
def test_not_a_number_stays_in_its_row(cols, dtype):
    """In 8 bits with the least scale."""
    g = torch.Generator().manual_seed(cols)
    x, w = torch.randn(9, cols, generator=g).to(dtype).to(DEV), torch.ones(cols, device=DEV)
    e4m3 = torch.float8_e4m3fn
    y0, _, s0 = gdn2.rms_norm_fwd(x, w, out_dtype=e4m3)
    x[4, cols // 2] = float('nan')
    y, _, s = gdn2.rms_norm_fwd(x, w, out_dtype=e4m3)
    others = [r for r in range(9) if r != 4]
    assert torch.equal(y.view(torch.uint8)[others], y0.view(torch.uint8)[others]) and torch.equal(s[others], s0[others])
    assert torch.all(torch.isnan(y[4].float())) and float(s[4]) == 2.0 ** -126
    assert torch.all(torch.isnan(gdn2.rms_norm_fwd(x, w)[0][4].float()))
