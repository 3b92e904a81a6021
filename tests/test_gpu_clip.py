"""gdn2_grad_norm / gdn2_clip_grads against float64: lists longer than a launch takes, tensors without
elements, at any element's address, of both types, values at the ends of the range."""
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

BF, F = torch.bfloat16, torch.float32
NAME = {BF: 'bf16', F: 'f32'}


def back(t):
    return t.float().cpu().numpy()


def make(seed, sizes, types, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(n, generator=g) * scale).to(t).to(DEV) for n, t in zip(sizes, types)]


def check(grads, max_norm, out=None, **kw):
    before = [back(g) for g in grads]
    n, tol = ref.grad_norm(before)
    norm = gdn2.clip_grads(grads, max_norm, out=out, **kw)
    if 'norm' not in kw:
        assert norm.shape == ()
        # (3.4028236e38 and more is infinity as a float)
        assert abs(float(norm) - n) <= tol if n < 3.4028235e38 else float(norm) == np.inf
    where = grads if out is None else out
    for t, w in zip(where, ref.clip(before, max_norm, [NAME[t.dtype] for t in where], kw.get('norm'))):
        oref.check('out', back(t), w)
    if out is not None:
        assert all(np.array_equal(back(g), b) for g, b in zip(grads, before) if not any(g is o for o in out))


@pytest.mark.parametrize('max_norm', [0.1, 1e6, 0.0])
@pytest.mark.parametrize('sizes', [[1], [7], [8], [16383, 16384, 16385], [0, 5, 0, 3], [100000, 1, 33, 2048 * 64], list(range(1, 150)),
                                   [3, 0] * 130, [40000] * 70])
def test_in_place(sizes, max_norm):
    print(f'[clip] {len(sizes)} tensors, {sum(sizes)} elements, {max_norm}', flush=True)
    types = [(BF, F)[i % 3 == 0] for i in range(len(sizes))]
    check(make(len(sizes), sizes, types), max_norm)


@pytest.mark.parametrize('out', ['bf16', 'f32', 'mixed', 'some in place'])
@pytest.mark.parametrize('max_norm', [0.5, 1e6])
def test_into_others(out, max_norm):
    sizes = [1000, 3, 0, 16384 * 3 + 5, 77, 4096]
    grads = make(3, sizes, [BF, F, BF, F, BF, F])
    ot = {'bf16': [BF] * 6, 'f32': [F] * 6}.get(out, [F, BF, F, BF, BF, F])
    o = [torch.full((n,), 9.0, dtype=t, device=DEV) for n, t in zip(sizes, ot)]
    if out == 'some in place':
        o[3], o[4] = grads[3], grads[4]
    check(grads, max_norm, o)


def test_addresses_of_any_element_and_nothing_beyond():
    """Views into one buffer, with gaps that stay."""
    for dt in (BF, F):
        buf = torch.randn(200000, device=DEV).to(dt)
        keep = buf.clone()
        spans = [(1, 20), (23, 24), (30, 20031), (20035, 60000), (60001, 200000 - 3)]
        views = [buf[a:b] for a, b in spans]
        check(views, 0.25)
        gaps = torch.ones(200000, dtype=torch.bool, device=DEV)
        for a, b in spans:
            gaps[a:b] = False
        assert torch.equal(buf[gaps], keep[gaps])


def test_norm_alone_and_given():
    grads = make(5, [5000, 300, 70000], [F, BF, F])
    n, tol = ref.grad_norm([back(g) for g in grads])
    norm = gdn2.grad_norm(grads)
    assert abs(float(norm) - n) <= tol
    assert float(gdn2.grad_norm([torch.empty(0, device=DEV)])) == 0
    # a norm over more than these tensors
    both = (norm.double() * 2).float()
    check(grads, 1.0, norm=both)
    assert float(both) == float(norm.double() * 2)


@pytest.mark.parametrize('scale', [1e30, 3e37, 1e-30, 1e-42])
def test_ends_of_the_range(scale):
    """Squares that no fp32 holds."""
    check(make(6, [3000, 17], [F, F], scale), scale / 10)


def test_not_finite():
    for bad, what in ((np.nan, np.isnan), (np.inf, None)):
        g = make(7, [100, 50], [F, BF])
        g[0][3] = float(bad)
        norm = gdn2.clip_grads(g, 1.0)
        assert not np.isfinite(float(norm))
        if what:
            assert all(np.all(np.isnan(back(t))) for t in g)
        else:   # max_norm / infinity is 0
            assert np.isnan(back(g[0])[3]) and np.all(back(g[1]) == 0) and np.all(np.delete(back(g[0]), 3) == 0)


def test_no_tensor_at_all_to_scale():
    z = torch.empty(0, device=DEV)
    assert float(gdn2.clip_grads([z, z], 1.0)) == 0


def test_below_the_largest_norm_nothing_is_written():
    """Same bits, NaN's payload and negative zeros included, in place and copied."""
    g = make(8, [70000], [BF])[0]
    g[5] = -0.0
    before = g.view(torch.int16).clone()
    o = torch.zeros_like(g)
    gdn2.clip_grads([g], 1e9, out=[o])
    gdn2.clip_grads([g], 1e9)
    assert torch.equal(g.view(torch.int16), before) and torch.equal(o.view(torch.int16), before)


def test_same_bits_and_captured():
    grads = make(9, [70000, 5, 300000, 16384], [F, BF, BF, F])
    outs = [torch.empty(g.shape, dtype=F, device=DEV) for g in grads]
    ws = torch.empty(gdn2.lib().gdn2_clip_grads_workspace_bytes(), dtype=torch.uint8, device=DEV)
    step = lambda: gdn2.clip_grads(grads, 1.0, out=outs, workspace=ws)   # noqa: E731
    n1 = step().clone()
    first = [o.clone() for o in outs]
    assert torch.equal(step(), n1) and all(torch.equal(a, b) for a, b in zip(first, outs))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = step()
    for i in range(4):
        grads[2].copy_(torch.randn_like(grads[2]) * (i + 1))
        graph.replay()
        torch.cuda.synchronize()
        got, gn = [o.clone() for o in outs], norm.clone()
        assert torch.equal(step(), gn) and all(torch.equal(a, b) for a, b in zip(got, outs)), i


def test_offsets_beyond_32_bits():
    n = (1 << 31) + 12345
    g = torch.full((n,), 0.5, dtype=BF, device=DEV)
    g[-1] = 3.0
    norm = gdn2.clip_grads([g], 1.0)
    want = np.sqrt(0.25 * (n - 1) + 9.0)
    assert abs(float(norm) - want) <= 2 * oref.U * want
    c = 1.0 / (want + 1e-6)
    for at, v in ((0, 0.5), (1 << 30, 0.5), (1 << 31, 0.5), (n - 2, 0.5), (n - 1, 3.0)):
        assert abs(float(g[at]) - v * c) <= (2.0 ** -8 + 1e-6) * v * c


def test_binding_refuses():
    g = torch.ones(8, device=DEV)
    for err, args, kw in [
            (ValueError, ([], 1.0), {}), (TypeError, ([g.half()], 1.0), {}), (ValueError, ([torch.ones(4, 4, device=DEV)[:, ::2]], 1.0), {}),
            (ValueError, ([g, g.cpu()], 1.0), {}), (ValueError, ([g], 1.0), dict(out=[g, g])), (ValueError, ([g], 1.0), dict(out=[g[:4]])),
            (ValueError, ([g], 1.0), dict(norm=torch.ones(2, device=DEV))), (ValueError, ([g], 1.0), dict(norm=torch.ones(()))),
            (gdn2.Gdn2Error, ([g, g], 1.0), {}), (gdn2.Gdn2Error, ([g, g[4:]], 1.0), {}), (gdn2.Gdn2Error, ([g], -1.0), {}),
            (gdn2.Gdn2Error, ([g], float('nan')), {}), (gdn2.Gdn2Error, ([g], 1.0), dict(norm=g[:1])),
            (ValueError, ([g], 1.0), dict(workspace=torch.empty(1 << 20, dtype=torch.uint8)))]:
        with pytest.raises(err):
            gdn2.clip_grads(*args, **kw)


def test_norm_of_gradients_that_overlap():
    """Nothing is written to them: one tensor twice, and a part of it, count as often as they are given."""
    g = make(10, [50000], [BF])[0]
    grads = [g, g, g[100:20000]]
    n, tol = ref.grad_norm([back(t) for t in grads])
    assert abs(float(gdn2.grad_norm(grads)) - n) <= tol


def test_norm_refuses_a_workspace_within_a_gradient():
    g = torch.ones(8192, device=DEV)
    with pytest.raises(gdn2.Gdn2Error):
        gdn2.grad_norm([g], workspace=g[1024:])
    assert torch.all(g == 1)


@pytest.mark.parametrize('max_norm', [1e-3, 1e-6, 1e-30, 1e-37])
@pytest.mark.parametrize('types', [[F, F], [BF, F]])
def test_factors_below_the_smallest_float(types, max_norm):
    """Gradients near the range's end and a small largest norm: their quotient is no normal number, the results are."""
    check(make(11, [3000, 17], types, 3e37), max_norm)
    grads = make(12, [20000, 33], types, 1e37)
    check(grads, max_norm, [torch.zeros_like(g, dtype=F) for g in grads])
