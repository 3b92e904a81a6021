"""Calls that the dense operators refuse, on the CPU: every check runs on the host before
anything is launched, so the made-up addresses below never reach a kernel."""
import ctypes

import pytest
import torch

import gated_delta_rule_wy_amd as gdn2

P = 0x10000
OK, INVALID, UNSUPPORTED, WORKSPACE = (gdn2.GDN2_OK, gdn2.GDN2_ERR_INVALID, gdn2.GDN2_ERR_UNSUPPORTED,
                                       gdn2.GDN2_ERR_WORKSPACE)
F32, BF16, E4M3 = gdn2.GDN2_F32, gdn2.GDN2_BF16, gdn2.GDN2_E4M3
lib = gdn2.lib()


def addresses(names):
    return {n: (i + 1) * P for i, n in enumerate(names.split())}


def linear_fwd(**kw):
    a = dict(x=P, w=2 * P, b=3 * P, r=4 * P, sx=None, sw=None, y=5 * P, z=6 * P, rows=4, K=100, N=60, act=1, dt=BF16, odt=BF16)
    a.update(kw)
    return lib.gdn2_linear_fwd(*(a[n] for n in a))


Q = dict(dt=E4M3, sx=7 * P, sw=8 * P, z=None)


@pytest.mark.parametrize('kw,status', [
    (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(y=None), INVALID),
    (dict(x=P + 8), INVALID), (dict(r=P + 4), INVALID), (dict(b=P + 4), INVALID), (dict(z=P + 2), INVALID),
    (dict(rows=-1), INVALID), (dict(K=0), INVALID), (dict(N=0), INVALID), (dict(N=-5), INVALID),
    (dict(act=-1), INVALID), (dict(act=4), INVALID), (dict(dt=3), INVALID), (dict(odt=E4M3), INVALID), (dict(odt=-1), INVALID),
    (dict(sx=7 * P), INVALID), (dict(sw=7 * P), INVALID),               # scales belong to 8 bits
    (dict(Q, sx=None), INVALID), (dict(Q, sw=None), INVALID), (dict(Q, z=6 * P), INVALID), (dict(Q, sx=7 * P + 4), INVALID),
    (dict(K=(1 << 20) + 1), UNSUPPORTED), (dict(N=(1 << 20) + 1), UNSUPPORTED), (dict(rows=1 << 31), UNSUPPORTED),
    (dict(rows=1 << 30, N=1 << 12), UNSUPPORTED),
    (dict(y=P), INVALID), (dict(y=2 * P), INVALID), (dict(y=3 * P), INVALID), (dict(y=6 * P), INVALID),
    (dict(z=P), INVALID), (dict(z=2 * P), INVALID), (dict(z=4 * P), INVALID), (dict(Q, y=7 * P), INVALID),
    (dict(Q, y=8 * P), INVALID)])
def test_linear_fwd_rejects(kw, status):
    assert linear_fwd(**kw) == status


def test_linear_fwd_of_no_rows():
    assert linear_fwd(rows=0, x=None, y=None, z=None, r=None) == OK


def linear_bwd(**kw):
    a = dict(dy=P, x=2 * P, w=3 * P, z=4 * P, dx=5 * P, dw=6 * P, db=7 * P, rows=4, K=100, N=60, act=1, dt=BF16, ddt=F32, ws=8 * P,
             wsb=1 << 30)
    a.update(kw)
    return lib.gdn2_linear_bwd(*(a[n] for n in a))


LB = lib.gdn2_linear_bwd_workspace_bytes


@pytest.mark.parametrize('kw,status', [
    (dict(dy=None), INVALID), (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(z=None), INVALID),
    (dict(dx=None, dw=None, db=None), INVALID), (dict(db=P + 4), INVALID), (dict(dw=P + 8), INVALID),
    (dict(rows=-1), INVALID), (dict(K=0), INVALID), (dict(act=9), INVALID), (dict(dt=E4M3), INVALID), (dict(ddt=E4M3), INVALID),
    (dict(rows=(1 << 22) + 1), UNSUPPORTED), (dict(N=1 << 21), UNSUPPORTED),
    (dict(ws=None), WORKSPACE), (dict(wsb=LB(4, 100, 60, 1, BF16, F32, 1, 1, 1) - 1), WORKSPACE)])
def test_linear_bwd_rejects(kw, status):
    assert linear_bwd(**kw) == status


def test_linear_bwd_rejects_an_output_that_is_another_argument():
    at = addresses('dy x w z dx dw db ws')
    for out in ('dx', 'dw', 'db', 'ws'):
        for name, p in at.items():
            if name != out:
                assert linear_bwd(**{**at, out: p}) == INVALID, (out, name)


def test_linear_bwd_workspace():
    assert LB(4, 100, 60, 0, F32, F32, 0, 0, 1) > 0 and LB(0, 100, 60, 0, F32, F32, 1, 1, 1) > 0
    assert LB(4, 100, 60, 7, F32, F32, 1, 1, 1) == 0 and LB(4, 0, 60, 0, F32, F32, 1, 1, 1) == 0
    assert LB(4, 100, 60, 0, E4M3, F32, 1, 1, 1) == 0 and LB((1 << 22) + 1, 8, 8, 0, F32, F32, 1, 1, 1) == 0
    # nothing is turned or copied where its gradient is not asked for
    assert LB(4096, 512, 512, 0, BF16, BF16, 1, 0, 0) < LB(4096, 512, 512, 0, BF16, BF16, 1, 1, 0)


def rms_fwd(**kw):
    a = dict(x=P, r=2 * P, w=3 * P, y=4 * P, sc=None, s=5 * P, rows=4, cols=100, eps=1e-5, dt=BF16, odt=F32)
    a.update(kw)
    return lib.gdn2_rms_norm_fwd(*(a[n] for n in a))


def rms_bwd(**kw):
    a = dict(dy=P, h=2 * P, w=3 * P, ds=4 * P, dh=5 * P, dw=6 * P, rows=4, cols=100, eps=1e-5, dt=BF16, odt=F32, ws=7 * P, wsb=1 << 30)
    a.update(kw)
    return lib.gdn2_rms_norm_bwd(*(a[n] for n in a))


SIZES = [(dict(w=None), INVALID), (dict(rows=-1), INVALID), (dict(cols=0), INVALID), (dict(eps=0.0), INVALID),
         (dict(eps=-1.0), INVALID), (dict(eps=float('nan')), INVALID), (dict(eps=float('inf')), INVALID), (dict(dt=E4M3), INVALID),
         (dict(dt=5), INVALID), (dict(odt=5), INVALID), (dict(w=P + 8), INVALID), (dict(cols=(1 << 20) + 1), UNSUPPORTED),
         (dict(rows=(1 << 40) + 1), UNSUPPORTED)]


@pytest.mark.parametrize('kw,status', SIZES + [
    (dict(x=None), INVALID), (dict(y=None), INVALID), (dict(s=P + 2), INVALID), (dict(s=4 * P), INVALID),
    (dict(sc=6 * P), INVALID), (dict(odt=E4M3), INVALID),                # a scale with 8 bits, and only then
    (dict(odt=E4M3, sc=6 * P + 4), INVALID), (dict(odt=E4M3, sc=P), INVALID), (dict(odt=E4M3, sc=4 * P), INVALID),
    (dict(odt=E4M3, sc=6 * P, y=P), INVALID), (dict(y=P), INVALID), (dict(y=3 * P), INVALID), (dict(s=3 * P), INVALID)])
def test_rms_norm_fwd_rejects(kw, status):
    assert rms_fwd(**kw) == status


@pytest.mark.parametrize('kw,status', SIZES + [
    (dict(dy=None), INVALID), (dict(h=None), INVALID), (dict(dh=None), INVALID), (dict(dw=None), INVALID), (dict(odt=E4M3), INVALID),
    (dict(dh=P), INVALID), (dict(ws=None), WORKSPACE), (dict(wsb=lib.gdn2_rms_norm_bwd_workspace_bytes(4, 100) - 1), WORKSPACE)])
def test_rms_norm_bwd_rejects(kw, status):
    assert rms_bwd(**kw) == status


def test_rms_norm_bwd_rejects_an_output_that_is_another_argument():
    at = addresses('dy h w ds dh dw ws')
    allowed = {('dh', 'dy'), ('dh', 'h'), ('dh', 'ds')}
    for out in ('dh', 'dw', 'ws'):
        for name, p in at.items():
            if name != out and (out, name) not in allowed:
                assert rms_bwd(**{**at, out: p}, odt=BF16) == INVALID, (out, name)


def arrays(ptrs, sizes, types):
    n = len(ptrs)
    return (ctypes.c_void_p * n)(*ptrs), (ctypes.c_int64 * n)(*sizes), (ctypes.c_int32 * n)(*types)


def clip(grads, out, sizes, types=None, otypes=None, max_norm=1.0, norm=0x100, given=0, ws=0x200, wsb=1 << 20):
    types = types or [F32] * len(grads)
    g, s, t = arrays(grads, sizes, types)
    o, _, ot = arrays(out, sizes, otypes or types)
    return lib.gdn2_clip_grads(g, o, s, t, ot, len(grads), max_norm, norm, given, ws, wsb)


def norm_of(grads, sizes, types=None, norm=0x100, ws=0x200, wsb=1 << 20):
    g, s, t = arrays(grads, sizes, types or [F32] * len(grads))
    return lib.gdn2_grad_norm(g, s, t, len(grads), norm, ws, wsb)


@pytest.mark.parametrize('kw,status', [
    (dict(grads=[None], sizes=[4]), INVALID), (dict(grads=[P], sizes=[-1]), INVALID), (dict(grads=[P], sizes=[4], types=[E4M3]), INVALID),
    (dict(grads=[P + 2], sizes=[4]), INVALID), (dict(grads=[P], sizes=[(1 << 40) + 1]), UNSUPPORTED),
    (dict(grads=[P], sizes=[4], norm=None), INVALID), (dict(grads=[P], sizes=[4], norm=0x102), INVALID),
    (dict(grads=[P], sizes=[4], ws=None), WORKSPACE), (dict(grads=[P], sizes=[4], wsb=16), WORKSPACE),
    (dict(grads=[P], sizes=[4], ws=0x208), INVALID), (dict(grads=[P], sizes=[4], norm=0x200), INVALID),
    (dict(grads=[P], sizes=[4], norm=P), INVALID), (dict(grads=[P], sizes=[4], ws=P), INVALID)])
def test_grad_norm_rejects(kw, status):
    assert norm_of(**kw) == status


@pytest.mark.parametrize('kw,status', [
    (dict(grads=[P], out=[None], sizes=[4]), INVALID), (dict(grads=[P], out=[P + 2], sizes=[4]), INVALID),
    (dict(grads=[P], out=[P], sizes=[4], max_norm=-1.0), INVALID), (dict(grads=[P], out=[P], sizes=[4], max_norm=float('nan')), INVALID),
    (dict(grads=[P], out=[P], sizes=[4], max_norm=float('inf')), INVALID),
    (dict(grads=[P], out=[P], sizes=[4], norm=None), INVALID), (dict(grads=[P], out=[P], sizes=[4], ws=None), WORKSPACE),
    (dict(grads=[P], out=[2 * P], sizes=[4], norm=2 * P), INVALID),
    (dict(grads=[P, P], out=[P, P], sizes=[4, 4]), INVALID),                       # the same gradient twice, in place
    (dict(grads=[P, P], out=[2 * P, 2 * P], sizes=[4, 4]), INVALID),               # two into one
    (dict(grads=[P], out=[P], sizes=[4], types=[F32], otypes=[BF16]), INVALID),    # in place with another type
    (dict(grads=[P], out=[P + 8], sizes=[4]), INVALID),                            # partly over its own
    (dict(grads=[P, 2 * P], out=[3 * P, P + 4], sizes=[4, 4]), INVALID),           # partly over another
    (dict(grads=[P, 2 * P], out=[3 * P, 3 * P + 12], sizes=[4, 4]), INVALID),      # two that overlap
    (dict(grads=[P, P + 8], out=[P, P + 8], sizes=[4, 4]), INVALID)])
def test_clip_grads_rejects(kw, status):
    assert clip(**kw) == status


@pytest.mark.parametrize('kw', [dict(norm=P + 0x44), dict(norm=2 * P + 0x3c), dict(ws=P - 0x100), dict(ws=2 * P + 0x20),
                                dict(norm=2 * P + 0x3c, given=1), dict(norm=0x200 + 64)])
def test_clip_grads_rejects_a_norm_or_workspace_within_what_is_written(kw):
    assert clip([P, P + 0x40], [2 * P, 2 * P + 0x40], [16, 16], **kw) == INVALID


@pytest.mark.parametrize('kw', [dict(norm=P + 4), dict(norm=P + 0x7c), dict(norm=0x200 + 64), dict(ws=P - 0x100), dict(ws=P + 0x40),
                                dict(ws=P + 0x70), dict(grads=[2 * P, P], ws=P + 0x10)])
def test_grad_norm_rejects_a_norm_or_workspace_within_a_gradient(kw):
    assert norm_of(**{'grads': [P, P + 0x40], 'sizes': [16, 16], **kw}) == INVALID


def test_binding_refuses_the_cpu_and_wrong_values():
    x, w = torch.zeros(4, 8), torch.zeros(5, 8)
    for call in (lambda: gdn2.linear_fwd(x, w), lambda: gdn2.linear_bwd(torch.zeros(4, 5), x, w),
                 lambda: gdn2.rms_norm_fwd(x, torch.ones(8)), lambda: gdn2.rms_norm_bwd(x, x, torch.ones(8)),
                 lambda: gdn2.grad_norm([x]), lambda: gdn2.clip_grads([x], 1.0), lambda: gdn2.clip_grads([], 1.0)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(ValueError):
        gdn2._act_code('relu')
