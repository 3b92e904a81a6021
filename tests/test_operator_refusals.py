"""Calls that the operators around the mixer refuse, on the CPU: every check runs
on the host before anything is launched, so the made-up aligned addresses below
never reach a kernel."""
import ctypes

import pytest
import torch

import gated_delta_rule_wy_amd as gdn2

P = 0x10000
vp = ctypes.c_void_p
OK, INVALID, UNSUPPORTED, WORKSPACE = (gdn2.GDN2_OK, gdn2.GDN2_ERR_INVALID, gdn2.GDN2_ERR_UNSUPPORTED,
                                       gdn2.GDN2_ERR_WORKSPACE)
F32, BF16 = gdn2.GDN2_F32, gdn2.GDN2_BF16
lib = gdn2.lib()


def recurrent(**kw):
    a = dict(q=P, k=P, v=P, la=P, b=P, w=P, gates=0, state=P, slot_in=None, slot_out=None, commit=None, o=P, cu=None,
             B=2, T=3, N=2, H=4, HK=2, slots=2, dk=64, dv=64, dt=BF16, odt=F32)
    a.update(kw)
    return lib.gdn2_recurrent_fwd(*(a[n] for n in a))


@pytest.mark.parametrize('kw,status', [
    (dict(q=None), INVALID), (dict(la=None), INVALID), (dict(o=None), INVALID), (dict(state=None), INVALID),
    (dict(w=P + 8), INVALID), (dict(slot_in=P + 4, slots=9), INVALID), (dict(commit=P + 4), INVALID),
    (dict(gates=8), INVALID), (dict(gates=-1), INVALID),
    (dict(B=0, N=0), INVALID), (dict(T=-1), INVALID), (dict(H=0), INVALID), (dict(HK=0), INVALID),
    (dict(HK=3), INVALID), (dict(HK=8), INVALID),             # HK divides H
    (dict(N=3), INVALID), (dict(cu=P), INVALID),              # N == B; cu_seqlens with B == 1
    (dict(slots=1), INVALID), (dict(slots=0, slot_in=P), INVALID),
    (dict(dt=2), INVALID), (dict(odt=5), INVALID),
    (dict(dk=48), UNSUPPORTED), (dict(dv=256), UNSUPPORTED), (dict(H=65536, HK=1), UNSUPPORTED),
    (dict(B=70000, N=70000, T=70000, slots=70000), UNSUPPORTED),
])
def test_recurrent_rejects(kw, status):
    assert recurrent(**kw) == status


def conv(**kw):
    c = gdn2.ShortConv(weight_q=P, weight_k=P, weight_v=P)
    for k, v in kw.items():
        setattr(c, k, v)
    return ctypes.byref(c)


IN = dict(state_in_q=P, state_in_k=P, state_in_v=P)
OUT = dict(state_out_q=P, state_out_k=P, state_out_v=P)
PRO = [
    (dict(q=None), INVALID), (dict(xb=None), INVALID), (dict(v=P + 2), INVALID), (dict(conv=None), INVALID),
    (dict(conv=conv(weight_q=None)), INVALID), (dict(conv=conv(state_in_q=P)), INVALID),
    (dict(conv=conv(bias_v=P + 4)), INVALID),
    (dict(conv=conv(**IN), slots=1), INVALID), (dict(conv=conv(**IN), slots=0, slot_in=P), INVALID),
    (dict(gates=4), INVALID), (dict(gates=8), INVALID), (dict(HK=3), INVALID), (dict(N=3), INVALID),
    (dict(cu=P), INVALID), (dict(dt=9), INVALID), (dict(slot_in=P + 4), INVALID),
    (dict(dk=100), UNSUPPORTED), (dict(dv=8), UNSUPPORTED), (dict(B=70000, N=70000, T=70000), UNSUPPORTED),
]


def prologue_fwd(**kw):
    a = dict(q=P, k=P, v=P, xb=P, xw=P, gates=0, conv=conv(), slot_in=None, slot_out=None, commit=None, yq=P, yk=P, yv=P,
             yb=P, yw=P, cu=None, B=2, T=3, N=2, H=4, HK=2, slots=0, dk=64, dv=64, dt=BF16)
    a.update(kw)
    return lib.gdn2_prologue_fwd(*(a[n] for n in a))


@pytest.mark.parametrize('kw,status', PRO + [
    (dict(yk=None), INVALID), (dict(yw=P + 4), INVALID), (dict(commit=P + 4), INVALID),
    (dict(conv=conv(**OUT), slots=1), INVALID),
])
def test_prologue_fwd_rejects(kw, status):
    assert prologue_fwd(**kw) == status


def prologue_bwd(**kw):
    a = dict(q=P, k=P, v=P, xb=P, xw=P, gates=0, conv=conv(), slot_in=None, dq=P, dk_=P, dv_=P, db=P, dw=P, gq=P, gk=P,
             gv=P, gb=P, gw=P, wq=P, wk=P, wv=P, bq=None, bk=None, bv=None, cu=None, B=2, T=3, N=2, H=4, HK=2, slots=0,
             dk=64, dv=64, dt=BF16, gdt=BF16, ws=P, wsb=1 << 30)
    a.update(kw)
    return lib.gdn2_prologue_bwd(*(a[n] for n in a))


@pytest.mark.parametrize('kw,status', PRO + [
    (dict(dq=None), INVALID), (dict(gw=None), INVALID), (dict(wk=None), INVALID), (dict(bq=P + 4), INVALID),
    (dict(gdt=3), INVALID), (dict(ws=None), WORKSPACE),
    (dict(wsb=lib.gdn2_prologue_bwd_workspace_bytes(2, 3, 2, 4, 2, 64, 64, 0) - 1), WORKSPACE),
])
def test_prologue_bwd_rejects(kw, status):
    assert prologue_bwd(**kw) == status


def test_prologue_bwd_workspace():
    W = lib.gdn2_prologue_bwd_workspace_bytes
    assert W(2, 3, 2, 4, 2, 64, 64, 0) > 0 and W(1, 0, 3, 4, 2, 64, 64, 1) > 0
    assert W(2, 3, 1, 4, 2, 64, 64, 0) == 0 and W(2, 3, 2, 4, 3, 64, 64, 0) == 0 and W(2, 3, 2, 4, 2, 60, 64, 0) == 0


def layer_norm_fwd(**kw):
    a = dict(x=P, res=P, w=P, b=P, y=P, s=2 * P, rows=4, cols=100, eps=1e-5, dt=BF16, odt=F32)
    a.update(kw)
    return lib.gdn2_layer_norm_fwd(*(a[n] for n in a))


def layer_norm_bwd(**kw):
    a = dict(dy=P, h=P, w=P, ds=None, dh=P, dw=P, db=P, rows=4, cols=100, eps=1e-5, dt=BF16, odt=F32, ws=P, wsb=1 << 30)
    a.update(kw)
    return lib.gdn2_layer_norm_bwd(*(a[n] for n in a))


LN = [(dict(w=None), INVALID), (dict(rows=-1), INVALID), (dict(cols=0), INVALID), (dict(eps=0.0), INVALID),
      (dict(eps=-1.0), INVALID), (dict(eps=float('nan')), INVALID), (dict(eps=float('inf')), INVALID),
      (dict(dt=2), INVALID), (dict(odt=-1), INVALID), (dict(w=P + 8), INVALID),
      (dict(cols=(1 << 20) + 1), UNSUPPORTED), (dict(rows=(1 << 40) + 1), UNSUPPORTED)]


@pytest.mark.parametrize('kw,status', LN + [(dict(x=None), INVALID), (dict(y=None), INVALID), (dict(s=P + 2), INVALID),
                                            (dict(res=P + 8), INVALID), (dict(s=P), INVALID)])
def test_layer_norm_fwd_rejects(kw, status):
    assert layer_norm_fwd(**kw) == status


@pytest.mark.parametrize('kw,status', LN + [
    (dict(dy=None), INVALID), (dict(dh=None), INVALID), (dict(dw=None), INVALID), (dict(ds=P + 4), INVALID),
    (dict(ws=None), WORKSPACE), (dict(wsb=lib.gdn2_layer_norm_bwd_workspace_bytes(4, 100) - 1), WORKSPACE)])
def test_layer_norm_bwd_rejects(kw, status):
    assert layer_norm_bwd(**kw) == status


def test_layer_norm_rejects_outputs_over_inputs():
    """In place is for one type: y over x or the residual, dh over dy; never over a weight."""
    at = dict(x=2 * P, res=3 * P, w=4 * P, b=5 * P, y=6 * P, s=7 * P)
    for kw in (dict(y=2 * P), dict(y=3 * P), dict(y=4 * P, odt=BF16), dict(s=5 * P)):
        assert layer_norm_fwd(**{**at, **kw}) == INVALID, kw
    at = dict(dy=2 * P, h=3 * P, w=4 * P, ds=5 * P, dh=6 * P, dw=7 * P, db=8 * P)
    for kw in (dict(dh=2 * P), dict(dh=4 * P), dict(dw=4 * P), dict(db=2 * P), dict(dw=6 * P)):
        assert layer_norm_bwd(**{**at, **kw}) == INVALID, kw


def test_layer_norm_workspace():
    W = lib.gdn2_layer_norm_bwd_workspace_bytes
    assert W(0, 64) > 0 and W(1 << 30, 1 << 20) > 0
    assert W(-1, 64) == 0 and W(4, 0) == 0 and W(4, (1 << 20) + 1) == 0
    assert W(1 << 30, 2048) <= 64 << 20


@pytest.mark.parametrize('name', ['q', 'k', 'v', 'la', 'b', 'w', 'state'])
def test_recurrent_rejects_an_output_that_is_an_input(name):
    ins = {n: (i + 2) * P for i, n in enumerate(('q', 'k', 'v', 'la', 'b', 'w', 'state'))}
    assert recurrent(**ins, o=ins[name]) == INVALID


@pytest.mark.parametrize('out', ['yq', 'yk', 'yv', 'yb', 'yw'])
@pytest.mark.parametrize('name', ['q', 'k', 'v', 'xb', 'xw'])
def test_prologue_fwd_rejects_an_output_that_is_an_input(out, name):
    if out in ('yb', 'yw') and name in ('xb', 'xw'):
        return   # (gates in place of their logits are allowed)
    at = {n: (i + 2) * P for i, n in enumerate(('q', 'k', 'v', 'xb', 'xw', 'yq', 'yk', 'yv', 'yb', 'yw'))}
    at[out] = at[name]
    assert prologue_fwd(**at) == INVALID


@pytest.mark.parametrize('out', ['gq', 'gk', 'gv', 'gb', 'gw'])
@pytest.mark.parametrize('name', ['q', 'k', 'v', 'xb', 'xw', 'dq', 'dk_', 'dv_', 'db', 'dw'])
def test_prologue_bwd_rejects_an_output_that_is_an_input(out, name):
    at = {n: (i + 2) * P for i, n in enumerate(('q', 'k', 'v', 'xb', 'xw', 'dq', 'dk_', 'dv_', 'db', 'dw', 'gq', 'gk',
                                                'gv', 'gb', 'gw'))}
    at[out] = at[name]
    assert prologue_bwd(**at) == INVALID


def test_rejects_more_threads_than_a_launch_takes():
    """2^32 threads or more, of sizes that every other check lets pass."""
    ins = {n: (i + 2) * P for i, n in enumerate(('q', 'k', 'v', 'la', 'b', 'w', 'state', 'o'))}
    many = dict(B=1 << 20, N=1 << 20, T=1, H=64, HK=1, slots=1 << 20, dk=128, dv=128)
    assert recurrent(**ins, **many) == UNSUPPORTED
    assert recurrent(**ins, **{**many, 'H': 128, 'dk': 64, 'dv': 64}) == UNSUPPORTED
    at = _apart('q', 'k', 'v', 'xb', 'xw', 'yq', 'yk', 'yv', 'yb', 'yw')
    many = dict(B=1 << 24, N=1 << 24, T=1, H=15, HK=1, dk=128, dv=128)
    assert prologue_fwd(**at, **many) == UNSUPPORTED
    assert prologue_fwd(**at, **many, gates=3) == UNSUPPORTED
    pools = conv(**{n: (i + 20) * P for i, n in enumerate(('state_out_q', 'state_out_k', 'state_out_v'))})
    assert prologue_fwd(**at, conv=pools, slots=4, slot_in=50 * P, cu=51 * P, B=1, N=(1 << 31) - 1, T=17, H=1, HK=1,
                        dk=16, dv=16) == UNSUPPORTED
    at = {n: (i + 2) * P for i, n in enumerate(('q', 'k', 'v', 'xb', 'xw', 'dq', 'dk_', 'dv_', 'db', 'dw', 'gq', 'gk', 'gv',
                                                'gb', 'gw', 'wq', 'wk', 'wv', 'ws'))}
    assert prologue_bwd(**at, **many, wsb=1 << 40) == UNSUPPORTED


def _apart(*names):
    return {n: (i + 2) * P for i, n in enumerate(names)}


@pytest.mark.parametrize('name', ['q', 'k', 'v', 'la', 'b', 'w', 'slot_in', 'slot_out', 'commit', 'cu', 'o'])
def test_recurrent_rejects_states_that_are_another_argument(name):
    at = _apart('q', 'k', 'v', 'la', 'b', 'w', 'slot_in', 'slot_out', 'commit', 'cu', 'o')
    assert recurrent(**at, state=at[name], B=1, T=6) == INVALID
    if name != 'o':
        assert recurrent(**{**at, 'o': at[name]}, state=P, B=1, T=6) == INVALID


CONV = ('weight_q', 'weight_k', 'weight_v', 'bias_q', 'bias_k', 'bias_v', 'state_in_q', 'state_in_k', 'state_in_v',
        'state_out_q', 'state_out_k', 'state_out_v')
FWD = ('q', 'k', 'v', 'xb', 'xw', 'slot_in', 'slot_out', 'commit', 'yq', 'yk', 'yv', 'yb', 'yw')
BWD = ('q', 'k', 'v', 'xb', 'xw', 'slot_in', 'dq', 'dk_', 'dv_', 'db', 'dw', 'gq', 'gk', 'gv', 'gb', 'gw', 'wq', 'wk',
       'wv', 'bq', 'bk', 'bv', 'ws')


def _call(fn, names, at):
    return fn(**{n: at[n] for n in names}, conv=conv(**{n: at[n] for n in CONV}), slots=2)


@pytest.mark.parametrize('out', ['yq', 'yk', 'yv', 'yb', 'yw', 'state_out_q', 'state_out_k', 'state_out_v'])
def test_prologue_fwd_rejects_an_output_that_is_another_argument(out):
    """Every other argument but a gate's own logits and a history's own pool."""
    own = {'yb': 'xb', 'yw': 'xw'}.get(out, out.replace('out', 'in'))
    for name in (*FWD, *CONV):
        if name not in (out, own):
            at = _apart(*FWD, *CONV)
            at[out] = at[name]
            assert _call(prologue_fwd, FWD, at) == INVALID, name


@pytest.mark.parametrize('out', ['gq', 'gk', 'gv', 'gb', 'gw', 'wq', 'wk', 'wv', 'bq', 'bk', 'bv', 'ws'])
def test_prologue_bwd_rejects_an_output_that_is_another_argument(out):
    for name in (*BWD, *CONV[:9]):
        if name != out:
            at = _apart(*BWD, *CONV)
            at[out] = at[name]
            assert _call(prologue_bwd, BWD, at) == INVALID, name


def test_layer_norm_bwd_rejects_an_output_that_is_another_argument():
    names = ('dy', 'h', 'w', 'ds', 'dh', 'dw', 'db', 'ws')
    for out in ('dh', 'dw', 'db', 'ws'):
        for name in names:
            if name != out and not (out == 'dh' and name in ('dy', 'h', 'ds')):
                at = _apart(*names)
                at[out] = at[name]
                assert layer_norm_bwd(**at, odt=BF16) == INVALID, (out, name)


# ---- the Python binding: wrong shapes, types and devices raise before the library is called

def _mix(B=1, T=4, H=2, HK=2, dk=32, dv=32, dt=torch.bfloat16):
    z = lambda *s: torch.zeros(s, dtype=dt)   # noqa: E731
    return [z(B, T, HK, dk), z(B, T, HK, dk), z(B, T, H, dv), torch.zeros(B, T, H, dk), z(B, T, H, dk), z(B, T, H, dv)]


def test_binding_refuses_cpu_tensors():
    x = _mix()
    with pytest.raises(ValueError, match='GPU'):
        gdn2.recurrent_fwd(*x, torch.zeros(1, 2, 32, 32))
    w = tuple(torch.zeros(64, 4) for _ in range(3))
    with pytest.raises(ValueError, match='GPU'):
        gdn2.prologue_fwd(x[0], x[1], x[2], x[4], x[5], w)
    with pytest.raises(ValueError, match='GPU'):
        gdn2.prologue_bwd(x[0], x[1], x[2], x[4], x[5], w, None, *(t.float() for t in (*x[:3], *x[4:])))
    with pytest.raises(ValueError, match='GPU'):
        gdn2.layer_norm_fwd(torch.zeros(4, 8), torch.ones(8))
    with pytest.raises(ValueError, match='GPU'):
        gdn2.layer_norm_bwd(torch.zeros(4, 8), torch.zeros(4, 8), torch.ones(8))


def test_binding_refuses_wrong_ranks():
    x = _mix()
    with pytest.raises(ValueError, match='must be'):
        gdn2.recurrent_fwd(x[0][0], *x[1:], torch.zeros(1, 2, 32, 32))
    with pytest.raises(ValueError, match='must be'):
        gdn2.recurrent_fwd(*x[:2], x[2][0], *x[3:], torch.zeros(1, 2, 32, 32))


@pytest.mark.gpu
@pytest.mark.parametrize('change', ['k shape', 'v dtype', 'la dtype', 'b shape', 'state shape', 'state dtype', 'slots',
                                    'slot dtype', 'slot length', 'commit device', 'strided', 'heads', 'cu dtype', 'out',
                                    'out dtype', 'half', 'misaligned'])
def test_recurrent_binding_refuses(change):
    dev = torch.device('cuda:0')
    q, k, v, la, b, w = (t.to(dev) for t in _mix())
    state, kw, cu = torch.zeros(2, 2, 32, 32, device=dev), {}, None
    idx = lambda *s, **o: torch.zeros(*s, **{'dtype': torch.int32, 'device': dev, **o})   # noqa: E731
    if change == 'k shape': k = k[:, :3].contiguous()   # noqa: E701
    if change == 'v dtype': v = v.float()   # noqa: E701
    if change == 'la dtype': la = la.bfloat16()   # noqa: E701
    if change == 'b shape': b = b[..., :16].contiguous()   # noqa: E701
    if change == 'state shape': state = state[..., :16].contiguous()   # noqa: E701
    if change == 'state dtype': state = state.bfloat16()   # noqa: E701
    if change == 'slots': cu, state = idx(4), state   # noqa: E701  (3 sequences, 2 slots)
    if change == 'slot dtype': kw['slot_in'] = idx(1, dtype=torch.int64)   # noqa: E701
    if change == 'slot length': kw['slot_in'] = idx(2)   # noqa: E701
    if change == 'commit device': kw['commit'] = idx(1, device='cpu')   # noqa: E701
    if change == 'strided': q = torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16, device=dev)[..., ::2]   # noqa: E701
    if change == 'heads': q = k = torch.zeros(1, 4, 3, 32, dtype=torch.bfloat16, device=dev)   # noqa: E701
    if change == 'cu dtype': cu = idx(2, dtype=torch.int64)   # noqa: E701
    if change == 'out': kw['out'] = torch.zeros(1, 4, 2, 16, device=dev)   # noqa: E701
    if change == 'out dtype': kw['out_dtype'] = torch.float16   # noqa: E701
    if change == 'half': q, k, v, b, w = (t.half() for t in (q, k, v, b, w))   # noqa: E701
    if change == 'misaligned':
        state = torch.zeros(2 * 2 * 32 * 32 + 1, device=dev)[1:].view(2, 2, 32, 32)
    with pytest.raises((ValueError, TypeError, gdn2.Gdn2Error)):
        gdn2.recurrent_fwd(q, k, v, la, b, w, state, cu, **kw)


@pytest.mark.gpu
@pytest.mark.parametrize('change', ['weight shape', 'weight count', 'bias count', 'bias dtype', 'pool dtype', 'pool slots', 'slots',
                                    'logit shape', 'out count', 'out shape', 'grad shape', 'grad dtype'])
def test_prologue_binding_refuses(change):
    dev = torch.device('cuda:0')
    q, k, v, _, b, w = (t.to(dev) for t in _mix())
    wt, bs = tuple(torch.zeros(64, 4, device=dev) for _ in range(3)), tuple(torch.zeros(64, device=dev) for _ in range(3))
    pool = tuple(torch.zeros(2, 2, 3, 32, dtype=torch.bfloat16, device=dev) for _ in range(3))
    kw, cu = dict(conv_state=pool), None
    if change == 'weight shape': wt = (wt[0], wt[1][:32].contiguous(), wt[2])   # noqa: E701
    if change == 'weight count': wt = wt[:2]   # noqa: E701
    if change == 'bias count': bs = bs[:2]   # noqa: E701
    if change == 'bias dtype': bs = tuple(x.bfloat16() for x in bs)   # noqa: E701
    if change == 'pool dtype': kw['conv_state'] = tuple(x.float() for x in pool)   # noqa: E701
    if change == 'pool slots': kw['conv_state'] = (pool[0], pool[1], pool[2][:1].contiguous())   # noqa: E701
    if change == 'slots': cu = torch.zeros(4, dtype=torch.int32, device=dev)   # noqa: E701
    if change == 'logit shape': b = b[..., :8].contiguous()   # noqa: E701
    grads = [torch.zeros(x.shape, device=dev) for x in (q, k, v, b, w)]
    if change == 'grad shape': grads[1] = grads[1][:, :2].contiguous()   # noqa: E701
    if change == 'grad dtype': grads[4] = grads[4].bfloat16()   # noqa: E701
    raises = pytest.raises((ValueError, TypeError, gdn2.Gdn2Error))
    if not change.startswith('grad'):
        out = dict(kw)
        if change == 'out count': out['out'] = (q, k, v, b)   # noqa: E701
        if change == 'out shape': out['out'] = (q.clone(), k.clone(), v.clone(), b.clone(), w[:, :1].contiguous())   # noqa: E701
        with raises:
            gdn2.prologue_fwd(q, k, v, b, w, wt, bs, cu, **out)
    if not change.startswith('out'):
        with raises:
            gdn2.prologue_bwd(q, k, v, b, w, wt, bs, *grads, cu, **kw)


@pytest.mark.gpu
@pytest.mark.parametrize('z', [0, 1, 2])
@pytest.mark.parametrize('name', ['conv_weight', 'conv_state', 'conv_state_out'])
@pytest.mark.parametrize('value', [None, 0])
def test_prologue_binding_refuses_a_triple_with_a_gap(name, z, value):
    """None in a triple, and a tensor without axes."""
    dev = torch.device('cuda:0')
    q, k, v, _, b, w = (t.to(dev) for t in _mix())
    pool = [torch.zeros(2, 2, 3, 32, dtype=torch.bfloat16, device=dev) for _ in range(3)]
    kw = dict(conv_weight=[torch.zeros(64, 4, device=dev) for _ in range(3)], conv_state=pool, conv_state_out=list(pool))
    kw[name] = list(kw[name])
    kw[name][z] = None if value is None else torch.zeros((), dtype=kw[name][z].dtype, device=dev)
    with pytest.raises(ValueError, match='conv_weight' if name == 'conv_weight' else 'conv_state'):
        gdn2.prologue_fwd(q, k, v, b, w, **kw)
    if name != 'conv_state_out':
        grads = [torch.zeros(x.shape, device=dev) for x in (q, k, v, b, w)]
        del kw['conv_state_out']
        with pytest.raises(ValueError, match=name):
            gdn2.prologue_bwd(q, k, v, b, w, kw.pop('conv_weight'), None, *grads, **kw)


@pytest.mark.gpu
def test_layer_norm_binding_refuses():
    dev = torch.device('cuda:0')
    x, w = torch.zeros(4, 16, device=dev), torch.ones(16, device=dev)
    bad = (ValueError, TypeError, gdn2.Gdn2Error)
    for args, kw in (((x, w[:8].contiguous()), {}), ((x, w.bfloat16()), {}), ((x.half(), w), {}), ((x.t(), w), {}),
                     ((x, w, w[:3].contiguous()), {}), ((x, w, None, x.bfloat16()), {}), ((x, w), dict(eps=0.0)),
                     ((x, w), dict(out_dtype=torch.float16)), ((x, w), dict(sum_out=x[:2].clone())),
                     ((x[:, :0], w[:0]), {}), ((x, w, None, x[:2].clone()), {})):
        with pytest.raises(bad):
            gdn2.layer_norm_fwd(*args, **kw)
    for args, kw in (((x[:2].clone(), x, w), {}), ((x.half(), x, w), {}), ((x, x, w.double()), {}),
                     ((x, x, w), dict(dsum=x.bfloat16())), ((x, x, w), dict(eps=-1.0)),
                     ((x, x, w), dict(out=x.bfloat16()))):
        with pytest.raises(bad):
            gdn2.layer_norm_bwd(*args, **kw)
