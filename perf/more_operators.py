"""Timed cases of the layer's dense half: its projections, the norm before them and the clipping of
their gradients.

* ``linear_fwd`` / ``linear_bwd``: a matrix product with bias, activation and residual in its
  epilogue, in bf16, fp32, or e4m3 with a scale a row and an output channel; and its gradient;
* ``rms_norm_fwd`` / ``rms_norm_bwd``: root-mean-square norm of x + residual, its output in bf16, fp32
  or e4m3 with a scale a row (what the product takes), and its gradient;
* ``clip``: the global norm over many gradients, and the gradients scaled to a largest norm.

``run`` computes a case with elementary torch operations in float32 (``own`` false) or through the
package (``own`` true); ``exact`` has the same values from the definitions in float64.

Sizes follow the library's workloads: model width 2048 (16 heads of 128 channels), 256 sequences in a
decode step, prompts of 65536 tokens, training batches of 8 x 4096 tokens; a feed-forward width of four times the model's.
"""
import math

import torch

own = False

DTYPES = {'bf16': torch.bfloat16, 'f32': torch.float32, 'e4m3': torch.float8_e4m3fn}
SIZE = {'bf16': 2, 'f32': 4, 'e4m3': 1}
EPS = 1e-5
TOP = 448.0          # the largest e4m3 value
CLIP_EPS = 1e-6


# ---- cases -------------------------------------------------------------------

def _linear(op, M, N, K, dtype='bf16', act='none', bias=False, residual=False, out=None):
    return dict(op=op, M=M, N=N, K=K, dtype=dtype, act=act, bias=bias, residual=residual,
                out=out or ('bf16' if dtype == 'e4m3' else dtype))


def _rms(op, rows, cols, dtype='bf16', out=None, residual=True):
    return dict(op=op, rows=rows, cols=cols, dtype=dtype, out=out or dtype, residual=residual)


def _clip(width, layers, dtype='bf16', out=None, clipped=True, odd=0):
    return dict(op='clip', width=width, layers=layers, dtype=dtype, out=out or dtype, clipped=clipped, odd=odd)


def listed():
    return [
        # a gate's logits for a few interactive users: latency
        dict(name='linear_4x2048x2048', **_linear('linear_fwd', 4, 2048, 2048, act='sigmoid', bias=True)),
        # the decode batch's output projection in 8 bits, added to the residual stream
        dict(name='linear_e4m3_256x2048x2048', **_linear('linear_fwd', 256, 2048, 2048, 'e4m3', residual=True)),
        # a small fine-tuning batch in float32, odd sizes
        dict(name='linear_f32_4999x1001x1021', **_linear('linear_fwd', 4999, 1001, 1021, 'f32', 'silu', True)),
        # the long prompt's output projection, added to the residual stream
        dict(name='linear_65536x2048x2048', **_linear('linear_fwd', 65536, 2048, 2048, residual=True)),
        # a feed-forward layer's first product in 8 bits, over packed prompts
        dict(name='linear_e4m3_32768x8192x2048', **_linear('linear_fwd', 32768, 8192, 2048, 'e4m3', 'silu')),
        # a small fine-tuning batch's gradient, odd sizes
        dict(name='linear_bwd_f32_1554x1001x777', **_linear('linear_bwd', 1554, 1001, 777, 'f32', bias=True)),
        # a training batch's gate projection
        dict(name='linear_bwd_32768x2048x2048', **_linear('linear_bwd', 32768, 2048, 2048, act='sigmoid', bias=True)),
        # the decode batch's norm before the projections, in 8 bits
        dict(name='rms_norm_256x2048_e4m3', **_rms('rms_norm_fwd', 256, 2048, out='e4m3')),
        # the same for the long prompt
        dict(name='rms_norm_65536x2048_e4m3', **_rms('rms_norm_fwd', 65536, 2048, out='e4m3')),
        # a training step's gradient over the long prompt
        dict(name='rms_norm_bwd_65536x2048', **_rms('rms_norm_bwd', 65536, 2048)),
        # one layer's gradients, an odd width, below the largest norm: nothing to scale, copied for the optimizer
        dict(name='clip_f32_1001x1', **_clip(1001, 1, 'f32', clipped=False, odd=3)),
        # a model's gradients: 7 layers, vectors and matrices, bf16, clipped into the optimizer's float32 buffers
        dict(name='clip_2048x7', **_clip(2048, 7, 'bf16', 'f32')),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def _kind(case):
    return case['op'], case['dtype'] == 'f32' and case['op'].startswith('linear')


_CAP = {}


def _caps():
    if not _CAP:
        for c in listed():
            w = work(c)
            k = _kind(c)
            old = _CAP.get(k, (0, 0))
            _CAP[k] = max(old[0], w['bytes']), max(old[1], w['flops'])
    return _CAP


def draw(rng):
    while True:
        op = rng.choice(['linear_fwd', 'linear_fwd', 'linear_bwd', 'rms_norm_fwd', 'rms_norm_bwd', 'clip'])
        if op == 'clip':
            dtype = rng.choice(['bf16', 'f32'])
            c = _clip(_log(rng, 16, 2048), rng.randint(1, 7), dtype, rng.choice(['bf16', 'f32']), rng.random() < 0.7,
                      rng.randrange(0, 9))
        elif op.startswith('rms'):
            dtype = rng.choice(['bf16', 'bf16', 'f32'])
            out = rng.choice([dtype, 'e4m3'] if op == 'rms_norm_fwd' else [dtype])
            c = _rms(op, _log(rng, 1, 65536), _log(rng, 16, 8192), dtype, out, rng.random() < 0.5)
        else:
            dtype = rng.choice(['bf16', 'bf16', 'f32'] + (['e4m3', 'e4m3'] if op == 'linear_fwd' else []))
            N, K = (_log(rng, 16, 8192) for _ in range(2))
            if rng.random() < 0.6:      # most programs have widths of whole vectors
                N, K = -(-N // 16) * 16, -(-K // 16) * 16
            c = _linear(op, _log(rng, 1, 65536), N, K, dtype, rng.choice(['none', 'none', 'sigmoid', 'silu', 'gelu_tanh']),
                        rng.random() < 0.5, op == 'linear_fwd' and rng.random() < 0.5)
        w, top = work(c), _caps().get(_kind(c))
        if w['bytes'] <= top[0] and w['flops'] <= top[1]:
            return c


def _shapes(case):
    """The gradients of a model: for each layer the norm's weight, three projections of the width and one
    to the gates, taps and biases of the short convolutions, and a feed-forward matrix; and a vector of its own."""
    W = case['width']
    out = []
    for _ in range(case['layers']):
        out += [(W,), (W, W), (W, W), (W, W), (max(1, W // 128), W), (W, 4), (W,), (4 * W, W)]
    return out + [(case['odd'],)]


def work(case):
    op = case['op']
    if op == 'clip':
        n = sum(math.prod(s) for s in _shapes(case))
        return {'bytes': n * (SIZE[case['dtype']] + SIZE[case['out']]), 'flops': 3 * n}
    e, o = SIZE[case['dtype']], SIZE[case['out']]
    if op == 'rms_norm_fwd':
        R, C = case['rows'], case['cols']
        n = R * C
        return {'bytes': n * (e * (3 if case['residual'] else 1) + o) + 4 * C + (4 * R if case['out'] == 'e4m3' else 0),
                'flops': n * (6 if case['residual'] else 5)}
    if op == 'rms_norm_bwd':
        n = case['rows'] * case['cols']
        return {'bytes': n * e * (4 if case['residual'] else 3) + 8 * case['cols'], 'flops': n * 11}
    M, N, K = case['M'], case['N'], case['K']
    if op == 'linear_fwd':
        return {'bytes': (M * K + N * K) * e + M * N * o * (2 if case['residual'] else 1) + (4 * N if case['bias'] else 0)
                + (4 * (M + N) if case['dtype'] == 'e4m3' else 0), 'flops': 2 * M * N * K}
    return {'bytes': 2 * (M * K + N * K) * e + M * N * e * (1 if case['act'] == 'none' else 2) + (4 * N if case['bias'] else 0),
            'flops': 4 * M * N * K}


# ---- inputs ------------------------------------------------------------------

def prepare(case, seed):
    dev = torch.device('cuda')
    g = torch.Generator(device=dev).manual_seed(seed)
    op = case['op']

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev)

    s = {'case': case}
    if op == 'clip':
        dt, out = DTYPES[case['dtype']], DTYPES[case['out']]
        s['grads'] = [(normal(*shape) * 10 ** (-2 + 2 * i / (7 * case['layers'] + 1))).to(dt)
                      for i, shape in enumerate(_shapes(case))]
        s['out'] = [torch.zeros(x.shape, dtype=out, device=dev) for x in s['grads']]
        s['max_norm'] = 1.0 if case['clipped'] else 1e6
        return s
    if op.startswith('rms'):
        R, C, dt = case['rows'], case['cols'], DTYPES[case['dtype']]
        s['weight'] = 1 + 0.1 * normal(C)
        # rows of an activation stream: their scales differ
        s['x'] = (normal(R, C) * (0.5 + 2 * torch.rand(R, 1, generator=g, device=dev))).to(dt)
        name = 'residual' if op == 'rms_norm_fwd' else 'dsum'
        s[name] = normal(R, C).to(dt) if case['residual'] else None
        if op == 'rms_norm_bwd':
            s['dy'] = normal(R, C).to(dt)
        return s

    M, N, K, dt = case['M'], case['N'], case['K'], DTYPES[case['dtype']]
    x, w = normal(M, K), normal(N, K) / math.sqrt(K)
    s['x_scale'] = s['weight_scale'] = None
    if case['dtype'] == 'e4m3':
        s['x_scale'], s['weight_scale'] = (t.abs().amax(1) / TOP for t in (x, w))
        x, w = x / s['x_scale'][:, None], w / s['weight_scale'][:, None]
    s['x'], s['weight'] = x.to(dt), w.to(dt)
    s['bias'] = 0.1 * normal(N) if case['bias'] else None
    if op == 'linear_fwd':
        s['residual'] = normal(M, N).to(DTYPES[case['out']]) if case['residual'] else None
    else:
        s['dy'] = normal(M, N).to(dt)
        s['preact'] = normal(M, N).to(dt) if case['act'] != 'none' else None
    return s


# ---- the operators in their plain form ---------------------------------------

def _sig(z):
    return 1 / (1 + torch.exp(-z))


_C0, _C1 = 2 * math.sqrt(2 / math.pi), 0.044715


def _plain_act(name, z):
    if name == 'sigmoid':
        return _sig(z)
    if name == 'silu':
        return z * _sig(z)
    if name == 'gelu_tanh':
        return z * _sig(_C0 * (z + _C1 * z * z * z))
    return z


def _plain_slope(name, z):
    if name == 'sigmoid':
        return _sig(z) * _sig(-z)
    if name == 'silu':
        return _sig(z) + z * _sig(z) * _sig(-z)
    u = _C0 * (z + _C1 * z * z * z)
    return _sig(u) + z * _sig(u) * _sig(-u) * _C0 * (1 + 3 * _C1 * z * z)


def _plain_linear_fwd(s):
    case = s['case']
    z = s['x'].float() @ s['weight'].float().t()
    if s['x_scale'] is not None:
        z = z * s['x_scale'][:, None] * s['weight_scale']
    if s['bias'] is not None:
        z = z + s['bias']
    y = _plain_act(case['act'], z)
    if s['residual'] is not None:
        y = y + s['residual'].float()
    return y.to(DTYPES[case['out']])


def _plain_linear_bwd(s):
    case = s['case']
    dt = DTYPES[case['dtype']]
    dz = s['dy'].float()
    if case['act'] != 'none':
        dz = dz * _plain_slope(case['act'], s['preact'].float())
    out = {'x': (dz @ s['weight'].float()).to(dt), 'weight': (dz.t() @ s['x'].float()).to(dt)}
    if case['bias']:
        out['bias'] = dz.sum(0, dtype=torch.float64).float()
    return out


def _plain_rms_norm_fwd(s):
    case = s['case']
    h = s['x'].float()
    if s['residual'] is not None:
        h = h + s['residual'].float()
    y = h / (h.square().mean(-1, keepdim=True) + EPS).sqrt() * s['weight']
    out = []
    if case['out'] == 'e4m3':
        scale = y.abs().amax(-1) / TOP
        out += [(y / scale[:, None]).to(DTYPES['e4m3']), scale]
    else:
        out += [y.to(DTYPES[case['out']])]
    if s['residual'] is not None:
        out += [h.to(s['x'].dtype)]
    return out


def _plain_rms_norm_bwd(s):
    h, dy = s['x'].float(), s['dy'].float()
    rstd = 1 / (h.square().mean(-1, keepdim=True) + EPS).sqrt()
    xh, g = h * rstd, dy * s['weight']
    dh = rstd * (g - xh * (g * xh).mean(-1, keepdim=True))
    if s['dsum'] is not None:
        dh = dh + s['dsum'].float()
    return {'x': dh.to(s['x'].dtype), 'weight': (dy * xh).sum(0, dtype=torch.float64).float()}


def _plain_clip(s):
    total = sum(x.double().square().sum() for x in s['grads'])
    norm = total.sqrt().float()
    scale = (s['max_norm'] / (norm + CLIP_EPS)).clamp_max(1)
    for x, y in zip(s['grads'], s['out']):
        y.copy_((x.float() * scale).to(y.dtype))
    return [norm] + s['out']


_PLAIN = {'linear_fwd': _plain_linear_fwd, 'linear_bwd': _plain_linear_bwd, 'rms_norm_fwd': _plain_rms_norm_fwd,
          'rms_norm_bwd': _plain_rms_norm_bwd, 'clip': _plain_clip}


# ---- the operators through the package ----------------------------------------

def _own(s):
    import gated_delta_rule_wy_amd as gdn2
    case = s['case']
    op = case['op']
    if op == 'linear_fwd':
        return gdn2.linear_fwd(s['x'], s['weight'], s['bias'], s['residual'], activation=case['act'],
                               x_scale=s['x_scale'], weight_scale=s['weight_scale'], out_dtype=DTYPES[case['out']])[0]
    if op == 'linear_bwd':
        return gdn2.linear_bwd(s['dy'], s['x'], s['weight'], s['preact'], activation=case['act'],
                               output_bias=case['bias'])
    if op == 'rms_norm_fwd':
        y, h, scale = gdn2.rms_norm_fwd(s['x'], s['weight'], s['residual'], eps=EPS,
                                        output_sum=s['residual'] is not None, out_dtype=DTYPES[case['out']])
        return [t for t in (y, scale, h) if t is not None]
    if op == 'rms_norm_bwd':
        return gdn2.rms_norm_bwd(s['dy'], s['x'], s['weight'], dsum=s['dsum'], eps=EPS)
    return [gdn2.clip_grads(s['grads'], s['max_norm'], out=s['out'])] + s['out']


def run(state):
    return _own(state) if own else _PLAIN[state['case']['op']](state)


# ---- the definitions in 64 bits -------------------------------------------------

def _exact_act(name, z):
    if name == 'sigmoid':
        return torch.sigmoid(z)
    if name == 'silu':
        return z * torch.sigmoid(z)
    if name == 'gelu_tanh':
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    return z


def _exact_linear_fwd(s):
    x, w = s['x'].double(), s['weight'].double()
    if s['x_scale'] is not None:
        x, w = x * s['x_scale'].double()[:, None], w * s['weight_scale'].double()[:, None]
    z = torch.mm(x, w.t())
    if s['bias'] is not None:
        z += s['bias'].double()
    y = _exact_act(s['case']['act'], z)
    return y if s['residual'] is None else y + s['residual'].double()


def _exact_linear_bwd(s):
    dz = s['dy'].double()
    if s['preact'] is not None:
        with torch.enable_grad():
            z = s['preact'].double().requires_grad_()
            dz, = torch.autograd.grad(_exact_act(s['case']['act'], z), z, dz)
    out = {'x': torch.mm(dz, s['weight'].double()), 'weight': torch.mm(dz.t(), s['x'].double())}
    if s['case']['bias']:
        out['bias'] = dz.sum(0)
    return out


def _exact_norm(h, weight):
    return h * torch.rsqrt(h.pow(2).mean(-1, keepdim=True) + EPS) * weight


def _exact_rms_norm_fwd(s):
    h = s['x'].double() + (0 if s['residual'] is None else s['residual'].double())
    y = _exact_norm(h, s['weight'].double())
    out = [y]
    if s['case']['out'] == 'e4m3':
        scale = y.abs().max(-1).values / TOP
        q = y / scale[:, None]
        # three bits behind the leading one, down to 2^-9; halves to the even neighbour
        step = torch.exp2(torch.floor(torch.log2(q.abs().clamp_min(2.0 ** -6))) - 3)
        out = [torch.round(q / step) * step, scale]
    return out if s['residual'] is None else out + [h]


def _exact_rms_norm_bwd(s):
    with torch.enable_grad():
        leaves = [s[x].double().requires_grad_() for x in ('x', 'weight')]
        dx, dw = torch.autograd.grad(_exact_norm(*leaves), leaves, s['dy'].double())
    return {'x': dx if s['dsum'] is None else dx + s['dsum'].double(), 'weight': dw}


def _exact_clip(s):
    norm = torch.linalg.vector_norm(torch.stack([torch.linalg.vector_norm(x.double()) for x in s['grads']]))
    scale = torch.clamp(s['max_norm'] / (norm + CLIP_EPS), max=1.0)
    return [norm] + [x.double() * scale for x in s['grads']]


_EXACT = {'linear_fwd': _exact_linear_fwd, 'linear_bwd': _exact_linear_bwd, 'rms_norm_fwd': _exact_rms_norm_fwd,
          'rms_norm_bwd': _exact_rms_norm_bwd, 'clip': _exact_clip}


def exact(case, seed):
    with torch.no_grad():
        return _EXACT[case['op']](prepare(case, seed))
