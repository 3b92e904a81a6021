"""Timed cases of the serving and training operators around the token mixer.

Three groups, each with its forms:

* ``recurrent``: the gated delta rule token by token over a pool of states reached through slot
  numbers (``recurrent_fwd``), one token a sequence up to a few dozen, with draft tokens whose effect
  is not kept;
* ``prologue_fwd`` / ``prologue_bwd``: short convolution, unit norm and sigmoid on the layer's
  projections, with the convolution history in the same slots, and its gradient;
* ``layer_norm_fwd`` / ``layer_norm_bwd``: the layer's closing LayerNorm(x + residual) and its
  gradient with the weights' reductions.

``run`` computes a case with elementary torch operations in float32 (``own`` false) or through the
package (``own`` true); ``exact`` has the same values from the definitions in float64.

Sizes follow the library's workloads: 16 heads of 128 channels (model width 2048), 256 sequences in a
decode step, packed sequences of mixed length, 32 heads.
"""
import math
import random

import torch

own = False

DTYPES = {'bf16': torch.bfloat16, 'f32': torch.float32}
TAPS = 4
EPS = 1e-5


# ---- cases -------------------------------------------------------------------

def _recurrent(N, T, H, dk, dv, dtype='bf16', out='f32', gates='channel', HK=None, ragged=False, commit=False,
               spare=0):
    return dict(op='recurrent', N=N, T=T, H=H, HK=HK or H, dk=dk, dv=dv, dtype=dtype, out=out, gates=gates,
                ragged=ragged, commit=commit, slots=N + spare)


def _prologue(op, N, T, H, dk, dv, dtype='bf16', HK=None, ragged=False, history=False, commit=False, gates='channel'):
    return dict(op=op, N=N, T=T, H=H, HK=HK or H, dk=dk, dv=dv, dtype=dtype, ragged=ragged, history=history,
                commit=commit, gates=gates)


def _layer_norm(op, rows, cols, dtype='bf16', residual=True):
    return dict(op=op, rows=rows, cols=cols, dtype=dtype, residual=residual)


def listed():
    return [
        # a few interactive users, one token each: latency
        dict(name='recurrent_4x1', **_recurrent(4, 1, 16, 128, 128, spare=4)),
        # the library's decode batch, its states scattered over a larger pool
        dict(name='recurrent_256x1', **_recurrent(256, 1, 16, 128, 128, spare=32)),
        # verification of drafts of up to 8 tokens, part of each accepted; one decay and gate a head,
        # two value heads to a key head, bf16 output for the output projection
        dict(name='recurrent_draft_128x8', **_recurrent(128, 8, 32, 128, 128, out='bf16', gates='head', HK=16,
                                                        ragged=True, commit=True, spare=16)),
        # short prompts of 0 to 64 tokens in float32, one erase and write gate a head
        dict(name='recurrent_f32_48x64', **_recurrent(48, 64, 16, 128, 64, dtype='f32', gates='kda', HK=4,
                                                      ragged=True)),
        # the decode batch's raw inputs, history in place
        dict(name='prologue_256x1', **_prologue('prologue_fwd', 256, 1, 16, 128, 128, history=True)),
        # packed prompts of mixed length, about 32 thousand tokens
        dict(name='prologue_32x2048', **_prologue('prologue_fwd', 32, 2048, 16, 128, 128, ragged=True, history=True)),
        # a small fine-tuning batch in float32, odd length, narrower heads
        dict(name='prologue_bwd_f32_2x777', **_prologue('prologue_bwd', 2, 777, 8, 64, 64, dtype='f32')),
        # a training batch of packed sequences
        dict(name='prologue_bwd_8x4096', **_prologue('prologue_bwd', 8, 4096, 16, 128, 128, ragged=True)),
        # the decode batch after the output projection
        dict(name='layer_norm_256x2048', **_layer_norm('layer_norm_fwd', 256, 2048)),
        # the library's long prompt
        dict(name='layer_norm_65536x2048', **_layer_norm('layer_norm_fwd', 65536, 2048)),
        # an odd width in float32
        dict(name='layer_norm_bwd_f32_1111x1001', **_layer_norm('layer_norm_bwd', 1111, 1001, dtype='f32')),
        # a training step over the long prompt
        dict(name='layer_norm_bwd_65536x2048', **_layer_norm('layer_norm_bwd', 65536, 2048, residual=False)),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


_CAP = {}


def _plain_cost(case):
    """State elements times tokens that the recurrent plain form passes over, with its empty steps."""
    return case['N'] * case['T'] * case['H'] * case['dk'] * case['dv'] if case['op'] == 'recurrent' else 0


def _caps():
    if not _CAP:
        for c in listed():
            op = c['op']
            old = _CAP.get(op, (0, 0))
            _CAP[op] = (max(old[0], work(c)['bytes']), max(old[1], _plain_cost(c)))
    return _CAP


def draw(rng):
    while True:
        op = rng.choice(['recurrent', 'recurrent', 'prologue_fwd', 'prologue_bwd', 'layer_norm_fwd', 'layer_norm_bwd'])
        dtype = rng.choice(['bf16', 'bf16', 'f32'])
        if op.startswith('layer_norm'):
            c = _layer_norm(op, _log(rng, 1, 65536), _log(rng, 16, 8192), dtype, rng.random() < 0.5)
        else:
            H = rng.choice([1, 2, 3, 4, 6, 8, 12, 16, 24, 32])
            HK = rng.choice([h for h in range(1, H + 1) if H % h == 0])
            dk, dv = (rng.choice([16, 32, 64, 128, 128]) for _ in range(2))
            gates = rng.choice(['channel', 'channel', 'head', 'kda'])
            N = _log(rng, 1, 256)
            if op == 'recurrent':
                c = _recurrent(N, _log(rng, 1, 64), H, dk, dv, dtype, rng.choice(['f32', 'bf16']), gates, HK,
                               rng.random() < 0.6, rng.random() < 0.5, rng.randrange(0, 17))
            else:
                hist = rng.random() < 0.6
                c = _prologue(op, min(N, 64), _log(rng, 1, 8192), H, dk, dv, dtype, HK, rng.random() < 0.6, hist,
                              hist and op == 'prologue_fwd' and rng.random() < 0.5, gates)
        top = _caps()[op]
        if work(c)['bytes'] <= top[0] and _plain_cost(c) <= top[1]:
            return c


def _lengths(case):
    """Tokens of each sequence: T, or for ragged batches 0 to T with one of T."""
    N, T = case['N'], case['T']
    if not case['ragged']:
        return [T] * N
    r = random.Random(1009 * N + T)
    lens = [r.randint(0, T) for _ in range(N)]
    lens[r.randrange(N)] = T
    return lens


def work(case):
    op, e = case['op'], 2 if case['dtype'] == 'bf16' else 4
    if op == 'layer_norm_fwd':
        n = case['rows'] * case['cols']
        return {'bytes': n * e * (4 if case['residual'] else 2) + 8 * case['cols'],
                'flops': n * (9 if case['residual'] else 8)}
    if op == 'layer_norm_bwd':
        n = case['rows'] * case['cols']
        return {'bytes': n * e * (4 if case['residual'] else 3) + 12 * case['cols'], 'flops': n * 17}
    lens = _lengths(case)
    tok, N, H, HK, dk, dv = sum(lens), case['N'], case['H'], case['HK'], case['dk'], case['dv']
    nb = H * (dk if case['gates'] == 'channel' else 1)
    nw = H * (dv if case['gates'] == 'channel' else 1)
    raw = 2 * HK * dk + H * dv + nb + nw
    if op == 'recurrent':
        na = H * (1 if case['gates'] == 'head' else dk)
        oe = 2 if case['out'] == 'bf16' else 4
        return {'bytes': tok * (raw * e + 4 * na + H * dv * oe) + 8 * H * dk * dv * sum(1 for n in lens if n),
                'flops': 7 * tok * H * dk * dv}
    conv = 2 * HK * dk + H * dv
    hist = 3 * conv * e * N if case['history'] else 0
    if op == 'prologue_fwd':
        return {'bytes': 2 * tok * raw * e + 2 * hist + 20 * conv, 'flops': tok * (8 * conv + 6 * HK * dk + 4 * (nb + nw))}
    return {'bytes': tok * raw * (2 * e + 4) + hist + 40 * conv,
            'flops': tok * (26 * conv + 16 * HK * dk + 7 * (nb + nw))}


# ---- inputs ------------------------------------------------------------------

def prepare(case, seed):
    dev = torch.device('cuda')
    g = torch.Generator(device=dev).manual_seed(seed)
    dt = DTYPES[case['dtype']]
    op = case['op']

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev)

    s = {'case': case}
    if op.startswith('layer_norm'):
        R, C = case['rows'], case['cols']
        s['weight'] = 1 + 0.1 * normal(C)
        s['bias'] = 0.1 * normal(C)
        # rows of an activation stream: their scales and offsets differ
        s['x'] = (normal(R, C) * (0.5 + 2 * torch.rand(R, 1, generator=g, device=dev)) + normal(R, 1)).to(dt)
        if op == 'layer_norm_fwd':
            s['residual'] = normal(R, C).to(dt) if case['residual'] else None
        else:
            s['dy'] = normal(R, C).to(dt)
            s['dsum'] = normal(R, C).to(dt) if case['residual'] else None
        return s

    lens = _lengths(case)
    N, tok, H, HK, dk, dv = case['N'], sum(lens), case['H'], case['HK'], case['dk'], case['dv']
    lead = (1, tok) if case['ragged'] else (N, case['T'])
    s['cu'] = torch.tensor([0] + lens, device=dev).cumsum(0).to(torch.int32) if case['ragged'] else None
    s['lens'] = lens
    if case['commit']:
        n = torch.tensor(lens, device=dev)
        s['commit'] = (torch.rand(N, generator=g, device=dev) * (n + 1)).to(torch.int32)
    else:
        s['commit'] = None
    gates = case['gates']
    bshape = (*lead, H, dk) if gates == 'channel' else (*lead, H)
    wshape = (*lead, H, dv) if gates == 'channel' else (*lead, H)
    if op == 'recurrent':
        slots = case['slots']

        def unit(*shape):
            x = normal(*shape)
            return (x / x.norm(dim=-1, keepdim=True)).to(dt)

        s['q'], s['k'], s['v'] = unit(*lead, HK, dk), unit(*lead, HK, dk), normal(*lead, H, dv).to(dt)
        s['b'], s['w'] = torch.sigmoid(normal(*bshape)).to(dt), torch.sigmoid(normal(*wshape)).to(dt)
        x = normal(*((*lead, H) if gates == 'head' else (*lead, H, dk))) - 3
        s['log_alpha'] = -torch.log1p(torch.exp(x))
        s['pool'] = 0.1 * normal(slots, H, dk, dv)
        s['slot'] = torch.rand(slots, generator=g, device=dev).argsort()[:N].to(torch.int32)
        return s

    widths = (HK * dk, HK * dk, H * dv)
    s['raw'] = (normal(*lead, HK, dk).to(dt), normal(*lead, HK, dk).to(dt), normal(*lead, H, dv).to(dt))
    s['b_logit'], s['w_logit'] = normal(*bshape).to(dt), normal(*wshape).to(dt)
    s['weight'] = tuple(torch.rand(n, TAPS, generator=g, device=dev) - 0.5 for n in widths)
    s['bias'] = tuple(torch.rand(n, generator=g, device=dev) - 0.5 for n in widths)
    s['slot'] = s['history'] = None
    if case['history']:
        slots = N + 3
        s['history'] = tuple(normal(slots, h, TAPS - 1, d).to(dt) for h, d in ((HK, dk), (HK, dk), (H, dv)))
        s['slot'] = torch.rand(slots, generator=g, device=dev).argsort()[:N].to(torch.int32)
    if op == 'prologue_bwd':
        s['grads'] = tuple(normal(*x.shape) for x in (*s['raw'], s['b_logit'], s['w_logit']))
    return s


# ---- the operators in their plain form ---------------------------------------

def _starts(s):
    """First token and length of each sequence, and the sequence of each token."""
    case = s['case']
    dev = s['slot'].device if s['slot'] is not None else s['raw'][0].device
    N, T = case['N'], case['T']
    if s['cu'] is None:
        start = torch.arange(N, device=dev) * T
        n = torch.full((N,), T, device=dev)
        seq = torch.arange(N * T, device=dev) // T
    else:
        cu = s['cu'].long()
        start, n = cu[:-1], cu[1:] - cu[:-1]
        seq = torch.searchsorted(cu[1:], torch.arange(sum(s['lens']), device=dev), right=True)
    return start, n, seq


def _plain_recurrent(s):
    case = s['case']
    H, dk, dv, rep = case['H'], case['dk'], case['dv'], case['H'] // case['HK']
    start, n, _ = _starts(s)
    tokens = sum(s['lens'])
    flat = lambda x: x.flatten(0, 1)  # noqa: E731
    q, k, v, la, b, w = (flat(s[x]) for x in ('q', 'k', 'v', 'log_alpha', 'b', 'w'))
    slot = s['slot'].long()
    S = s['pool'][slot]
    commit = n if s['commit'] is None else s['commit'].long()
    kept = S
    # one row behind the last takes what the shorter sequences have no token for
    o = torch.empty(tokens + 1, H, dv, dtype=DTYPES[case['out']], device=S.device)
    per = lambda x, d: x.float() if x.dim() == 3 else x.float()[..., None].expand(-1, -1, d)  # noqa: E731
    for t in range(max(s['lens'])):
        live = t < n
        at = torch.where(live, start + t, 0)
        kt = k[at].float().repeat_interleave(rep, 1)
        qt = q[at].float().repeat_interleave(rep, 1)
        bk = per(b[at], dk) * kt
        S_new = torch.exp(per(la[at], dk))[..., None] * S
        delta = per(w[at], dv) * v[at].float() - (S_new * bk[..., None]).sum(-2)
        S_new = S_new + kt[..., None] * delta[..., None, :]
        o[torch.where(live, at, tokens)] = (S_new * qt[..., None]).sum(-2).to(o.dtype)
        S = torch.where(live[:, None, None, None], S_new, S)
        kept = torch.where((commit == t + 1)[:, None, None, None], S, kept)
    s['pool'][slot] = kept
    return o[:tokens].view(*s['v'].shape), s['pool']


def _plain_rows(s, x, hist, back):
    """x of ``back`` tokens earlier in the same sequence; before its start the history, or zeros."""
    start, _, seq = _starts(s)
    src = torch.arange(x.shape[0], device=x.device) - back
    before = src - start[seq]
    y = x[src.clamp_min(0)]
    if hist is None:
        old = torch.zeros((), dtype=x.dtype, device=x.device)
    else:
        old = hist[s['slot'].long()[seq], :, (TAPS - 1 + before).clamp(0, TAPS - 2)]
    return torch.where((before >= 0)[:, None, None], y, old).float()


def _plain_conv(s, i):
    x = s['raw'][i].flatten(0, 1)
    hist = None if s['history'] is None else s['history'][i]
    w = s['weight'][i].view(*x.shape[1:], TAPS)
    rows = [_plain_rows(s, x, hist, TAPS - 1 - j) for j in range(TAPS)]
    return rows, w, sum((w[..., j] * rows[j] for j in range(TAPS)), s['bias'][i].view(*x.shape[1:]))


def _plain_prologue_fwd(s):
    out = []
    for i, x in enumerate(s['raw']):
        _, _, y = _plain_conv(s, i)
        if i < 2:
            y = y / y.square().sum(-1, keepdim=True).sqrt().clamp_min(1e-12)
        out.append(y.to(x.dtype).view(x.shape))
    out += [(1 / (1 + torch.exp(-x.float()))).to(x.dtype) for x in (s['b_logit'], s['w_logit'])]
    if s['history'] is None:
        return out
    start, n, _ = _starts(s)
    commit = n if s['commit'] is None else s['commit'].long()
    slot = s['slot'].long()
    for x, hist in zip(s['raw'], s['history']):
        x = x.flatten(0, 1)
        back = commit[:, None] + torch.arange(1 - TAPS, 0, device=x.device)      # position of each kept input
        old = hist[slot].transpose(1, 2).gather(1, (back + TAPS - 1).clamp(0, TAPS - 2)[:, :, None, None].expand(
            -1, -1, *x.shape[1:]))
        new = x[(start[:, None] + back).clamp(0, x.shape[0] - 1)]
        hist[slot] = torch.where((back >= 0)[:, :, None, None], new, old).transpose(1, 2)
    return out + list(s['history'])


def _plain_prologue_bwd(s):
    start, n, seq = _starts(s)
    end = (start + n)[seq]
    out = {}
    for i, name in enumerate('qkv'):
        x = s['raw'][i]
        rows, w, y = _plain_conv(s, i)
        dy = s['grads'][i].flatten(0, 1)
        if i < 2:
            norm = y.square().sum(-1, keepdim=True).sqrt()
            u = y / norm.clamp_min(1e-12)
            along = torch.where(norm > 1e-12, (u * dy).sum(-1, keepdim=True), 0.0)
            dy = (dy - u * along) / norm.clamp_min(1e-12)
        dx = torch.zeros_like(dy)
        for j in range(TAPS):
            to = torch.arange(dy.shape[0], device=dy.device) + (TAPS - 1 - j)
            later = torch.where((to < end)[:, None, None], dy[to.clamp_max(dy.shape[0] - 1)], 0.0)
            dx = dx + w[..., j] * later
        out[name + '_raw'] = dx.to(x.dtype).view(x.shape)
        out['weight_' + name] = torch.stack([(dy * r).sum(0, dtype=torch.float64).flatten() for r in rows], -1).float()
        out['bias_' + name] = dy.sum(0, dtype=torch.float64).flatten().float()
    for name, d in zip(('b_logit', 'w_logit'), s['grads'][3:]):
        g = 1 / (1 + torch.exp(-s[name].float()))
        out[name] = (d * g * (1 - g)).to(s[name].dtype)
    return out


def _plain_layer_norm_fwd(s):
    h = s['x'].float()
    if s['residual'] is not None:
        h = h + s['residual'].float()
    c = h - h.mean(-1, keepdim=True)
    y = c / (c.square().mean(-1, keepdim=True) + EPS).sqrt() * s['weight'] + s['bias']
    y = y.to(s['x'].dtype)
    return y if s['residual'] is None else (y, h.to(s['x'].dtype))


def _plain_layer_norm_bwd(s):
    h, dy = s['x'].float(), s['dy'].float()
    c = h - h.mean(-1, keepdim=True)
    rstd = 1 / (c.square().mean(-1, keepdim=True) + EPS).sqrt()
    xh = c * rstd
    g = dy * s['weight']
    dh = rstd * (g - g.mean(-1, keepdim=True) - xh * (g * xh).mean(-1, keepdim=True))
    if s['dsum'] is not None:
        dh = dh + s['dsum'].float()
    return {'x': dh.to(s['x'].dtype), 'weight': (dy * xh).sum(0, dtype=torch.float64).float(),
            'bias': dy.sum(0, dtype=torch.float64).float()}


_PLAIN = {'recurrent': _plain_recurrent, 'prologue_fwd': _plain_prologue_fwd, 'prologue_bwd': _plain_prologue_bwd,
          'layer_norm_fwd': _plain_layer_norm_fwd, 'layer_norm_bwd': _plain_layer_norm_bwd}


# ---- the operators through the package ----------------------------------------

def _own(s):
    import gated_delta_rule_wy_amd as gdn2
    case = s['case']
    op = case['op']
    if op == 'recurrent':
        o = gdn2.recurrent_fwd(s['q'], s['k'], s['v'], s['log_alpha'], s['b'], s['w'], s['pool'], s['cu'],
                               slot_in=s['slot'], slot_out=s['slot'], commit=s['commit'],
                               out_dtype=DTYPES[case['out']])
        return o, s['pool']
    if op == 'prologue_fwd':
        out = gdn2.prologue_fwd(*s['raw'], s['b_logit'], s['w_logit'], s['weight'], s['bias'], s['cu'],
                                conv_state=s['history'], conv_state_out=s['history'], slot_in=s['slot'],
                                slot_out=s['slot'], commit=s['commit'])
        return list(out) if s['history'] is None else list(out) + list(s['history'])
    if op == 'prologue_bwd':
        return gdn2.prologue_bwd(*s['raw'], s['b_logit'], s['w_logit'], s['weight'], s['bias'], *s['grads'],
                                 s['cu'], conv_state=s['history'], slot_in=s['slot'])
    if op == 'layer_norm_fwd':
        y, h = gdn2.layer_norm_fwd(s['x'], s['weight'], s['bias'], s['residual'], eps=EPS,
                                   output_sum=s['residual'] is not None)
        return y if h is None else (y, h)
    return gdn2.layer_norm_bwd(s['dy'], s['x'], s['weight'], dsum=s['dsum'], eps=EPS)


def run(state):
    return _own(state) if own else _PLAIN[state['case']['op']](state)


# ---- the definitions in 64 bits -------------------------------------------------

def _exact_recurrent(s):
    """The printed form of the update, S <- (I - k (b*k)^T) Diag(alpha) S + k (w*v)^T, as matrix
    products, sequences of one length together."""
    case = s['case']
    H, dk, dv, rep = case['H'], case['dk'], case['dv'], case['H'] // case['HK']
    first = [sum(s['lens'][:i]) for i in range(case['N'])]
    by_len = {}
    for i, n in enumerate(s['lens']):
        by_len.setdefault(n, []).append(i)
    wide = lambda x, d: x if x.dim() == 3 else x[..., None].expand(*x.shape, d)  # noqa: E731
    tok = {x: s[x].flatten(0, 1).double() for x in ('q', 'k', 'v', 'log_alpha', 'b', 'w')}
    o = torch.zeros(sum(s['lens']), H, dv, dtype=torch.float64, device=s['v'].device)
    pool = s['pool'].double()
    commit = s['lens'] if s['commit'] is None else s['commit'].tolist()
    slot = s['slot'].tolist()
    eye = torch.eye(dk, dtype=torch.float64, device=o.device)
    for n, seqs in by_len.items():
        for part in (seqs[i:i + 64] for i in range(0, len(seqs), 64)):
            S = pool[[slot[i] for i in part]].reshape(-1, dk, dv)
            for t in range(n + 1):
                done = [j for j, i in enumerate(part) if commit[i] == t]
                if done:
                    pool[[slot[part[j]] for j in done]] = S.view(len(part), H, dk, dv)[done]
                if t == n:
                    break
                at = [first[i] + t for i in part]
                k, q = (tok[x][at].repeat_interleave(rep, 1).reshape(-1, dk, 1) for x in ('k', 'q'))
                b, a = (wide(tok[x][at], dk).reshape(-1, dk, 1) for x in ('b', 'log_alpha'))
                u = (wide(tok['w'][at], dv) * tok['v'][at]).reshape(-1, 1, dv)
                M = (eye - k * (b * k).reshape(-1, 1, dk)) * torch.exp(a).reshape(-1, 1, dk)
                S = torch.bmm(M, S) + k * u
                o[at] = torch.bmm(q.reshape(-1, 1, dk), S).view(len(part), H, dv)
    return o.view(s['v'].shape), pool


def _exact_mix(s, i, x, w, bias):
    """The convolution of one raw tensor, sequence by sequence over its padded rows."""
    out, at = [], 0
    rows = x.flatten(0, 1)
    for j, n in enumerate(s['lens']):
        if s['history'] is None:
            before = torch.zeros(TAPS - 1, *rows.shape[1:], dtype=rows.dtype, device=rows.device)
        else:
            before = s['history'][i][int(s['slot'][j])].transpose(0, 1).double()
        ext = torch.cat([before, rows[at:at + n]])
        y = bias.view(rows.shape[1:]).expand(n, *rows.shape[1:])
        for m in range(TAPS):
            y = y + ext[m:m + n] * w[:, m].view(rows.shape[1:])
        out.append(y)
        at += n
    y = torch.cat(out).view(x.shape)
    return y / torch.linalg.vector_norm(y, dim=-1, keepdim=True).clamp_min(1e-12) if i < 2 else y


def _exact_prologue_fwd(s):
    out = [_exact_mix(s, i, x.double(), s['weight'][i].double(), s['bias'][i].double())
           for i, x in enumerate(s['raw'])]
    out += [torch.sigmoid(x.double()) for x in (s['b_logit'], s['w_logit'])]
    if s['history'] is None:
        return out
    commit = s['lens'] if s['commit'] is None else s['commit'].tolist()
    for x, hist in zip(s['raw'], s['history']):
        rows, new, at = x.flatten(0, 1).double(), hist.double(), 0
        for j, n in enumerate(s['lens']):
            p = int(s['slot'][j])
            new[p] = torch.cat([new[p].transpose(0, 1), rows[at:at + commit[j]]])[-(TAPS - 1):].transpose(0, 1)
            at += n
        out.append(new)
    return out


def _exact_prologue_bwd(s):
    out = {}
    with torch.enable_grad():
        for i, name in enumerate('qkv'):
            leaves = [t.double().requires_grad_() for t in (s['raw'][i], s['weight'][i], s['bias'][i])]
            y = _exact_mix(s, i, *leaves)
            out[name + '_raw'], out['weight_' + name], out['bias_' + name] = torch.autograd.grad(
                y, leaves, s['grads'][i].double())
        for name, d in zip(('b_logit', 'w_logit'), s['grads'][3:]):
            x = s[name].double().requires_grad_()
            out[name], = torch.autograd.grad(torch.sigmoid(x), x, d.double())
    return out


def _exact_norm(h, weight, bias):
    var, mean = torch.var_mean(h, dim=-1, keepdim=True, correction=0)
    return (h - mean) / torch.sqrt(var + EPS) * weight + bias


def _exact_layer_norm_fwd(s):
    h = s['x'].double() + (0 if s['residual'] is None else s['residual'].double())
    y = _exact_norm(h, s['weight'].double(), s['bias'].double())
    return y if s['residual'] is None else (y, h)


def _exact_layer_norm_bwd(s):
    with torch.enable_grad():
        leaves = [s[x].double().requires_grad_() for x in ('x', 'weight', 'bias')]
        dx, dw, db = torch.autograd.grad(_exact_norm(*leaves), leaves, s['dy'].double())
    return {'x': dx if s['dsum'] is None else dx + s['dsum'].double(), 'weight': dw, 'bias': db}


_EXACT = {'recurrent': _exact_recurrent, 'prologue_fwd': _exact_prologue_fwd, 'prologue_bwd': _exact_prologue_bwd,
          'layer_norm_fwd': _exact_layer_norm_fwd, 'layer_norm_bwd': _exact_layer_norm_bwd}


def exact(case, seed):
    with torch.no_grad():
        return _EXACT[case['op']](prepare(case, seed))
