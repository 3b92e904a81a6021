"""The dense operators as a layer uses them, around the mixer, against float64:

* serving: residual stream -> RMS norm in 8 bits -> projections to q, k, v and the gates -> prologue ->
  recurrence -> output projection onto the residual stream;
* a training step of a feed-forward pair, norm -> product with silu -> product onto the residual,
  back through both, and the clipping of all gradients;
* a training step of a whole layer around the mixer, from end to end in float64 (its own bar there).

The references take each operator's inputs from the previous one's result on the GPU where that was
rounded to 8 or 16 bits (a rounding that falls to the other side is then not carried along), so every
operator is held to its own tolerance."""
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

E4M3 = torch.float8_e4m3fn


def back(t):
    return t.float().cpu().numpy()


def eight_bits(w):
    s = w.abs().amax(1) / 448
    return (w / s[:, None]).to(E4M3), s


def test_serving_layer():
    B, T, H, d = 2, 5, 4, 64
    D, rows = H * d, B * T
    g = torch.Generator().manual_seed(1)
    n = lambda *s: torch.randn(s, generator=g).to(DEV)   # noqa: E731
    stream, last = n(rows, D).bfloat16(), n(rows, D).bfloat16()
    norm_w = 1 + 0.1 * n(D)
    proj = {k: eight_bits(n(D, D) / D ** 0.5) for k in ('q', 'k', 'v', 'b', 'w', 'o')}
    wf, bf = tuple(torch.rand(D, 4, generator=g).to(DEV) - 0.5 for _ in range(3)), 0.1 * n(D)
    la = -torch.nn.functional.softplus(n(B, T, H, d) - 3)
    state = torch.zeros(B, H, d, d, device=DEV)

    y, h, scale = gdn2.rms_norm_fwd(last, norm_w, stream, output_sum=True, out_dtype=E4M3)
    (wq, ws, wh) = ref.rms_norm_fwd(back(last), back(norm_w), back(stream), out_dtype='e4m3', in_dtype='bf16')
    oref.check('q', back(y), wq)
    oref.check('scale', back(scale), ws)
    oref.check('h', back(h), wh)
    raw = {}
    for k in 'qkvbw':
        w8, sw = proj[k]
        raw[k], _ = gdn2.linear_fwd(y, w8, bf if k in 'bw' else None, x_scale=scale, weight_scale=sw)
        want, _ = ref.linear_fwd(back(y), back(w8), back(bf) if k in 'bw' else None, None, 'none', back(scale), back(sw), 'bf16')
        oref.check(k, back(raw[k]), want)
    q, k, v, b, w = gdn2.prologue_fwd(*(raw[c].view(B, T, H, d) for c in 'qkvbw'), wf)
    o = gdn2.recurrent_fwd(q, k, v, la, b, w, state, out_dtype=torch.bfloat16)
    o8 = o.view(rows, D).float()
    so = o8.abs().amax(1) / 448
    o8 = (o8 / so[:, None]).to(E4M3)
    out, _ = gdn2.linear_fwd(o8, proj['o'][0], None, h, x_scale=so, weight_scale=proj['o'][1], out=h.clone())
    want, _ = ref.linear_fwd(back(o8), back(proj['o'][0]), None, back(h), 'none', back(so), back(proj['o'][1]), 'bf16')
    oref.check('stream', back(out), want)
    # the sigmoid in the projection's epilogue is the prologue's
    gate, _ = gdn2.linear_fwd(y, proj['b'][0], bf, activation='sigmoid', x_scale=scale, weight_scale=proj['b'][1], out_dtype=torch.float32)
    # (from bf16 logits there: half a step of the logit, a quarter of it in the gate, and the gate's own)
    lim = (np.abs(back(raw['b'])) / 4 + 1) * 2.0 ** -8 + 1e-5
    assert np.all(np.abs(back(gate) - back(b).reshape(rows, D)) <= lim)


@pytest.mark.parametrize('dtype', ['bf16', 'f32'])
def test_training_step(dtype):
    M, D, F = 700, 160, 500
    dt = {'bf16': torch.bfloat16, 'f32': torch.float32}[dtype]
    g = torch.Generator().manual_seed(2)
    n = lambda *s: torch.randn(s, generator=g).to(DEV)   # noqa: E731
    x, r, dout = n(M, D).to(dt), n(M, D).to(dt), n(M, D).to(dt)
    wn, w1, b1, w2, b2 = 1 + 0.1 * n(D), (n(F, D) / D ** 0.5).to(dt), 0.1 * n(F), (n(D, F) / F ** 0.5).to(dt), 0.1 * n(D)

    y, h, _ = gdn2.rms_norm_fwd(x, wn, r, output_sum=True)
    u, z = gdn2.linear_fwd(y, w1, b1, activation='silu', output_preact=True)
    out, _ = gdn2.linear_fwd(u, w2, b2, h)
    g2 = gdn2.linear_bwd(dout, u, w2)
    g1 = gdn2.linear_bwd(g2['x'], y, w1, z, activation='silu')
    gn = gdn2.rms_norm_bwd(g1['x'], h, wn, dsum=dout)
    grads = [gn['weight'], g1['weight'], g1['bias'], g2['weight'], g2['bias']]
    raw = [back(t) for t in grads]
    norm = gdn2.clip_grads(grads, 0.5)

    f = back
    oref.check('y', f(y), ref.rms_norm_fwd(f(x), f(wn), f(r), out_dtype=dtype)[0])
    wu, wz = ref.linear_fwd(f(y), f(w1), f(b1), None, 'silu', out_dtype=dtype, z_dtype=dtype)
    oref.check('u', f(u), wu)
    oref.check('z', f(z), wz)
    oref.check('out', f(out), ref.linear_fwd(f(u), f(w2), f(b2), f(h), out_dtype=dtype)[0])
    for got, want in ((g2, ref.linear_bwd(f(dout), f(u), f(w2), dtype=dtype)),
                      (gn, ref.rms_norm_bwd(f(g1['x']), f(h), f(wn), f(dout), dtype=dtype)),
                      (g1, ref.linear_bwd(f(g2['x']), f(y), f(w1), f(z), 'silu', dtype))):
        if got is not gn:
            oref.check('dx', f(got['x']), want['x'])
        else:
            oref.check('dh', f(got['x']), want['x'])
    wantn, tol = ref.grad_norm(raw)
    assert abs(float(norm) - wantn) <= tol
    for t, w in zip(grads, ref.clip(raw, 0.5, ['bf16' if t.dtype == torch.bfloat16 else 'f32' for t in grads])):
        oref.check('clipped', f(t), w)
    # and the weights' gradients themselves
    for t, (w, tol) in zip(raw, (ref.rms_norm_bwd(f(g1['x']), f(h), f(wn), dtype=dtype)['weight'],
                                 *(ref.linear_bwd(f(g2['x']), f(y), f(w1), f(z), 'silu', dtype)[k] for k in ('weight', 'bias')),
                                 *(ref.linear_bwd(f(dout), f(u), f(w2), dtype=dtype)[k] for k in ('weight', 'bias')))):
        oref.check('gradient', t, (w, tol))


def test_training_layer():
    """One layer's training step in fp32, whole: norm, projections, prologue, mixer, output projection onto the
    residual stream, all of it back, and the clipping of the weights' gradients. Against one float64 run from end to end:
    the mixer's own bar on such inputs is 1e-4 on values of order 1, and the steps around it multiply that by at most
    rstd |W| |weight| (below 10 here) in each direction, so results are held to 1e-3 of the largest reference value."""
    import oracle
    from gpu_util import threads
    lens, H, d = [70, 0, 130, 5], 2, 32
    T, D = sum(lens), H * d
    rng = np.random.default_rng(5)
    f = lambda *s: rng.standard_normal(s).astype(np.float32)   # noqa: E731
    x, r, dout, la = f(T, D), f(T, D), f(T, D), -np.logaddexp(0, f(T, H, d) - 3).astype(np.float32)
    wn, W, bias = 1 + f(D) / 10, {k: f(D, D) / np.float32(np.sqrt(D)) for k in 'qkvbwo'}, {k: f(D) / 10 for k in 'bw'}
    taps, tb = [rng.uniform(-.5, .5, (D, 4)).astype(np.float32) for _ in range(3)], [rng.uniform(-.5, .5, D).astype(np.float32) for _ in range(3)]
    cu_np = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)

    def near(name, got, want):
        got = got.detach().double().cpu().numpy().reshape(want.shape)
        err, top = np.abs(got - want).max(), np.abs(want).max()
        print(f'{name}: {err / top:.1e} of the largest value', flush=True)
        assert np.all(np.isfinite(got)) and err <= 1e-3 * top, f'{name}: off by {err:.3e}, largest value {top:.3e}'

    # float64
    (y, _), (h, _) = ref.rms_norm_fwd(x, wn, r)
    raw = {k: ref.linear_fwd(y, W[k], bias.get(k))[0][0].reshape(T, H, d) for k in 'qkvbw'}
    pro, _ = oref.prologue_fwd([raw[k] for k in 'qkv'], [raw[k] for k in 'bw'], taps, tb, lens)
    q, k, v, b, w = (t for t, _ in pro)
    o, _ = oracle.forward(q, k, v, la, b, w, None, cu_seqlens=cu_np, nthreads=threads())
    out = ref.linear_fwd(o.reshape(T, D), W['o'], None, h)[0][0]
    go = {n: t for n, (t, _) in ref.linear_bwd(dout, o.reshape(T, D), W['o']).items()}
    gm = oracle.backward(q, k, v, la, b, w, None, go['x'].reshape(T, H, d), None, cu_seqlens=cu_np)
    gp = oref.prologue_bwd([raw[k] for k in 'qkv'], [raw[k] for k in 'bw'], taps, tb, [gm[n] for n in 'qkvbw'], lens)
    at = dict(zip('qkvbw', ('q_raw', 'k_raw', 'v_raw', 'b_logit', 'w_logit')))
    gl = {c: {n: t for n, (t, _) in ref.linear_bwd(gp[at[c]][0].reshape(T, D), y, W[c]).items()} for c in 'qkvbw'}
    gn = {n: t for n, (t, _) in ref.rms_norm_bwd(sum(g['x'] for g in gl.values()), h, wn, dout).items()}

    # the library
    G = lambda t: torch.from_numpy(np.ascontiguousarray(t)).to(DEV)   # noqa: E731
    X, R, DO, WN, LA, CU = G(x), G(r), G(dout), G(wn), G(la).unsqueeze(0), G(cu_np)
    WG, BG, TAPS, TB = {c: G(t) for c, t in W.items()}, {c: G(t) for c, t in bias.items()}, tuple(map(G, taps)), tuple(map(G, tb))
    Y, Hs, _ = gdn2.rms_norm_fwd(X, WN, R, output_sum=True)
    RAW = [gdn2.linear_fwd(Y, WG[c], BG.get(c))[0].view(1, T, H, d) for c in 'qkvbw']
    MIX = gdn2.prologue_fwd(*RAW, TAPS, TB, CU)
    args = (*MIX[:3], LA, *MIX[3:], None)
    O, _, ws = gdn2.chunk_fwd_keep(*args, CU)
    O = O.view(T, D)
    OUT, _ = gdn2.linear_fwd(O, WG['o'], None, Hs)
    GO = gdn2.linear_bwd(DO, O, WG['o'], output_bias=False)
    GM = gdn2.chunk_bwd_kept(*args, GO['x'].view(1, T, H, d), None, CU, workspace=ws)
    GP = gdn2.prologue_bwd(*RAW, TAPS, TB, *(GM[c] for c in 'qkvbw'), CU)
    GL = {c: gdn2.linear_bwd(GP[at[c]].view(T, D), Y, WG[c], output_bias=c in BG) for c in 'qkvbw'}
    DY = sum(g['x'] for g in GL.values())
    GN = gdn2.rms_norm_bwd(DY, Hs, WN, dsum=DO)

    near('out', OUT, out)
    near('dx', GN['x'], gn['x'])
    near('d norm', GN['weight'], gn['weight'])
    near('d log_alpha', GM['log_alpha'], gm['log_alpha'])
    near('dWo', GO['weight'], go['weight'])
    grads, want = [GN['weight'], GO['weight']], [gn['weight'], go['weight']]
    for c in 'qkvbw':
        for n in ('weight', 'bias') if c in BG else ('weight',):
            near(f'd{n} {c}', GL[c][n], gl[c][n])
            grads.append(GL[c][n])
            want.append(gl[c][n])
    for n in sorted(set(gp) - set(at.values())):
        near(f'd{n}', GP[n], gp[n][0])
        grads.append(GP[n])
        want.append(gp[n][0])
    raw_grads = [back(t) for t in grads]
    norm = gdn2.clip_grads(grads, 0.5)
    n64 = np.sqrt(sum((t ** 2).sum() for t in want))
    assert abs(float(norm) - n64) <= 1e-3 * n64
    assert float(norm) > 0.5    # (so that they are clipped)
    for t, (c, tol) in zip(grads, ref.clip(raw_grads, 0.5, ['f32'] * len(grads))):
        oref.check('clipped', back(t), (c, tol))
