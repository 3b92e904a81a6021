"""The operators as they are used together, against float64:

* a training step of the whole layer between its projections: prologue_fwd,
  chunk_fwd_keep, an output projection (torch), layer_norm_fwd, and back through
  layer_norm_bwd, chunk_bwd_kept and prologue_bwd to the projections' outputs;
* serving with states and convolution histories in slots: prompts, single
  tokens, and drafts of which a part is accepted and the rest sent again.

All inputs are fp32. The mixer's own bar on such inputs is 1e-4 on values of
order 1; the steps around it multiply that by at most rstd |W| |weight| (below
10 here) in each direction, so the results are held to 1e-3 of the largest
reference value, far below what any wrong term would move."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip('torch')
if not torch.cuda.is_available():
    pytest.skip('no GPU', allow_module_level=True)

import gated_delta_rule_wy_amd as gdn2  # noqa: E402
import operator_reference as ref  # noqa: E402
import oracle  # noqa: E402
from gpu_util import DEV, threads  # noqa: E402

BAR = 1e-3


def close(name, got, want):
    got = got.detach().double().cpu().numpy().reshape(want.shape)
    err, top = np.abs(got - want).max(), np.abs(want).max()
    assert np.all(np.isfinite(got)) and err <= BAR * top, f'{name}: off by {err:.3e}, largest value {top:.3e}'
    print(f'{name}: {err / top:.1e} of the largest value', flush=True)


def gpu(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(DEV)


class Layer:
    def __init__(self, seed, T, H, d):
        rng = np.random.default_rng(seed)
        f = lambda *s: rng.standard_normal(s).astype(np.float32)   # noqa: E731
        self.T, self.H, self.d, self.D = T, H, d, H * d
        self.raw = [f(T, H, d) for _ in range(5)]
        self.la = -np.logaddexp(0, f(T, H, d) - 3).astype(np.float32)
        self.weight = [rng.uniform(-.5, .5, (H * d, 4)).astype(np.float32) for _ in range(3)]
        self.bias = [rng.uniform(-.5, .5, H * d).astype(np.float32) for _ in range(3)]
        self.proj = f(self.D, self.D) / np.float32(np.sqrt(self.D))
        self.x = f(T, self.D)
        self.ln_w, self.ln_b = 1 + f(self.D) / 10, f(self.D) / 10


def test_training_step():
    lens, H, d = [70, 0, 130, 5], 2, 32
    L = Layer(1, sum(lens), H, d)
    T, D = L.T, L.D
    dy = np.random.default_rng(2).standard_normal((T, D)).astype(np.float32)
    cu_np = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)

    # float64, operator by operator
    pro, _ = ref.prologue_fwd(L.raw[:3], L.raw[3:], L.weight, L.bias, lens)
    q, k, v, b, w = (x for x, _ in pro)
    o, _ = oracle.forward(q, k, v, L.la, b, w, None, cu_seqlens=cu_np, nthreads=threads())
    P = L.proj.astype(np.float64)
    (y, _), (h, _) = ref.layer_norm_fwd(L.x, L.ln_w, L.ln_b, o.reshape(T, D) @ P)
    ln = ref.layer_norm_bwd(dy, h, L.ln_w)
    do = (ln['x'][0] @ P.T).reshape(T, H, d)
    g = oracle.backward(q, k, v, L.la, b, w, None, do, None, cu_seqlens=cu_np)
    pg = ref.prologue_bwd(L.raw[:3], L.raw[3:], L.weight, L.bias, [g[n] for n in ('q', 'k', 'v', 'b', 'w')], lens)

    raw = [gpu(x).unsqueeze(0) for x in L.raw]
    weight, bias = tuple(map(gpu, L.weight)), tuple(map(gpu, L.bias))
    la, cu = gpu(L.la).unsqueeze(0), torch.from_numpy(cu_np).to(DEV)
    mix = gdn2.prologue_fwd(*raw, weight, bias, cu)
    args = (*mix[:3], la, *mix[3:], None)
    go, _, ws = gdn2.chunk_fwd_keep(*args, cu)
    gp = gpu(L.proj)
    gy, gh = gdn2.layer_norm_fwd(gpu(L.x), gpu(L.ln_w), gpu(L.ln_b), go.view(T, D) @ gp, output_sum=True)
    gl = gdn2.layer_norm_bwd(gpu(dy), gh, gpu(L.ln_w))
    gdo = (gl['x'] @ gp.T).view(1, T, H, d)
    gg = gdn2.chunk_bwd_kept(*args, gdo, None, cu, workspace=ws)
    gr = gdn2.prologue_bwd(*raw, weight, bias, gg['q'], gg['k'], gg['v'], gg['b'], gg['w'], cu)
    torch.cuda.synchronize()

    close('y', gy, y)
    for n in ('x', 'weight', 'bias'):
        close(f'layer norm d{n}', gl[n], ln[n][0])
    close('d log_alpha', gg['log_alpha'], g['log_alpha'])
    for n in pg:
        close(f'd{n}', gr[n], pg[n][0])


def test_serving_with_drafts():
    """Three requests in a pool of six slots. Every call mixes a prompt, single tokens and drafts;
    a draft's rejected tail is replaced by the true tokens in the next call."""
    H, d, slots = 4, 64, 6
    total = [37, 29, 41]
    L = Layer(3, sum(total), H, d)
    first = np.concatenate([[0], np.cumsum(total)])
    # (tokens sent, tokens kept) of each request in each call; what is not kept is sent again
    calls = [[(20, 20), (9, 9), (30, 30)], [(1, 1), (6, 2), (1, 1)], [(8, 8), (1, 1), (0, 0)], [(5, 0), (3, 3), (4, 1)],
             [(1, 1), (8, 5), (1, 1)], [(7, 7), (9, 9), (8, 8)]]
    assert [sum(c[i][1] for c in calls) for i in range(3)] == total
    slot = [4, 0, 5]
    rng = np.random.default_rng(4)
    hist = tuple(gpu(rng.standard_normal((slots, H, 3, d))) for _ in range(3))
    state = gpu(rng.standard_normal((slots, H, d, d)) / 10)
    hist0, state0 = [x.cpu().numpy() for x in hist], state.cpu().numpy()
    weight, bias = tuple(map(gpu, L.weight)), tuple(map(gpu, L.bias))
    sl = torch.tensor(slot, dtype=torch.int32, device=DEV)
    y = np.zeros((L.T, L.D))
    done = [0, 0, 0]
    for call in calls:
        at, ok = [], []
        for i, (sent, kept) in enumerate(call):
            rows = np.arange(first[i] + done[i], first[i] + done[i] + sent)
            at.append(np.minimum(rows, first[i + 1] - 1))   # (a draft past the end repeats the last row)
            ok += [r < kept for r in range(sent)]
        lens = [len(a) for a in at]
        at, ok = np.concatenate(at), np.array(ok, bool)
        rows = [x[at].copy() for x in (*L.raw, L.la)]
        for x in rows:
            x[~ok] = -np.abs(x[~ok][..., ::-1])   # wrong guesses
        cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device=DEV)
        keep = torch.tensor([c[1] for c in call], dtype=torch.int32, device=DEV)
        *raw, la = (gpu(x).unsqueeze(0) for x in rows)
        q, k, v, b, w = gdn2.prologue_fwd(*raw, weight, bias, cu, conv_state=hist, conv_state_out=hist, slot_in=sl,
                                          commit=keep)
        o = gdn2.recurrent_fwd(q, k, v, la, b, w, state, cu, slot_in=sl, commit=keep)
        out = gdn2.layer_norm_fwd(gpu(L.x[at]), gpu(L.ln_w), gpu(L.ln_b), o.view(len(at), L.D))[0]
        y[at[ok]] = out.double().cpu().numpy()[ok]
        done = [n + c[1] for n, c in zip(done, call)]
    # one run over the true tokens
    pro, pools = ref.prologue_fwd(L.raw[:3], L.raw[3:], L.weight, L.bias, total, hist0, slot)
    q, k, v, b, w = (x for x, _ in pro)
    (o, _), (after, _) = ref.recurrent(q, k, v, L.la, b, w, state0, total, slot)
    want = ref.layer_norm_fwd(L.x, L.ln_w, L.ln_b, o.reshape(L.T, L.D))[0][0]
    close('y', torch.from_numpy(y), want)
    close('states', state, after)
    for got, exp in zip(hist, pools):
        assert np.array_equal(got.cpu().numpy(), exp.astype(np.float32))
