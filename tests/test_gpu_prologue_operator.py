"""gdn2_prologue_fwd / gdn2_prologue_bwd (the prologue on its own and its
gradient) against float64: head sizes and ratios, types, gate layouts; lengths
around the tiles; histories in slots, commits, empty sequences; streams and
captured graphs. Histories are copies of raw inputs and must match bit for bit."""
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
NAMES = ('q', 'k', 'v', 'b', 'w')


class Batch:
    def __init__(self, seed, lens, H=2, HK=None, dk=32, dv=32, dtype='bf16', gates='channel', slots=None, bias=True,
                 tail=0):
        rng = np.random.default_rng(seed)
        HK = HK or H
        T = sum(lens) + tail
        rnd = gi.bf16_round if dtype == 'bf16' else (lambda x: np.asarray(x, np.float32))
        n = lambda *s: rng.standard_normal(s).astype(np.float32)   # noqa: E731
        shapes = ((HK, dk), (HK, dk), (H, dv))
        self.lens, self.dtype = lens, dtype
        self.raw = [rnd(n(T, *s)) for s in shapes]
        chan = gates == 'channel'
        self.logits = [rnd(2 * n(T, H, dk) if chan else 2 * n(T, H)), rnd(2 * n(T, H, dv) if chan else 2 * n(T, H))]
        self.weight = [rng.uniform(-.5, .5, (s[0] * s[1], 4)).astype(np.float32) for s in shapes]
        self.bias = [rng.uniform(-.5, .5, s[0] * s[1]).astype(np.float32) if bias else None for s in shapes]
        self.hist = None if slots is None else [rnd(n(slots, s[0], 3, s[1])) for s in shapes]
        self.grads = [n(*x.shape) for x in (*self.raw, *self.logits)]
        self.cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)

    def gpu(self):
        to = lambda x, dt: torch.from_numpy(x).to(DEV).to(dt)   # noqa: E731
        dt = DT[self.dtype]
        raw = [to(x, dt).unsqueeze(0) for x in (*self.raw, *self.logits)]
        weight = tuple(to(x, torch.float32) for x in self.weight)
        bias = None if self.bias[0] is None else tuple(None if x is None else to(x, torch.float32) for x in self.bias)
        hist = None if self.hist is None else tuple(to(x, dt) for x in self.hist)
        return raw, weight, bias, hist, to(self.cu, torch.int32)


def ints(x):
    return None if x is None else torch.tensor(x, dtype=torch.int32, device=DEV)


def back(t):
    return t.float().cpu().numpy()


def check_fwd(p, label, inplace=True, **kw):
    print(f'[{label}] lens={p.lens} {p.dtype}', flush=True)
    raw, weight, bias, hist, cu = p.gpu()
    out_hist = None if hist is None else (hist if inplace else tuple(h.clone() for h in hist))
    out = gdn2.prologue_fwd(*raw, weight, bias, cu, conv_state=hist, conv_state_out=out_hist,
                            **{k: ints(v) for k, v in kw.items()})
    n = sum(p.lens)
    want, pools = ref.prologue_fwd([x[:n] for x in p.raw], [x[:n] for x in p.logits], p.weight, p.bias, p.lens, p.hist,
                                   dtype=p.dtype, **kw)
    worst = [ref.check(f'{label} {m}', back(x)[0, :n], y) for m, x, y in zip(NAMES, out, want)]
    if pools is not None:
        for m, got, exp in zip(NAMES, out_hist, pools):
            assert np.array_equal(back(got), exp.astype(np.float32)), f'{label}: history of {m}'
    print(f'{label}: {max(worst):.3f} of the tolerance', flush=True)


def check_bwd(p, label, slot_in=None):
    print(f'[{label}] lens={p.lens} {p.dtype}', flush=True)
    raw, weight, bias, hist, cu = p.gpu()
    grads = [torch.from_numpy(x).to(DEV).unsqueeze(0) for x in p.grads]
    g = gdn2.prologue_bwd(*raw, weight, bias, *grads, cu, conv_state=hist, slot_in=ints(slot_in))
    n = sum(p.lens)
    want = ref.prologue_bwd([x[:n] for x in p.raw], [x[:n] for x in p.logits], p.weight, p.bias,
                            [x[:n] for x in p.grads], p.lens, p.hist, slot_in, dtype=p.dtype)
    assert sorted(want) == sorted(g)
    worst = 0
    for m in want:
        x = back(g[m])
        worst = max(worst, ref.check(f'{label} {m}', x[0, :n] if m.endswith(('raw', 'logit')) else x, want[m]))
    print(f'{label}: {worst:.3f} of the tolerance', flush=True)


SHORT = [1, 0, 2, 3, 0, 4, 5]                       # 15 tokens: one thread walks a sequence
LONG = [1, 0, 33, 2, 64, 0, 0, 3, 31, 5, 100, 32]   # tiles that sequences start and end in


@pytest.mark.parametrize('dtype', ['bf16', 'f32'])
@pytest.mark.parametrize('dk,dv', [(16, 16), (16, 128), (32, 64), (64, 32), (128, 128)])
def test_head_sizes(dk, dv, dtype):
    for lens in (SHORT, LONG):
        p = Batch(dk + dv, lens, H=3, dk=dk, dv=dv, dtype=dtype)
        check_fwd(p, f'fwd {dk}x{dv}')
        check_bwd(p, f'bwd {dk}x{dv}')


@pytest.mark.parametrize('gates', ['channel', 'head'])
@pytest.mark.parametrize('H,HK', [(4, 2), (5, 1), (16, 16)])
@pytest.mark.parametrize('bias', [True, False])
def test_heads_gates_bias(H, HK, gates, bias):
    p = Batch(2, LONG, H=H, HK=HK, dk=64, dv=32, gates=gates, bias=bias)
    check_fwd(p, f'fwd {H}/{HK} {gates}')
    check_bwd(p, f'bwd {H}/{HK} {gates}')


@pytest.mark.parametrize('lens', [SHORT, LONG])
@pytest.mark.parametrize('inplace', [True, False])
@pytest.mark.parametrize('dtype', ['bf16', 'f32'])
def test_histories(lens, inplace, dtype):
    N = len(lens)
    rng = np.random.default_rng(N)
    p = Batch(3, lens, H=4, HK=2, dk=32, dv=64, dtype=dtype, slots=N + 4)
    slot = rng.permutation(N + 4)[:N].tolist()
    check_fwd(p, 'slots', inplace, slot_in=slot)
    check_fwd(p, 'commit', inplace, slot_in=slot, commit=[max(n - i % 4, 0) for i, n in enumerate(lens)])
    check_bwd(p, 'bwd slots', slot)


@pytest.mark.parametrize('dtype', ['bf16', 'f32'])
@pytest.mark.parametrize('top', [1, 2, 3, 4, 6, 9])
def test_packed_short_sequences(top, dtype):
    """Sequences of 0 .. top tokens, packed: tiles of one to four tokens that several sequences share and that cut
    sequences within their first three tokens; the pools in place, kept in their slots or moved."""
    rng = np.random.default_rng(top)
    lens = rng.integers(0, top + 1, 61).tolist()
    N = len(lens)
    commit = rng.integers(-1, top + 2, N).tolist()
    perm = rng.permutation(2 * N + 3)
    p = Batch(20 + top, lens, H=4, HK=2, dk=32, dv=64, dtype=dtype, slots=2 * N + 3)
    check_fwd(p, f'kept {top}', True, slot_in=perm[:N].tolist())
    check_fwd(p, f'commit {top}', True, slot_in=perm[:N].tolist(), commit=commit)
    check_fwd(p, f'moved {top}', True, slot_in=perm[:N].tolist(), slot_out=perm[N:2 * N].tolist(), commit=commit)
    check_bwd(p, f'bwd {top}', perm[:N].tolist())


@pytest.mark.parametrize('N', [17, 70, 300])
def test_packed_single_tokens(N):
    p = Batch(40 + N, [1] * N, H=4, HK=4, dk=128, dv=128, slots=N + 2)
    slot = np.random.default_rng(N).permutation(N + 2)[:N].tolist()
    check_fwd(p, f'single {N}', True, slot_in=slot)


@pytest.mark.parametrize('lens', [SHORT, LONG])
def test_history_slots_none_forked_and_moved(lens):
    """None in, none out, two sequences from one slot, another slot out, negative and large commits."""
    N = len(lens)
    slot_in, slot_out = list(range(N)), list(range(N))
    slot_in[0], slot_in[2], slot_in[3], slot_out[3], slot_out[5] = -1, 1, N + 40, N + 2, -7
    slot_in[1], slot_out[2] = 1, N + 1
    p = Batch(4, lens, H=2, dk=32, dv=32, slots=N + 3)
    check_fwd(p, 'slots', False, slot_in=slot_in, slot_out=slot_out, commit=[-1 if i == 4 else 99 for i in range(N)])
    check_bwd(p, 'bwd', slot_in)


@pytest.mark.parametrize('N,T', [(1, 1), (5, 1), (3, 8), (4, 16), (2, 17), (3, 45), (1, 300)])
def test_uniform_batches(N, T):
    print(f'[uniform] N={N} T={T}', flush=True)
    p = Batch(5, [T] * N, H=2, dk=64, dv=128, slots=N)
    raw, weight, bias, hist, _ = p.gpu()
    raw = [x.reshape(N, T, *x.shape[2:]) for x in raw]
    out = gdn2.prologue_fwd(*raw, weight, bias, conv_state=hist, conv_state_out=hist)
    want, pools = ref.prologue_fwd(p.raw, p.logits, p.weight, p.bias, p.lens, p.hist, dtype='bf16')
    for m, x, y in zip(NAMES, out, want):
        ref.check(m, back(x).reshape(y[0].shape), y)
    for got, exp in zip(hist, pools):
        assert np.array_equal(back(got), exp.astype(np.float32))
    grads = [torch.from_numpy(x).to(DEV).reshape(r.shape) for x, r in zip(p.grads, raw)]
    g = gdn2.prologue_bwd(*raw, weight, bias, *grads)
    want = ref.prologue_bwd(p.raw, p.logits, p.weight, p.bias, p.grads, p.lens, dtype='bf16')
    for m in want:
        ref.check(m, back(g[m]), want[m])


def test_long_batch():
    """Several tiles of the gradient a sequence, sums over many partial rows."""
    p = Batch(6, [1500, 0, 2100, 7], H=8, dk=128, dv=128)
    check_fwd(p, 'long fwd')
    check_bwd(p, 'long bwd')


@pytest.mark.parametrize('lens', [[3, 5], [40, 55]])
def test_rows_behind_the_last_sequence(lens):
    p = Batch(7, lens, H=2, dk=32, dv=32, tail=37)
    raw, weight, bias, _, cu = p.gpu()
    n = sum(lens)
    out = [torch.full_like(x, 3.5) for x in raw]
    gdn2.prologue_fwd(*raw, weight, bias, cu, out=out)
    assert all(torch.all(x[0, n:] == 3.5) for x in out)
    want, _ = ref.prologue_fwd([x[:n] for x in p.raw], [x[:n] for x in p.logits], p.weight, p.bias, lens, dtype='bf16')
    for m, x, y in zip(NAMES, out, want):
        ref.check(m, back(x)[0, :n], y)
    check_bwd(p, 'bwd with a tail')


def test_no_tokens():
    """Only histories move; the taps' gradients are zeros."""
    p = Batch(8, [0, 0], H=2, dk=32, dv=32, slots=4)
    raw, weight, bias, hist, cu = p.gpu()
    gdn2.prologue_fwd(*raw, weight, bias, cu, conv_state=hist, conv_state_out=hist, slot_in=ints([1, -1]),
                      slot_out=ints([3, 0]))
    for got, old in zip(hist, p.hist):
        got = back(got)
        assert np.array_equal(got[3], old[1]) and np.all(got[0] == 0) and np.array_equal(got[[1, 2]], old[[1, 2]])
    g = gdn2.prologue_bwd(*raw, weight, bias, *(x.float() for x in raw), cu)
    assert all(torch.all(g[f'{w}_{n}'] == 0) for w in ('weight', 'bias') for n in 'qkv')


def test_zero_rows_have_zero_norm():
    """y = 0 (zero inputs, no bias): q = 0, and the gradient is dq / 1e-12 as the formula has it."""
    p = Batch(9, [9], H=1, dk=16, dv=16, dtype='f32', bias=False)
    for x in p.raw:
        x[:] = 0
    p.grads = [x * np.float32(1e-12) for x in p.grads]
    check_fwd(p, 'zeros')
    check_bwd(p, 'zeros bwd')


def test_extreme_logits():
    p = Batch(10, [40], H=1, dk=16, dv=16, dtype='f32')
    for x in p.logits:
        x.reshape(-1)[:6] = [-1e4, 1e4, -100, 100, -np.inf, np.inf]
    raw, weight, bias, _, cu = p.gpu()
    out = gdn2.prologue_fwd(*raw, weight, bias, cu)
    for x in out[3:]:
        got = back(x).reshape(-1)[:6]
        assert np.array_equal(got[[0, 1, 3, 4, 5]], [0, 1, 1, 0, 1]) and 0 <= got[2] < 1e-38
    g = gdn2.prologue_bwd(*raw, weight, bias, *(torch.from_numpy(x).to(DEV).unsqueeze(0) for x in p.grads), cu)
    for n in ('b_logit', 'w_logit'):
        assert torch.all(g[n].reshape(-1)[:6].abs() <= 1e-37)


def test_matches_the_fused_prologue():
    """prologue_fwd then chunk_fwd on its fp32 outputs, against chunk_fwd_prologue."""
    p = Batch(11, [70, 9], H=2, dk=64, dv=64, dtype='f32')
    raw, weight, bias, _, cu = p.gpu()
    la = -torch.rand((1, 79, 2, 64), device=DEV) * 0.2
    q, k, v, b, w = gdn2.prologue_fwd(*raw, weight, bias, cu)
    o, S = gdn2.chunk_fwd(q, k, v, la, b, w, None, cu)
    o2, S2, _ = gdn2.chunk_fwd_prologue(raw[0], raw[1], raw[2], la, raw[3], raw[4], weight, bias, None, cu)
    assert torch.allclose(o, o2, rtol=0, atol=2e-4) and torch.allclose(S, S2, rtol=0, atol=2e-4)


def test_gradient_dtype_and_determinism():
    p = Batch(12, [500, 30], H=4, dk=64, dv=64)
    raw, weight, bias, _, cu = p.gpu()
    grads = [torch.from_numpy(x).to(DEV).unsqueeze(0) for x in p.grads]
    a = gdn2.prologue_bwd(*raw, weight, bias, *grads, cu, grad_dtype=torch.float32)
    b = gdn2.prologue_bwd(*raw, weight, bias, *grads, cu, grad_dtype=torch.float32)
    c = gdn2.prologue_bwd(*raw, weight, bias, *grads, cu)
    want = ref.prologue_bwd(p.raw, p.logits, p.weight, p.bias, p.grads, p.lens)
    for n in want:
        assert torch.equal(a[n], b[n])
        ref.check(n, back(a[n]).reshape(want[n][0].shape), want[n])
        assert torch.equal(a[n].to(c[n].dtype), c[n])


def test_some_biases():
    p = Batch(13, [20], H=2, dk=32, dv=32)
    p.bias[1] = None
    raw, weight, bias, _, cu = p.gpu()
    out = gdn2.prologue_fwd(*raw, weight, bias, cu)
    want, _ = ref.prologue_fwd(p.raw, p.logits, p.weight, p.bias, p.lens, dtype='bf16')
    for m, x, y in zip(NAMES, out, want):
        ref.check(m, back(x)[0], y)
    g = gdn2.prologue_bwd(*raw, weight, bias, *(x.float() for x in raw), cu)
    assert 'bias_q' in g and 'bias_k' not in g and 'bias_v' in g


@pytest.mark.parametrize('T', [1, 40])
def test_captured_and_replayed(T):
    p = Batch(14, [T] * 3, H=2, dk=64, dv=64, slots=5)
    raw, weight, bias, hist, cu = p.gpu()
    slot = ints([4, 0, 2])
    out = [torch.empty_like(x) for x in raw]
    grads = [torch.from_numpy(x).to(DEV).unsqueeze(0) for x in p.grads]
    ws = torch.empty(1 << 20, dtype=torch.uint8, device=DEV)

    def step(h):
        gdn2.prologue_fwd(*raw, weight, bias, cu, conv_state=h, conv_state_out=h, slot_in=slot, out=out)
        return gdn2.prologue_bwd(*raw, weight, bias, *grads, cu, conv_state=h, slot_in=slot, workspace=ws)

    step(tuple(h.clone() for h in hist))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g = step(hist)
    for i in range(4):
        new = Batch(60 + i, [T] * 3, H=2, dk=64, dv=64, slots=5).gpu()[0]
        for x, y in zip(raw, new):
            x.copy_(y)
        eh = tuple(h.clone() for h in hist)
        eg = {n: x.clone() for n, x in step(eh).items()}
        eo = [x.clone() for x in out]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(out, eo)) and all(torch.equal(x, y) for x, y in zip(hist, eh))
        assert all(torch.equal(g[n], eg[n]) for n in eg)


@pytest.mark.parametrize('lens', [SHORT, LONG])
def test_history_out_without_one_in(lens):
    """No history in is zeros in, for sequences with and without tokens."""
    N = len(lens)
    p = Batch(15, lens, H=4, HK=2, dk=32, dv=64, slots=N + 2)
    raw, weight, bias, hist, cu = p.gpu()
    commit, slot = ints([i % 4 for i in range(N)]), ints(list(range(N))[::-1])
    zeros, a, b = (tuple(f(h) for h in hist) for f in (torch.zeros_like, torch.clone, torch.clone))
    x = gdn2.prologue_fwd(*raw, weight, bias, cu, conv_state=zeros, conv_state_out=a, slot_in=slot, commit=commit)
    y = gdn2.prologue_fwd(*raw, weight, bias, cu, conv_state_out=b, slot_in=slot, commit=commit)
    assert all(torch.equal(s, t) for s, t in zip(x, y)) and all(torch.equal(s, t) for s, t in zip(a, b))


@pytest.mark.parametrize('value', [float('nan'), float('inf')])
def test_not_finite_stays_in_its_sequence(value):
    """Three sequences in a few tiles, the middle one, its history and the rows behind the last one not finite:
    the others' outputs, histories and gradients keep their bits."""
    lens = [5, 6, 7]
    p = Batch(16, lens, H=2, dk=64, dv=32, slots=4, tail=9)
    raw, weight, bias, hist, cu = p.gpu()
    grads = [torch.from_numpy(x).to(DEV).unsqueeze(0) for x in p.grads]
    names = ('q_raw', 'k_raw', 'v_raw', 'b_logit', 'w_logit')

    def run():
        h = tuple(x.clone() for x in hist)
        o = gdn2.prologue_fwd(*raw, weight, bias, cu, conv_state=h, conv_state_out=h, slot_in=slot)
        g = gdn2.prologue_bwd(*raw, weight, bias, *grads, cu, conv_state=hist, slot_in=slot)
        return [x.clone() for x in o] + [g[n] for n in names], h

    slot = ints([2, 0, 1])
    rows, pools = run()
    for x in (*raw, *grads):
        x[0, 5:11] = value
        x[0, 18:] = value
    for h in hist:
        h[0] = value
        h[3] = value
    rows2, pools2 = run()
    for x, y in zip(rows, rows2):
        assert torch.equal(x[0, :5], y[0, :5]) and torch.equal(x[0, 11:18], y[0, 11:18])
    for x, y in zip(pools, pools2):
        assert torch.equal(x[1], y[1]) and torch.equal(x[2], y[2])
    assert not torch.isfinite(rows2[0][0, 5:11]).all()


def test_past_32_bit_offsets():
    """Tokens behind 2^31 elements: the same bits as in a small call."""
    n, heads, d = 70, 16, 128
    T = (1 << 31) // (heads * d) + n + 9
    p = Batch(17, [n], H=heads, dk=d, dv=d, gates='head')
    raw, weight, bias, _, cu = p.gpu()
    grads = [torch.from_numpy(x).to(DEV).unsqueeze(0) for x in p.grads]
    small = gdn2.prologue_fwd(*raw, weight, bias, cu)
    small_g = gdn2.prologue_bwd(*raw, weight, bias, *grads, cu)

    def large(x):
        y = torch.zeros((1, T, *x.shape[2:]), dtype=x.dtype, device=DEV)
        y[:, -n:] = x
        return y

    cu2 = ints([0, T - n, T])
    big = [large(x) for x in raw]
    out = gdn2.prologue_fwd(*big, weight, bias, cu2)
    assert all(torch.equal(x[:, -n:], y) for x, y in zip(out, small))
    del out
    g = gdn2.prologue_bwd(*big, weight, bias, *(large(x) for x in grads), cu2)
    for m in ('q_raw', 'k_raw', 'v_raw', 'b_logit', 'w_logit'):
        assert torch.equal(g[m][:, -n:], small_g[m]), m


@pytest.mark.parametrize('value', [float('nan'), float('inf')])
@pytest.mark.parametrize('dtype', ['bf16', 'f32'])
@pytest.mark.parametrize('lens', [[7, 9], [30, 41]])
@pytest.mark.parametrize('d', [16, 128])
def test_one_channel_not_finite(d, lens, dtype, value):
    """One channel of one token: NaN wherever the formulas have it (the head's other channels, whose norm it is
    part of, and their gradients), the formulas' values everywhere else."""
    p = Batch(18, lens, H=2, dk=d, dv=d, dtype=dtype)
    n, at = sum(lens), lens[0] + 3
    for x in p.raw:
        x[at, 1, 5] = value
    print(f'[one channel] d={d} lens={lens} {dtype} {value}', flush=True)
    raw, weight, bias, _, cu = p.gpu()
    out = gdn2.prologue_fwd(*raw, weight, bias, cu)
    grads = [torch.from_numpy(x).to(DEV).unsqueeze(0) for x in p.grads]
    g = gdn2.prologue_bwd(*raw, weight, bias, *grads, cu)
    with np.errstate(all='ignore'):
        want, _ = ref.prologue_fwd(p.raw, p.logits, p.weight, p.bias, lens, dtype=dtype)
        wantg = ref.prologue_bwd(p.raw, p.logits, p.weight, p.bias, p.grads, lens, dtype=dtype)
    pairs = [(m, back(x)[0, :n], y) for m, x, y in zip(NAMES, out, want)]
    pairs += [(m, back(g[m])[0, :n] if m.endswith(('raw', 'logit')) else back(g[m]), wantg[m]) for m in wantg]
    for m, x, (y, tol) in pairs:
        x = x.reshape(y.shape)
        assert np.array_equal(np.isnan(x), np.isnan(y)), f'{m}: NaN in {np.isnan(x).sum()} places, not {np.isnan(y).sum()}'
        fin = np.isfinite(y)
        assert np.array_equal(x[~fin & ~np.isnan(y)], y[~fin & ~np.isnan(y)]), m
        # (no tolerance, NaN, at the zeros that dividing by an infinite norm leaves: those are exact)
        ref.check(m, x[fin], (y[fin], np.nan_to_num(tol[fin])))
    assert value == value or (np.isnan(want[0][0][at, 1]).all() and np.isnan(wantg['bias_q'][0].reshape(2, d)[1]).all())


@pytest.mark.parametrize('grad', ['f32', 'bf16'])
@pytest.mark.parametrize('gates', ['channel', 'head'])
def test_gradient_of_large_logits(gates, grad):
    """The sigmoid's gradient s (1 - s), where s is next to one or to zero, to the precision of its type.

    Tolerance: with e = exp(-|x|), off by 2^-22 + |x| 2^-24 of itself (8 + 2 |x| units of 2^-24 with the rounding of
    its argument), the gradient is d e / (1 + e)^2: 1 + e one rounding, its reciprocal 2^-23 and squared, two
    products; 16 units in all. Below the smallest normal float anything may be zero."""
    p = Batch(19, [64], H=4, dk=16, dv=16, dtype='f32', gates=gates)
    for x in p.logits:
        x[:] = np.linspace(-90, 90, x.size, dtype=np.float32).reshape(x.shape)
    raw, weight, bias, _, cu = p.gpu()
    grads = [torch.from_numpy(x).to(DEV).unsqueeze(0) for x in p.grads]
    g = gdn2.prologue_bwd(*raw, weight, bias, *grads, cu, grad_dtype=DT[grad])
    for m, x, d in zip(('b_logit', 'w_logit'), p.logits, p.grads[3:]):
        x, d = x.astype(np.float64), d.astype(np.float64)
        e = np.exp(-np.abs(x))
        want = d * e / (1 + e) ** 2
        ref.check(m, back(g[m])[0], (want, ref.rounded(want, np.abs(want) * (16 + 2 * np.abs(x)) * ref.U, grad)))


def test_gates_over_their_logits():
    """b and w written over their own logits, the histories over their own pools."""
    p = Batch(21, SHORT, H=2, dk=32, dv=64, slots=9)
    raw, weight, bias, hist, cu = p.gpu()
    want = gdn2.prologue_fwd(*raw, weight, bias, cu, conv_state=hist)
    q, k, v = (torch.empty_like(x) for x in raw[:3])
    got = gdn2.prologue_fwd(*raw, weight, bias, cu, conv_state=hist, conv_state_out=hist, out=(q, k, v, raw[3], raw[4]))
    assert got[3] is raw[3] and all(torch.equal(x, y) for x, y in zip(got, want))
