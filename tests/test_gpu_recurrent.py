"""gdn2_recurrent_fwd (the recurrence token by token on a pool of states) against
the float64 oracle: every head size, gate layout, type and head ratio; lengths
around its 8-token blocks; slots, commits and empty sequences; and its calls on
other streams and inside a captured graph."""
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


class Batch:
    """Seeded inputs; numpy arrays hold exactly what the GPU receives."""

    def __init__(self, seed, lens, H=2, HK=None, dk=32, dv=32, dtype='bf16', gates='channel', slots=None, decay=None,
                 tail=0):
        rng = np.random.default_rng(seed)
        HK = HK or H
        T = sum(lens) + tail
        rnd = gi.bf16_round if dtype == 'bf16' else (lambda x: np.asarray(x, np.float32))
        n = lambda *s: rng.standard_normal(s).astype(np.float32)   # noqa: E731
        unit = lambda x: x / np.maximum(np.linalg.norm(x, axis=-1, keepdims=True), 1e-6)   # noqa: E731
        sig = lambda x: 1 / (1 + np.exp(-x))   # noqa: E731
        self.lens, self.H, self.HK, self.dk, self.dv, self.dtype = lens, H, HK, dk, dv, dtype
        self.q, self.k, self.v = rnd(unit(n(T, HK, dk))), rnd(unit(n(T, HK, dk))), rnd(n(T, H, dv))
        self.b = rnd(sig(n(T, H, dk) if gates == 'channel' else n(T, H)))
        self.w = rnd(sig(n(T, H, dv) if gates == 'channel' else n(T, H)))
        x = n(T, H) if gates == 'head' else n(T, H, dk)
        self.la = (-np.logaddexp(0, x - 3) if decay is None else np.full_like(x, decay)).astype(np.float32)
        self.slots = slots or len(lens)
        self.state = n(self.slots, H, dk, dv)
        self.cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)

    def gpu(self):
        to = lambda x, dt: torch.from_numpy(x).to(DEV).to(dt).unsqueeze(0)   # noqa: E731
        dt = DT[self.dtype]
        args = [to(x, dt) for x in (self.q, self.k, self.v)] + [to(self.la, torch.float32)] + [
            to(x, dt) for x in (self.b, self.w)]
        return args, torch.from_numpy(self.state).to(DEV), torch.from_numpy(self.cu).to(DEV)

    def reference(self, out='f32', **kw):
        n = sum(self.lens)
        wide = lambda x, d: x[:n] if x.ndim == 3 else np.repeat(x[:n, :, None], d, 2)   # noqa: E731
        return ref.recurrent(self.q[:n], self.k[:n], self.v[:n], wide(self.la, self.dk), wide(self.b, self.dk),
                             wide(self.w, self.dv), self.state, self.lens, out_dtype=out, **kw)


def ints(x):
    return None if x is None else torch.tensor(x, dtype=torch.int32, device=DEV)


def run(p, out='f32', **kw):
    args, state, cu = p.gpu()
    o = gdn2.recurrent_fwd(*args, state, cu, out_dtype=DT[out], **{k: ints(v) for k, v in kw.items()})
    torch.cuda.synchronize()
    return o[0].float().cpu().numpy(), state.cpu().numpy()


def check(p, label, out='f32', **kw):
    print(f'[{label}] lens={p.lens} H={p.H}/{p.HK} dk={p.dk} dv={p.dv} {p.dtype}->{out}', flush=True)
    o, state = run(p, out, **kw)
    (o_ref, s_ref) = p.reference(out, **kw)
    a = ref.check(f'{label} o', o[:sum(p.lens)], o_ref)
    written = s_ref[1].reshape(p.slots, -1).max(1) > 0
    b = ref.check(f'{label} state', state[written], (s_ref[0][written], s_ref[1][written])) if written.any() else 0
    # states no token touched are copies: bit for bit
    assert np.array_equal(state[~written].astype(np.float64), s_ref[0][~written]), f'{label}: an untouched state changed'
    print(f'{label}: o {a:.3f}, state {b:.3f} of the tolerance', flush=True)


LENS = [1, 0, 2, 7, 8, 9, 17]


@pytest.mark.parametrize('dtype', ['bf16', 'f32'])
@pytest.mark.parametrize('dk', [16, 32, 64, 128])
@pytest.mark.parametrize('dv', [16, 32, 64, 128])
def test_head_sizes(dk, dv, dtype):
    check(Batch(10 + dk + dv, LENS, H=3, dk=dk, dv=dv, dtype=dtype), f'sizes {dk}x{dv}')


@pytest.mark.parametrize('gates', ['channel', 'head', 'kda'])
@pytest.mark.parametrize('H,HK', [(4, 4), (4, 2), (6, 1)])
@pytest.mark.parametrize('dtype,out', [('bf16', 'f32'), ('bf16', 'bf16'), ('f32', 'bf16')])
def test_gates_heads_types(gates, H, HK, dtype, out):
    check(Batch(7, LENS, H=H, HK=HK, dk=64, dv=64, dtype=dtype, gates=gates), f'{gates} {H}/{HK}', out)


@pytest.mark.parametrize('N,H,T', [(1, 1, 1), (5, 2, 1), (3, 16, 1), (40, 16, 1), (2, 3, 64), (1, 2, 133)])
def test_uniform_batches(N, H, T):
    """No cu_seqlens: [N, T, H, d] tensors (few chains and many, which differ in their launch)."""
    p = Batch(100 + N + T, [T] * N, H=H, dk=128, dv=128)
    args, state, _ = p.gpu()
    args = [x.reshape(N, T, *x.shape[2:]) for x in args]
    print(f'[uniform] N={N} H={H} T={T}', flush=True)
    o = gdn2.recurrent_fwd(*args, state)
    (o_ref, s_ref) = p.reference()
    ref.check('uniform o', o.reshape(N * T, H, 128).cpu().numpy(), o_ref)
    ref.check('uniform state', state.cpu().numpy(), s_ref)


@pytest.mark.parametrize('decay', [0.0, -5.0, -30.0, -200.0, float('-inf')])
@pytest.mark.parametrize('gates', ['channel', 'head'])
def test_decay_strengths(decay, gates):
    p = Batch(3, [5, 19], H=2, dk=64, dv=32, dtype='f32', gates=gates, decay=decay)
    with np.errstate(divide='ignore', invalid='ignore'):
        check(p, f'decay {decay}')


def test_mixed_decay_in_a_block():
    """Full forgets, none and mild decay alternate over tokens and channels."""
    p = Batch(4, [24], H=2, dk=32, dv=32, dtype='f32')
    p.la[::3] = -np.inf
    p.la[1::3, :, ::2] = 0
    p.la[2::3, :, 1::2] = -40
    check(p, 'mixed decay')


@pytest.mark.parametrize('commit', [[0, 0, 0, 0], [1, 3, 8, 9], [4, 5, 99, 16], [-3, 2, 12, 17]])
def test_commit(commit):
    check(Batch(5, [4, 5, 12, 17], H=2, dk=64, dv=128), f'commit {commit}', commit=commit)


def test_commit_equals_a_shorter_run():
    """The kept state of a draft is bit for bit that of a call on its accepted tokens alone."""
    lens, commit = [8, 5, 20, 3], [3, 5, 11, 0]
    p = Batch(6, lens, H=2, dk=128, dv=64)
    _, kept = run(p, commit=commit)
    short = Batch(6, lens, H=2, dk=128, dv=64)
    at = np.concatenate([np.arange(c, c + n) for c, n in zip(np.cumsum([0] + lens[:-1]), commit)])
    for n in ('q', 'k', 'v', 'b', 'w', 'la'):
        setattr(short, n, getattr(short, n)[at])
    short.lens, short.cu = commit, np.concatenate([[0], np.cumsum(commit)]).astype(np.int32)
    _, want = run(short)
    assert np.array_equal(kept, want)


def test_slots():
    """Scattered slots, in != out, none in, none out, a forked slot, an empty sequence's copy."""
    lens = [3, 9, 0, 0, 4, 2, 6, 5]
    slot_in = [7, 2, 4, 4, -1, 2, 99, 8]
    slot_out = [7, 0, 1, 4, 3, 9, 10, -5]
    check(Batch(8, lens, H=3, dk=32, dv=64, slots=12), 'slots', slot_in=slot_in, slot_out=slot_out,
          commit=[3, 4, 0, 0, 4, 0, 6, 2])


def test_slot_out_defaults_to_slot_in():
    check(Batch(9, [2, 3], H=1, dk=16, dv=16, slots=5), 'slot_in alone', slot_in=[4, 0])


def test_slot_out_alone():
    check(Batch(9, [2, 3], H=1, dk=16, dv=16, slots=5), 'slot_out alone', slot_out=[4, 2])


def test_rows_behind_the_last_sequence():
    p = Batch(11, [3, 10], H=2, dk=64, dv=64, tail=6)
    args, state, cu = p.gpu()
    out = torch.full((1, 19, 2, 64), 7.25, device=DEV)
    gdn2.recurrent_fwd(*args, state, cu, out=out)
    (o_ref, s_ref) = p.reference()
    ref.check('o', out[0, :13].cpu().numpy(), o_ref)
    assert torch.all(out[0, 13:] == 7.25)
    ref.check('state', state.cpu().numpy(), s_ref)


def test_no_tokens_at_all():
    p = Batch(12, [0, 0], H=2, dk=32, dv=32, slots=4)
    args, state, cu = p.gpu()
    gdn2.recurrent_fwd(*args, state, cu, slot_in=ints([0, -1]), slot_out=ints([3, 1]))
    got = state.cpu().numpy()
    assert np.array_equal(got[3], p.state[0]) and np.all(got[1] == 0)
    assert np.array_equal(got[[0, 2]], p.state[[0, 2]])


@pytest.mark.parametrize('name', ['q', 'k', 'v', 'b', 'w', 'la'])
@pytest.mark.parametrize('value', [float('nan'), float('inf')])
def test_not_finite_reaches_no_earlier_token(name, value):
    """A NaN or an infinity in one token leaves the tokens before it in its block, the other
    sequences and a prefix kept without it as they are."""
    lens, at = [6, 8, 11], 6 + 5
    clean = Batch(13, lens, H=2, dk=32, dv=32, dtype='f32')
    o0, s0 = run(clean, commit=[6, 4, 11])
    dirty = Batch(13, lens, H=2, dk=32, dv=32, dtype='f32')
    getattr(dirty, name)[at, 1] = value
    o1, s1 = run(dirty, commit=[6, 4, 11])
    keep = np.ones(25, bool)
    keep[at:14] = False
    (o_ref, s_ref) = clean.reference(commit=[6, 4, 11])
    for o in (o0, o1):
        ref.check('o', o[keep], (o_ref[0][keep], o_ref[1][keep]))
    assert np.array_equal(s0, s1)
    assert np.array_equal(o0[:, 0], o1[:, 0]) or name in 'qk'   # the other head, where it has its own input
    assert not np.all(np.isfinite(o1[at, 1]))


def test_large_keys_under_strong_decay():
    """A key that overflows when it is divided by its block's decay, and does not by itself."""
    p = Batch(16, [8, 3, 8], H=2, dk=32, dv=32, dtype='f32', decay=-5.0)   # down to 2^-58 over a block
    p.k[6, 0, :4] *= np.float32(1e25)   # over a decay of e^-35: past the largest float
    p.state[0] *= np.float32(1e-20)   # (what the key meets stays small)
    p.v *= np.float32(1e-10)
    check(p, 'large key')


@pytest.mark.parametrize('dtype', ['bf16', 'f32'])
@pytest.mark.parametrize('at', [1, 4, 5, 7])
@pytest.mark.parametrize('d', [32, 128])
def test_overflow_reaches_no_earlier_token(d, at, dtype):
    """A finite token whose product with the state overflows: the tokens before it in its block and the prefix
    kept without it keep their bits."""
    lens = [3, 8, 8]
    kept = min(at, 4)

    def one(k):
        p = Batch(14, lens, H=2, dk=d, dv=d, dtype=dtype)
        p.state[1:] *= np.float32(1e20)
        p.k[3 + at, 1] *= k
        return run(p, commit=[3, kept, 8])

    o0, s0 = one(np.float32(1))
    o1, s1 = one(np.float32(2.0 ** 70))
    assert np.all(np.isfinite(o0)) and not np.all(np.isfinite(o1[3 + at, 1]))
    assert np.array_equal(o0[:3 + at], o1[:3 + at]) and np.array_equal(o0[11:], o1[11:])
    assert np.array_equal(o0[:, 0], o1[:, 0]) and np.array_equal(s0, s1) and np.all(np.isfinite(s1))


def test_matches_decode_step():
    """Tokens one by one through gdn2_decode_step give the same outputs and states."""
    p = Batch(14, [5] * 3, H=4, dk=128, dv=128)
    args, state, _ = p.gpu()
    args = [x.reshape(3, 5, *x.shape[2:]) for x in args]
    S = state.clone()
    o = gdn2.recurrent_fwd(*args, state)
    q, k, v, la, b, w = args
    for t in range(5):
        step = [x[:, t].contiguous() for x in (q, k, v, la, b, w)]
        ot = gdn2.decode_step(*step, S)
        assert torch.allclose(o[:, t], ot, rtol=0, atol=2e-5 * float(ot.abs().max()))
    assert torch.allclose(state, S, rtol=0, atol=2e-5 * float(S.abs().max()))


def test_deterministic():
    p = Batch(15, [3, 40, 9], H=4, dk=128, dv=128)
    first = run(p)
    second = run(p)
    assert np.array_equal(first[0], second[0]) and np.array_equal(first[1], second[1])


def test_other_stream():
    p = Batch(16, [3, 12], H=2, dk=64, dv=64)
    args, state, cu = p.gpu()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        state.mul_(2)
        o = gdn2.recurrent_fwd(*args, state, cu)
        o2 = o + 0
    side.synchronize()
    p.state = p.state * 2
    (o_ref, s_ref) = p.reference()
    ref.check('o', o2[0].cpu().numpy(), o_ref)
    ref.check('state', state.cpu().numpy(), s_ref)


def test_captured_and_replayed():
    """A captured serving step replays on new inputs and slots in the same buffers."""
    p = Batch(17, [1] * 6, H=4, dk=128, dv=128, slots=9)
    args, state, cu = p.gpu()
    slot = ints([8, 1, 0, 5, 2, 7])
    out = torch.empty((1, 6, 4, 128), device=DEV)
    gdn2.recurrent_fwd(*args, state, cu, slot_in=slot, slot_out=slot, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdn2.recurrent_fwd(*args, state, cu, slot_in=slot, slot_out=slot, out=out)
    for step in range(4):
        n = Batch(200 + step, [1] * 6, H=4, dk=128, dv=128, slots=9)
        new, _, _ = n.gpu()
        for x, y in zip(args, new):
            x.copy_(y)
        perm = np.random.default_rng(step).permutation(9)[:6]
        slot.copy_(ints(perm.tolist()))
        eager_state = state.clone()
        eager = gdn2.recurrent_fwd(*new, eager_state, cu, slot_in=slot, slot_out=slot)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager) and torch.equal(state, eager_state)


def test_pool_past_32_bit_offsets():
    """A slot whose elements lie more than 2^32 bytes, and 2^30 elements, into the pool."""
    H, d = 16, 128
    slots = (5 << 30) // (H * d * d * 4)
    state = torch.empty((slots, H, d, d), device=DEV)
    p = Batch(18, [3, 2], H=H, dk=d, dv=d)
    args, small, cu = p.gpu()
    at = [slots - 1, slots - 2]
    state[at] = small
    o = gdn2.recurrent_fwd(*args, state, cu, slot_in=ints(at))
    (o_ref, s_ref) = p.reference()
    ref.check('o', o[0].cpu().numpy(), o_ref)
    ref.check('state', state[at].cpu().numpy(), s_ref)


@pytest.mark.parametrize('decay', [None, -12.0])
@pytest.mark.parametrize('gates', ['channel', 'head'])
def test_many_chains(gates, decay):
    """More chains than half the compute units: a workgroup owns a whole chain. Ragged lengths,
    scattered slots, commits; a decay that cuts blocks (e^-96 over eight tokens)."""
    rng = np.random.default_rng(19)
    N = 20
    lens = rng.integers(0, 40, N).tolist()
    slot = rng.permutation(N + 5)[:N].tolist()
    commit = [int(rng.integers(0, n + 2)) for n in lens]
    p = Batch(19, lens, H=8, HK=4, dk=128, dv=128, gates=gates, slots=N + 5, decay=decay)
    check(p, f'many chains {gates} {decay}', slot_in=slot, commit=commit)


def test_long_sequence():
    check(Batch(20, [1000], H=1, dk=64, dv=64, dtype='f32'), 'long')


def test_two_streams_share_a_pool():
    """Two calls at once on two streams, on slots of one pool that do not meet."""
    a, b = Batch(21, [9] * 8, H=4, dk=64, dv=64, slots=16), Batch(22, [9] * 8, H=4, dk=64, dv=64, slots=16)
    b.state = a.state
    (args_a, state, cu), (args_b, _, _) = a.gpu(), b.gpu()
    sa, sb = ints(list(range(0, 16, 2))), ints(list(range(1, 16, 2)))
    torch.cuda.synchronize()
    outs = {}
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s, args, slot, name in ((streams[0], args_a, sa, 'a'), (streams[1], args_b, sb, 'b')):
        with torch.cuda.stream(s):
            outs[name] = gdn2.recurrent_fwd(*args, state, cu, slot_in=slot)
    torch.cuda.synchronize()
    for p, slot, name in ((a, sa, 'a'), (b, sb, 'b')):
        at = slot.cpu().numpy()
        (o_ref, s_ref) = p.reference(slot_in=at)
        ref.check(f'o {name}', outs[name][0].cpu().numpy(), o_ref)
        ref.check(f'state {name}', state.cpu().numpy()[at], (s_ref[0][at], s_ref[1][at]))


def _cut(pairs, d, dtype, moved, decay=None, gates='channel'):
    """A draft of n tokens with c kept for each (n, c) of ``pairs``, in scattered slots; moved: into other ones."""
    N = len(pairs)
    perm = np.random.default_rng(N).permutation(2 * N + 1)
    p = Batch(23, [n for n, _ in pairs], H=2, dk=d, dv=d, dtype=dtype, gates=gates, slots=2 * N + 1, decay=decay)
    kw = dict(slot_in=perm[:N].tolist(), commit=[c for _, c in pairs])
    if moved:
        kw['slot_out'] = perm[N:2 * N].tolist()
    return p, kw


@pytest.mark.parametrize('moved', [False, True])
@pytest.mark.parametrize('decay', [-5.5, -6.0, -12.0, -30.0, float('-inf')])
@pytest.mark.parametrize('d,dtype,gates,top', [(32, 'f32', 'channel', 17), (64, 'bf16', 'head', 17), (128, 'bf16', 'channel', 9)])
def test_commit_in_a_block_cut_for_its_decay(d, dtype, gates, top, decay, moved):
    """Every commit of every length around one and two blocks, with decays that cut them."""
    p, kw = _cut([(n, c) for n in range(2, top + 1) for c in range(n + 1)], d, dtype, moved, decay, gates)
    with np.errstate(divide='ignore', invalid='ignore'):
        check(p, f'commit under {decay}', **kw)


@pytest.mark.parametrize('decay', [-6.0, -12.0])
def test_commit_in_a_cut_block_of_few_chains(decay):
    """The same where two workgroups share a chain."""
    p, kw = _cut([(8, c) for c in range(9)], 128, 'bf16', False, decay)
    check(p, f'few chains {decay}', **kw)


@pytest.mark.parametrize('moved', [False, True])
@pytest.mark.parametrize('channels', [slice(3, 4), slice(None)])
@pytest.mark.parametrize('n', [2, 3, 4, 5, 6, 7, 8, 9, 12, 16, 17])
def test_commit_around_a_full_forget(n, channels, moved):
    """One token that forgets a channel, or all, at each place before and behind each commit."""
    at = [t for t in range(n) for _ in range(n + 1)]
    p, kw = _cut([(n, i % (n + 1)) for i in range(n * (n + 1))], 32, 'f32', moved)
    for i, t in enumerate(at):
        p.la[i * n + t, :, channels] = -np.inf
    with np.errstate(divide='ignore', invalid='ignore'):
        check(p, f'forget in {n}', **kw)


def test_commit_where_only_the_last_block_is_cut():
    """Mild decay up to the sequence's last block, which decays by more than 2^60."""
    pairs = [(n, c) for n in range(9, 25) for c in range(n + 1)]
    p, kw = _cut(pairs, 32, 'f32', True)
    for end, n in zip(p.cu[1:], p.lens):
        p.la[end - ((n - 1) % 8 + 1):end] = -9
    check(p, 'last block', **kw)
