"""Every form of the products that gdn2_linear_fwd / gdn2_linear_bwd choose from, with whole numbers whose every
partial sum, in whatever order, fp32 holds: the results have to be the exact ones, rounded once where they are bf16."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip('torch')
if not torch.cuda.is_available():
    pytest.skip('no GPU', allow_module_level=True)

import gated_delta_rule_wy_amd as gdn2  # noqa: E402
from gpu_util import DEV  # noqa: E402

DT = {'bf16': torch.bfloat16, 'f32': torch.float32, 'e4m3': torch.float8_e4m3fn}


def whole(seed, most, *shape):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randint(-most, most + 1, shape, generator=g, device=DEV).float()


def same(name, got, want):
    want = want.to(got.dtype)
    if not torch.equal(got, want):
        bad = (got != want).nonzero()
        at = tuple(bad[0].tolist())
        raise AssertionError(f'{name}: {len(bad)} of {got.numel()} differ, the first at {at}: {float(got[at])} for {float(want[at])}')


# Few rows: blocks of the waves that share the contraction, from 16 x 16 to 32 x 64, with one to many steps a wave
# (fewer than it keeps under way, as many, one and more rounds of them), and a part of a step at the rows' end
BLOCKS = [(1, 500), (20, 48), (16, 8192), (31, 4100), (60, 4096), (100, 2040), (64, 8192), (250, 2048)]


@pytest.mark.parametrize('dtype', ['bf16', 'f32', 'e4m3'])
@pytest.mark.parametrize('K', [40, 1024, 2560, 5232, 8192])
@pytest.mark.parametrize('M,N', BLOCKS)
def test_blocks(M, N, K, dtype):
    forward(M, N, K, dtype)


# the same with rows that are no whole chunks
@pytest.mark.parametrize('dtype', ['bf16', 'f32', 'e4m3'])
@pytest.mark.parametrize('K', [33, 2049, 5001])
@pytest.mark.parametrize('M,N', BLOCKS)
def test_blocks_of_odd_rows(M, N, K, dtype):
    forward(M, N, K, dtype)


# tiles of 128 x 64, 128 x 128, 256 x 256, with parts of tiles at both ends; N or K in no whole vectors
@pytest.mark.parametrize('dtype', ['bf16', 'f32', 'e4m3'])
@pytest.mark.parametrize('K', [40, 528, 2560, 2049])
@pytest.mark.parametrize('M,N', [(600, 2056), (2100, 1992), (3190, 2680), (3500, 3608), (700, 2001)])
def test_tiles(M, N, K, dtype):
    forward(M, N, K, dtype)


def forward(M, N, K, dtype):
    print(f'[forward] {M}x{N}x{K} {dtype}', flush=True)
    x, w, b = whole(M, 3, M, K), whole(N, 3, N, K), whole(K, 50, N)
    want = (x.double() @ w.double().t() + b).float()
    scale = dict(x_scale=torch.full((M,), 2.0, device=DEV), weight_scale=torch.full((N,), 0.5, device=DEV)) if dtype == 'e4m3' else {}
    x, w = x.to(DT[dtype]), w.to(DT[dtype])
    for out in ('f32', 'bf16'):
        r = whole(M + N, 50, M, N).to(DT[out])
        y, _ = gdn2.linear_fwd(x, w, b, r, out_dtype=DT[out], **scale)
        same(f'y in {out}', y, want + r)
        y, z = gdn2.linear_fwd(x, w, b, out_dtype=DT[out], output_preact=dtype != 'e4m3', **scale)
        same(f'y in {out}', y, want)
        if z is not None:
            same('z', z, want)


# dweight by columns of dy and x, 128 x 128 and 256 x 256, whole and in parts (of bf16 rows of whole chunks); turned
# around first, in few tiles' parts up to the most there are; dx in parts; fp32 read down the columns
@pytest.mark.parametrize('dtype', ['bf16', 'f32'])
@pytest.mark.parametrize('M,N,K', [
    (4133, 2050, 2056), (130, 3600, 3400), (64, 4000, 3600), (9001, 2100, 2000), (700, 1500, 1496), (3001, 520, 256), (20000, 304, 296),
    (20000, 300, 301), (4100, 2050, 2041), (33, 8200, 256), (64, 16384, 128), (200, 30000, 512), (1000, 1001, 1003), (1554, 1001, 777),
    (1000, 5, 3000), (1, 2048, 2048)])
def test_gradient(M, N, K, dtype):
    gradient(M, N, K, dtype, 3, 2)


@pytest.mark.parametrize('N,K', [(2, 3), (16, 24)])
@pytest.mark.parametrize('dtype', ['bf16', 'f32'])
def test_gradient_of_the_most_rows(N, K, dtype):
    """Sums of 2^22 terms in 256 parts."""
    gradient(2 ** 22, N, K, dtype, 1, 1)


def gradient(M, N, K, dtype, top_dy, top_x):
    print(f'[gradient] {M}x{N}x{K} {dtype}', flush=True)
    dy, x, w = whole(M, top_dy, M, N), whole(K, top_x, M, K), whole(N, top_x, N, K)
    assert max(M, N) * top_dy * top_x <= 2 ** 24
    d = lambda t: t.double()   # noqa: E731
    want = {'x': (d(dy) @ d(w)).float(), 'weight': (d(dy).t().contiguous() @ d(x)).float(), 'bias': d(dy).sum(0).float()}
    dt = DT[dtype]
    for ddt in (dt, torch.float32 if dtype == 'bf16' else torch.bfloat16):
        got = gdn2.linear_bwd(dy.to(ddt), x.to(dt), w.to(dt))
        for n in want:
            same(f'd{n}', got[n], want[n])
    # each product alone takes its operands in its own way
    for n in ('x', 'weight'):
        got = gdn2.linear_bwd(dy.to(dt), x.to(dt), w.to(dt), output_x=n == 'x', output_weight=n == 'weight', output_bias=False)
        same(f'd{n} alone', got[n], want[n])


@pytest.mark.parametrize('dtype,act', [('bf16', 'none'), ('bf16', 'silu'), ('f32', 'none')])
@pytest.mark.parametrize('M,N,K', [(4133, 2050, 2056), (130, 3600, 3400), (700, 1500, 1496), (77, 64, 40), (64, 16384, 128), (3001, 520, 256)])
def test_gradient_with_nothing_beyond_the_tensors(M, N, K, dtype, act):
    """Operands and a workspace that are followed by NaN, outputs that are followed by numbers that stay."""
    print(f'[beyond] {M}x{N}x{K} {dtype} {act}', flush=True)
    dt = DT[dtype]
    dy, x, w = whole(1, 3, M, N), whole(2, 2, M, K), whole(3, 2, N, K)
    z = torch.full((M, N), 200.0, device=DEV) if act == 'silu' else None   # (where its slope is 1)
    want = {'x': (dy.double() @ w.double()).to(dt), 'weight': (dy.double().t().contiguous() @ x.double()).to(dt), 'bias': dy.double().sum(0).float()}

    def inside(t):
        flat = torch.full((t.numel() + 8192,), float('nan'), device=DEV, dtype=dt)
        flat[:t.numel()] = t.flatten()
        return flat

    code = gdn2.GDN2_BF16 if dtype == 'bf16' else gdn2.GDN2_F32
    a, lib = 2 if z is not None else 0, gdn2.lib()
    out = {n: torch.full((t.numel() + 8192,), 7.0, device=DEV, dtype=t.dtype) for n, t in want.items()}
    need = lib.gdn2_linear_bwd_workspace_bytes(M, K, N, a, code, code, 1, 1, 1)
    ws = torch.full((need + 8192,), 0xff, dtype=torch.uint8, device=DEV)   # (NaN as well)
    args = [inside(dy), inside(x), inside(w), inside(z) if z is not None else None]
    lib.gdn2_set_stream(torch.cuda.current_stream().cuda_stream)
    p = lambda t: None if t is None else t.data_ptr()   # noqa: E731
    assert lib.gdn2_linear_bwd(*map(p, args), p(out['x']), p(out['weight']), p(out['bias']), M, K, N, a, code, code, p(ws), need) == 0
    for n, t in want.items():
        same(f'd{n}', out[n][:t.numel()].view(t.shape), t)
        assert torch.all(out[n][t.numel():] == 7.0)
    assert torch.all(ws[need:] == 0xff)


# the most features that are taken, and one fewer
@pytest.mark.parametrize('dtype', ['bf16', 'f32', 'e4m3'])
@pytest.mark.parametrize('M,N,K', [(1, 48, 2 ** 20), (300, 40, 2 ** 20 - 1), (600, 520, 2 ** 20), (700, 257, 2 ** 20 - 1), (33, 2 ** 20, 40),
                                   (1, 2 ** 20 - 1, 33), (300, 2 ** 20, 16)])
def test_the_most_features(M, N, K, dtype):
    print(f'[features] {M}x{N}x{K} {dtype}', flush=True)
    x, w = whole(M, 3, M, K), whole(N, 3, N, K)
    want = torch.cat([x.double() @ w[n:n + 65536].double().t() for n in range(0, N, 65536)], 1).float()
    scale = dict(x_scale=torch.ones(M, device=DEV), weight_scale=torch.ones(N, device=DEV)) if dtype == 'e4m3' else {}
    y, _ = gdn2.linear_fwd(x.to(DT[dtype]), w.to(DT[dtype]), out_dtype=torch.float32, **scale)
    same('y', y, want)


@pytest.mark.parametrize('dtype', ['bf16', 'f32'])
@pytest.mark.parametrize('M,N,K', [(64, 2 ** 20, 16), (70, 24, 2 ** 20), (33, 2 ** 20 - 1, 9), (40, 9, 2 ** 20 - 1)])
def test_gradient_of_the_most_features(M, N, K, dtype):
    gradient(M, N, K, dtype, 3, 2)
