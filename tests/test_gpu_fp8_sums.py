"""How products of 8-bit matrices are added up: in fp32 in every call that does not ask for fast sums, with the loss
that the header states in those that do."""
import numpy as np
import pytest

from oracle import fp8_ref as R

from gpu_util import mark

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
tg = pytest.importorskip("tile_shape_autotuning_amd")

E4M3 = torch.float8_e4m3fn
BOTH = (torch.bfloat16, torch.float32)

# one tile of the stream and several, each tile of the kernel for many rows, whole and ragged, reductions in parts
SHAPES = [(1, 40, 384), (16, 300, 1000), (64, 80, 260), (65, 80, 260), (100, 1000, 9000), (200, 100, 2600),
          (300, 4000, 1400), (513, 129, 2048), (2050, 8200, 260), (1500, 5000, 260), (2048, 2100, 130)]


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _np(t):
    return t.double().cpu().numpy()


def _f8(codes, scales, K, block):
    def cuda(a):
        return torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return tg.F8(cuda(codes).view(E4M3), cuda(np.asarray(scales, np.float32)), K, block)


def _cancelling(rng, M, N, K, block, lead=()):
    """A and B whose products in each row's own eight k are 448 * 448 and seven of 1, and in another eight -448 * 448:
    (A, B, product).  Sums of 200711 at most, in whole numbers: exact in fp32 in any order, and 7 of a scale as bf16."""
    C, Kp = K // 128, -(-K // 128) * 128               # in whole chunks of 128
    m = np.arange(M)
    chunk, own = m % C, m % 16
    other = (own + 1 + m // 16 % 15) % 16
    a = np.zeros((M, Kp))
    for i in range(8):
        a[m, 128 * chunk + 8 * own + i] = 448.0 if i == 0 else 1.0
    a[m, 128 * chunk + 8 * other] = -448.0
    sign = rng.choice([-1.0, 1.0], (*lead, N))
    b = np.ones((*lead, N, Kp))
    b[..., ::8] = 448.0
    b[..., K:] = 0.0
    b = sign[..., None] * b
    powers = np.array([0.5, 1.0, 2.0], np.float32)
    sa, sb = rng.choice(powers, (M, Kp // 128)), rng.choice(powers, (*lead, -(-N // block), Kp // 128))
    of_column = sb[..., np.arange(N) // block, :]      # [.., N, chunk]
    want = 7.0 * sa[m, chunk][:, None] * np.moveaxis(of_column[..., chunk], -1, -2) * sign[..., None, :]
    return _f8(R.nearest(a), sa, K, 1), _f8(R.nearest(b), sb, K, block), want


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("block", [1, 128])
def test_small_products_survive_large_ones_that_cancel(M, N, K, block):
    A, B, want = _cancelling(np.random.default_rng(M + N), M, N, K, block)
    mark(f"gemm_fp8 cancelling {M}x{N}x{K} block {block}")
    for dt in BOTH:
        assert np.array_equal(_np(tg.gemm_fp8(A, B, out_dtype=dt)), want), dt


@pytest.mark.parametrize("n,E,N", [(5, 3, 40), (60, 2, 300), (400, 2, 520), (2100, 3, 600), (900, 30, 130)])
@pytest.mark.parametrize("block", [1, 128])
def test_small_products_of_experts_survive(n, E, N, block):
    rng = np.random.default_rng(n + N)
    A, B, all_of = _cancelling(rng, n, N, 384, block, (E,))
    offsets = np.concatenate([[0], np.sort(rng.integers(0, n + 1, E - 1)), [n]]).astype(np.int32)
    want = np.concatenate([all_of[e, offsets[e]:offsets[e + 1]] for e in range(E)])
    mark(f"moe_gemm_fp8 cancelling {n} rows {E} experts {N} block {block}")
    for dt in BOTH:
        C = tg.moe_gemm_fp8(A, B, torch.from_numpy(offsets).cuda(), out_dtype=dt)
        assert np.array_equal(_np(C), want), dt


def _random(rng, R_, K, block, lead=()):
    """Normal elements in columns of different size, quantised: (F8, codes' values, a scale for each row and chunk)."""
    x = rng.standard_normal((*lead, R_, K)) * np.exp(rng.standard_normal(K))
    parts = [R.quantise(f.astype(np.float32).astype(np.float64), block) for f in x.reshape(-1, R_, K)]
    codes, scales = np.stack([p[0] for p in parts]), np.stack([p[1] for p in parts])
    q = _f8(codes.reshape(*lead, *codes.shape[1:]), scales.reshape(*lead, *scales.shape[1:]), K, block)
    rows = scales[:, np.arange(R_) // block].astype(np.float64)
    return q, R.VALUES[codes].reshape(*lead, R_, -1), rows.reshape(*lead, R_, -1)


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("block", [1, 128])
def test_bf16_results_are_the_fp32_results_rounded(M, N, K, block):
    rng = np.random.default_rng(M + N + K)
    A, B = _random(rng, M, K, 1)[0], _random(rng, N, K, block)[0]
    bias = torch.from_numpy(rng.standard_normal(N).astype(np.float32)).cuda()
    for kw in (dict(), dict(bias=bias, act="gelu")):
        D, C = (tg.gemm_fp8(A, B, out_dtype=dt, **kw) for dt in BOTH)
        assert torch.equal(D, C.to(torch.bfloat16)), kw


@pytest.mark.parametrize("n", [5, 60, 700])
@pytest.mark.parametrize("block", [1, 128])
def test_bf16_results_of_experts_are_the_fp32_results_rounded(n, block):
    rng = np.random.default_rng(n)
    A, B = _random(rng, n, 700, 1)[0], _random(rng, 200, 700, block, (3,))[0]
    offsets = torch.tensor([0, n // 3, n // 3, n], dtype=torch.int32, device="cuda")
    D, C = (tg.moe_gemm_fp8(A, B, offsets, out_dtype=dt) for dt in BOTH)
    assert torch.equal(D, C.to(torch.bfloat16))


def _sums(a, sa, b, sb):
    """(product, how far fast sums may be off) of codes' values [R, Kp] with scales [R, chunk].

    Each product that is no multiple of its eight's step, 2^-13 of the power of two of the largest, may lose less than
    that step.  What is left is added up in fp32: 16 eights and a starting sum a chunk, eight products each, and the
    chunks', each addition off by at most 2^-23 of the sum of magnitudes (whether it rounds or cuts)."""
    M, N, C = len(a), len(b), sa.shape[1]
    want, off = np.zeros((M, N)), np.zeros((M, N))
    size = np.zeros((M, N))
    for c in range(C):
        at = np.s_[:, 128 * c:128 * (c + 1)]
        p = (a[at][:, None] * b[at][None]).reshape(M, N, 16, 8)
        top = np.abs(p).max(axis=3, keepdims=True)
        step = 2.0 ** (np.floor(np.log2(np.where(top > 0, top, 1.0))) - 13)
        cut = np.where(p / step != np.rint(p / step), step, 0.0).sum(axis=(2, 3))
        s = sa[:, c][:, None] * sb[:, c][None]
        want += s * p.sum(axis=(2, 3))
        off += s * cut
        size += s * np.abs(p).sum(axis=(2, 3))
    return want, off + (130 + 2 * C) * 2.0 ** -23 * size


@pytest.mark.parametrize("M,N,K", [(66, 40, 260), (100, 100, 2600), (513, 129, 384), (2050, 300, 200), (100, 64, 9000)])
@pytest.mark.parametrize("block", [1, 128])
def test_fast_sums_lose_what_the_header_says(M, N, K, block):
    rng = np.random.default_rng(M * N)
    (A, a, sa), (B, b, sb) = _random(rng, M, K, 1), _random(rng, N, K, block)
    rows = np.unique(np.r_[0:40, M - 27:M])            # of the first and the last tiles
    want, off = _sums(a[rows], sa[rows], b, sb)
    mark(f"gemm_fp8 fast sums {M}x{N}x{K} block {block}")
    C = _np(tg.gemm_fp8(A, B, out_dtype=torch.float32, fast_sums=True))[rows]
    assert (np.abs(C - want) <= off).all()
    D = _np(tg.gemm_fp8(A, B, fast_sums=True))[rows]
    assert (np.abs(D - want) <= off + 2.0 ** -8 * (np.abs(want) + off)).all()


@pytest.mark.parametrize("n", [400, 1500])
@pytest.mark.parametrize("block", [1, 128])
def test_fast_sums_of_experts_lose_what_the_header_says(n, block):
    rng = np.random.default_rng(n)
    (A, a, sa), (B, b, sb) = _random(rng, n, 400, 1), _random(rng, 140, 400, block, (2,))
    ends = np.array([0, n // 4, n], np.int32)
    C = _np(tg.moe_gemm_fp8(A, B, torch.from_numpy(ends).cuda(), out_dtype=torch.float32, fast_sums=True))
    for e in range(2):
        rows = np.unique(np.r_[ends[e]:ends[e] + 20, ends[e + 1] - 20:ends[e + 1]])
        want, off = _sums(a[rows], sa[rows], b[e], sb[e])
        assert (np.abs(C[rows] - want) <= off).all()


def test_few_rows_have_the_same_bits_with_fast_sums():
    rng = np.random.default_rng(2)
    for M in (1, 64):
        A, B = _random(rng, M, 700, 1)[0], _random(rng, 90, 700, 128)[0]
        for dt in BOTH:
            assert torch.equal(tg.gemm_fp8(A, B, out_dtype=dt), tg.gemm_fp8(A, B, out_dtype=dt, fast_sums=True))


@pytest.mark.parametrize("n,N,K", [(7, 150, 1000), (90, 300, 777), (1500, 260, 400)])
@pytest.mark.parametrize("block", [1, 128])
def test_sums_of_experts_are_fp32(n, N, K, block):
    rng = np.random.default_rng(n + K)
    (A, a, sa), (B, b, sb) = _random(rng, n, K, 1), _random(rng, N, K, block, (3,))
    ends = np.array([0, n // 2, n // 2 + 1, n], np.int32)
    C = _np(tg.moe_gemm_fp8(A, B, torch.from_numpy(ends).cuda(), out_dtype=torch.float32))
    for e in range(3):
        at = np.s_[ends[e]:ends[e + 1]]
        left, right = a[at] * np.repeat(sa[at], 128, axis=1), b[e] * np.repeat(sb[e], 128, axis=1)
        # additions as in _sums; nothing is cut
        off = (130 + 2 * sa.shape[1]) * 2.0 ** -23 * (np.abs(left) @ np.abs(right).T)
        assert (np.abs(C[at] - left @ right.T) <= off).all()
