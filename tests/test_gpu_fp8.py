"""GPU parity of 8-bit matrices, their products and sorted experts against the fp64 oracle.

Quantisation, sorting and copying are compared bit by bit.  Products of small
integers with powers of two as scales are exact in fp32, in any order: fp32
results are the oracle's bits and bf16 results its rounding.  Elsewhere the
bounds are derived beside the test: a rounding to bf16 is off by at most 2^-9 of
the next power of two, so 2^-8 of the value, one to fp32 by 2^-24.
"""
import numpy as np
import pytest

from oracle import fp8_ref as R
from oracle import gemm_ref

from gpu_util import mark

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
tg = pytest.importorskip("tile_shape_autotuning_amd")

E4M3 = torch.float8_e4m3fn


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _np(t):
    return t.double().cpu().numpy()


def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _put(a, name):
    """fp64 values that the type holds, on the GPU."""
    return _cuda(np.asarray(a, np.float32)).to(_dtype(name))


def _held(a, name):
    return R.round_bf16(a) if name == "bf16" else np.asarray(a, np.float32).astype(np.float64)


def _f8(codes, scales, K, block):
    return tg.F8(_cuda(codes).view(E4M3), _cuda(np.asarray(scales, np.float32)), K, block)


def _codes(t):
    return t.view(torch.uint8).cpu().numpy()


# ---------------------------------------------------------------- quantisation
QUANT = [(1, 1), (1, 128), (3, 130), (128, 128), (129, 257), (5, 1000), (200, 96), (64, 4096), (17, 777), (300, 384),
         (1, 4099), (255, 1), (130, 640)]


@pytest.mark.parametrize("R_,K", QUANT)
@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("dtype,along", [("bf16", True), ("f32", True), ("bf16", False), ("f32", False)])
def test_quantize_gives_the_oracles_codes(R_, K, block, dtype, along):
    rng = np.random.default_rng(R_ * 7 + K)
    x = rng.standard_normal((2, R_, K)) * 10.0 ** rng.uniform(-3, 3, (2, R_, 1))
    # quotients on and next to the middle of two codes, a row of zeros, tiny and subnormal rows
    mids = (R.VALUES[1:127] + R.VALUES[:126]) / 2
    x[0, 0] = rng.choice(mids, K) * rng.choice([-1, 1], K)
    x[0, 0, 0] = 448.0
    x[0, R_ // 2, : K // 2] = 0.0
    x[1, R_ // 2] = rng.choice(mids, K) * (1 + rng.choice([-1, 0, 1], K) * 2.0 ** -23) * 3.7
    x[1, 0] *= 2.0 ** -125
    x[1, R_ - 1] *= 2.0 ** -140 if dtype == "f32" else 2.0 ** -118
    x = _held(x, dtype)
    t = _put(x, dtype)
    if not along:
        t = t.transpose(1, 2).contiguous().transpose(1, 2)
    mark(f"fp8_quantize {R_}x{K} block {block} {dtype} along {along}")
    q, values = tg.fp8_quantize(t, block, values=True)
    torch.cuda.synchronize()
    assert values.dtype == t.dtype and values.shape == t.shape and values.stride() == t.stride()
    for i in range(2):
        codes, scales = R.quantise(x[i], block)
        assert np.array_equal(q.scales[i].cpu().numpy(), scales)
        assert np.array_equal(_codes(q.codes[i]), codes), "codes, and zeros past K"
        # one product of fp32, rounded to fp32, then to the type
        v = _held(R.dense(codes, scales, K, block).astype(np.float32), dtype)
        assert np.array_equal(_np(values[i]), v)
    again = tg.fp8_quantize(t, block)
    assert torch.equal(again.codes.view(torch.uint8), q.codes.view(torch.uint8))


@pytest.mark.parametrize("along", [True, False])
@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_quantize_rounds_every_kind_of_quotient(block, along, dtype):
    # every sign, exponent and leading mantissa bits of a bf16 against scales of 1 and 448 / 300
    bits = np.arange(1 << 16, dtype=np.uint32) << 16
    v = bits.view(np.float32)
    v = v[np.isfinite(v) & (np.abs(v) <= 300)].astype(np.float64)
    for top in (448.0, 300.0):
        x = np.concatenate([v, np.zeros(-len(v) % 127)]).reshape(-1, 127)
        x = np.concatenate([np.full((len(x), 1), top), x], axis=1)
        t = _put(x, dtype)
        t = t if along else t.transpose(0, 1).contiguous().transpose(0, 1)
        q = tg.fp8_quantize(t, block)
        codes, scales = R.quantise(x, block)
        assert np.array_equal(q.scales.cpu().numpy(), scales) and np.array_equal(_codes(q.codes), codes)


@pytest.mark.parametrize("along", [True, False])
@pytest.mark.parametrize("block", [1, 128])
def test_quantize_marks_blocks_that_are_not_finite(block, along):
    x = torch.ones((260, 300), device="cuda")
    x[3, 5], x[200, 290] = float("nan"), float("-inf")
    t = x if along else x.transpose(0, 1).contiguous().transpose(0, 1)
    q, v = tg.fp8_quantize(t, block, values=True)
    codes, scales = R.quantise(x.double().cpu().numpy(), block)
    assert np.array_equal(q.scales.cpu().numpy(), scales, equal_nan=True)
    assert np.array_equal(_codes(q.codes), codes)
    assert np.array_equal(np.isnan(_np(v)), codes[:, :300] == 0x7F)


def test_quantize_the_transpose_is_the_transpose_of_blocks():
    W = torch.randn((400, 270), device="cuda").to(torch.bfloat16)
    a, b = tg.fp8_quantize(W, 128), tg.fp8_quantize(W.transpose(0, 1), 128)
    assert torch.equal(a.scales, b.scales.t())
    assert torch.equal(a.codes[:, :270].view(torch.uint8), b.codes[:, :400].view(torch.uint8).t())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("along", [True, False])
def test_quantize_every_short_length(dtype, along):
    """Rows of 1 to 19 elements (of 1 to 19 matrices' columns) between elements that are not numbers."""
    rng = np.random.default_rng(19)
    for n in range(1, 20):
        x = _held(rng.standard_normal((9, n)), dtype)
        buf = torch.full((9 * n + 14,), float("nan"), device="cuda", dtype=_dtype(dtype))
        t = buf[7:7 + 9 * n].view(9, n)
        t.copy_(_put(x, dtype))
        view, want = (t, x) if along else (t.transpose(0, 1), x.T)
        for block in (1, 128):
            q, values = tg.fp8_quantize(view, block, values=True)
            codes, scales = R.quantise(np.ascontiguousarray(want), block)
            assert np.array_equal(q.scales.cpu().numpy(), scales) and np.array_equal(_codes(q.codes), codes), n
            v = _held(R.dense(codes, scales, want.shape[1], block).astype(np.float32), dtype)
            assert np.array_equal(_np(values), v), n


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_quantize_many_rows(dtype):
    """More chunks than a lane takes one at a time, the last ones ragged in rows and in K."""
    rng = np.random.default_rng(8)
    x = _held(rng.standard_normal((8003, 1030)) * 10.0 ** rng.uniform(-3, 3, (8003, 1)), dtype)
    q = tg.fp8_quantize(_put(x, dtype))
    codes, scales = R.quantise(x, 1)
    assert np.array_equal(q.scales.cpu().numpy(), scales) and np.array_equal(_codes(q.codes), codes)


def test_quantize_a_view_off_16_bytes():
    base = torch.randn(70 * 256 + 3, device="cuda").to(torch.bfloat16)
    for off in (1, 3):
        t = base[off:off + 70 * 256].view(70, 256)
        for block in (1, 128):
            q = tg.fp8_quantize(t, block)
            codes, scales = R.quantise(_np(t), block)
            assert np.array_equal(q.scales.cpu().numpy(), scales) and np.array_equal(_codes(q.codes), codes)


# ---------------------------------------------------------------- products
def _integers(rng, R_, K, block, lead=()):
    """Small integers with powers of two as scales: (F8, fp64 elements)."""
    Kp = -(-K // 128) * 128
    v = np.zeros((*lead, R_, Kp))
    v[..., :K] = rng.integers(-4, 5, (*lead, R_, K))
    scales = rng.choice(np.array([0.5, 1.0, 2.0], np.float32), (*lead, -(-R_ // block), Kp // 128))
    codes = R.nearest(v)
    flat, fs = codes.reshape(-1, R_, Kp), scales.reshape(-1, *scales.shape[-2:])
    dense = np.stack([R.dense(c, s, K, block) for c, s in zip(flat, fs)]).reshape(*lead, R_, K)
    return _f8(codes, scales, K, block), dense


GEMMS = [(1, 1, 1), (1, 16, 128), (1, 256, 4096), (3, 17, 33), (16, 300, 1000), (17, 64, 256), (33, 257, 513),
         (64, 1001, 777), (65, 80, 128), (100, 48, 2100), (128, 128, 128), (130, 257, 640), (256, 256, 1024),
         (257, 520, 300), (300, 1000, 130), (513, 129, 2048), (2, 3000, 96), (1, 40, 9000), (70, 33, 9000),
         (1000, 260, 384), (40, 5000, 260), (520, 770, 1280),
         # each tile, whole and ragged, and reductions in parts
         (2050, 8200, 260), (600, 4100, 390), (2048, 2100, 130), (1500, 5000, 260), (3000, 2996, 200), (100, 1000, 9000),
         (128, 1100, 4100), (300, 4000, 1400), (66, 250, 5000), (200, 100, 2600),
         (2706, 2903, 100), (2852, 666, 100), (395, 900, 2600), (72, 4157, 5000), (1060, 192, 5000), (1607, 283, 5000)]


@pytest.mark.parametrize("M,N,K", GEMMS)
@pytest.mark.parametrize("block", [1, 128])
def test_gemm_is_exact_on_integers(M, N, K, block):
    # elements up to 4 * 2, products 64 in quarters: sums below 64 * 4 * 9000 < 2^24 quarters
    rng = np.random.default_rng(M + 3 * N + K)
    A, a = _integers(rng, M, K, 1)
    B, b = _integers(rng, N, K, block)
    want = a @ b.T
    mark(f"gemm_fp8 {M}x{N}x{K} block {block}")
    C = tg.gemm_fp8(A, B, out_dtype=torch.float32)
    torch.cuda.synchronize()
    assert np.array_equal(_np(C), want)
    assert np.array_equal(_np(tg.gemm_fp8(A, B)), R.round_bf16(want))
    bias = rng.integers(-50, 50, N).astype(np.float32)
    assert np.array_equal(_np(tg.gemm_fp8(A, B, _cuda(bias), act="relu")), R.round_bf16(np.maximum(want + bias, 0)))


def _random(rng, R_, K, block, lead=()):
    x = rng.standard_normal((*lead, R_, K)) * np.exp(rng.standard_normal(K))
    flat = x.reshape(-1, R_, K)
    parts = [R.quantise(_held(f, "f32"), block) for f in flat]
    codes, scales = np.stack([p[0] for p in parts]), np.stack([p[1] for p in parts])
    dense = np.stack([R.dense(c, s, K, block) for c, s in parts])
    return (_f8(codes.reshape(*lead, *codes.shape[1:]), scales.reshape(*lead, *scales.shape[1:]), K, block),
            dense.reshape(*lead, R_, K))


def _bound(a, b, K):
    """How far fp32 sums may be off: 128 products and a starting sum a chunk, each addition off by at most 2^-23 of the
    sum of magnitudes (whether it rounds or cuts), the two scales' product, its product with the sum, and the additions
    of the chunks."""
    return (130 + 2 * -(-K // 128)) * 2.0 ** -23 * (np.abs(a) @ np.abs(b).T)


def _cut(a, b):
    """What the matrix cores' 8-bit form may cut off: 7 * 2^-13 of the largest of each eight products, which is at most
    that of the sum of their magnitudes."""
    return 7 * 2.0 ** -13 * (np.abs(a) @ np.abs(b).T)


@pytest.mark.parametrize("M,N,K", [(1, 300, 1000), (40, 130, 777), (200, 257, 1500), (300, 512, 4096), (64, 64, 20000), (70, 64, 20000)])
@pytest.mark.parametrize("block", [1, 128])
def test_gemm_within_the_bound_of_its_sums(M, N, K, block):
    rng = np.random.default_rng(M + K)
    A, a = _random(rng, M, K, 1)
    B, b = _random(rng, N, K, block)
    want, off = a @ b.T, _bound(a, b, K)
    mark(f"gemm_fp8 random {M}x{N}x{K} block {block}")
    C = _np(tg.gemm_fp8(A, B, out_dtype=torch.float32))
    assert (np.abs(C - want) <= off).all()
    # what fp32 sums are off by in practice: no more than a few of their roundings in the mean
    assert np.sqrt(np.mean((C - want) ** 2)) <= 8 * 2.0 ** -24 * np.sqrt(np.mean((np.abs(a) @ np.abs(b).T) ** 2))
    # bf16 results: of each eight products seven may be cut by up to 2^-13 of the largest; and the rounding
    off = off + _cut(a, b)
    D = _np(tg.gemm_fp8(A, B))
    assert (np.abs(D - want) <= off + 2.0 ** -8 * (np.abs(want) + off)).all()
    # in the mean a few 1e-5 of the result (rounding to bf16: 1.7e-3, 2^-8 / sqrt 3 at the most)
    assert np.sqrt(np.mean((D - want) ** 2)) <= 2.0 ** -8 / 3 ** 0.5 * np.sqrt(np.mean(want ** 2))


def test_gemm_gelu_and_bias():
    rng = np.random.default_rng(5)
    for M in (5, 130):
        A, a = _random(rng, M, 300, 1)
        B, b = _random(rng, 70, 300, 128)
        bias = rng.standard_normal(70).astype(np.float32)
        z = a @ b.T / 8 + bias
        B = B._replace(scales=B.scales / 8)
        want = gemm_ref.gelu(z) if hasattr(gemm_ref, "gelu") else None
        if want is None:
            from math import erf
            want = 0.5 * z * (1 + np.vectorize(erf)(z / np.sqrt(2)))
        C = _np(tg.gemm_fp8(A, B, _cuda(bias), act="gelu", out_dtype=torch.float32))
        # GELU's slope is below 1.13; its form here is off by 0.5 |z| 1.5e-7, and 8 roundings
        off = 1.13 * (_bound(a, b, 300) / 8 + 2.0 ** -23 * np.abs(z)) + np.abs(z) * (0.75e-7 + 8 * 2.0 ** -24)
        assert (np.abs(C - want) <= off).all()


def test_gemm_nan_stays_in_its_rows_and_columns():
    rng = np.random.default_rng(8)
    for M in (4, 200):
        A, a = _integers(rng, M, 384, 1)
        B, b = _integers(rng, 150, 384, 1)
        want = a @ b.T
        codes = A.codes.view(torch.uint8).clone()
        codes[2, 5] = 0x7F
        scales = B.scales.clone()
        scales[77, 1] = float("nan")
        C = _np(tg.gemm_fp8(A._replace(codes=codes.view(E4M3)), B._replace(scales=scales), out_dtype=torch.float32))
        bad = np.zeros_like(want, bool)
        bad[2], bad[:, 77] = True, True
        assert np.isnan(C[bad]).all() and np.array_equal(C[~bad], want[~bad])


def test_gemm_writes_its_output_only():
    rng = np.random.default_rng(9)
    for M, N in ((3, 77), (65, 131), (257, 200)):
        A, a = _integers(rng, M, 200, 1)
        B, b = _integers(rng, N, 200, 128)
        for dt in (torch.float32, torch.bfloat16):
            buf = torch.full((M * N + 128,), 9.0, device="cuda", dtype=dt)
            out = buf[64:64 + M * N].view(M, N)
            r = tg.gemm_fp8(A, B, out=out)
            assert r.data_ptr() == out.data_ptr()
            assert bool((buf[:64] == 9).all()) and bool((buf[64 + M * N:] == 9).all())
            assert np.array_equal(_np(out), _held(a @ b.T, "bf16" if dt == torch.bfloat16 else "f32"))


@pytest.mark.parametrize("M,N", [(3, 64), (300, 72), (1030, 2056), (2050, 4104)])
def test_gemm_into_rows_off_alignment(M, N):
    """Outputs that begin 2, 8 and 16 bytes past an aligned address: element, four- and eight-element stores."""
    rng = np.random.default_rng(M)
    A, a = _integers(rng, M, 136, 1)
    B, b = _integers(rng, N, 136, 128)
    want = R.round_bf16(a @ b.T)
    for off in (1, 4, 8):
        buf = torch.full((M * N + 32,), 9.0, device="cuda", dtype=torch.bfloat16)
        out = buf[off:off + M * N].view(M, N)
        tg.gemm_fp8(A, B, out=out)
        assert np.array_equal(_np(out), want)
        assert bool((buf[:off] == 9).all()) and bool((buf[off + M * N:] == 9).all())


def test_experts_that_hardly_any_or_all_rows_are_for():
    """Averages of few rows an expert, but one has them all; and the other way round."""
    rng = np.random.default_rng(6)
    for E, n in ((64, 1500), (300, 40)):
        A, a = _integers(rng, n, 200, 1)
        B, b = _integers(rng, 80, 200, 128, (E,))
        offsets = np.zeros(E + 1, np.int32)
        offsets[E // 2 + 1:] = n - 1
        offsets[E] = n                                 # all but one in the middle, one at the end
        C = _np(tg.moe_gemm_fp8(A, B, _cuda(offsets), out_dtype=torch.float32))
        assert np.array_equal(C[:n - 1], a[:n - 1] @ b[E // 2].T) and np.array_equal(C[n - 1:], a[n - 1:] @ b[E - 1].T)


def test_a_layers_gradients():
    """The three products of a training step against the formula on the values that the codes stand for."""
    rng = np.random.default_rng(10)
    T, N, K = 200, 150, 270
    x, W, dy = (_put(rng.standard_normal(s), "bf16") for s in ((T, K), (N, K), (T, N)))

    def both(t, block):
        q, v = tg.fp8_quantize(t.float(), block, values=True)
        return q, _np(v)

    for left, right, block in ((x, W, 128), (dy, W.transpose(0, 1), 128), (dy.transpose(0, 1), x.transpose(0, 1), 1)):
        lf = left.float() if left.is_contiguous() else left.transpose(0, 1).float().transpose(0, 1)
        rf = right.float() if right.is_contiguous() else right.transpose(0, 1).float().transpose(0, 1)
        (A, a), (B, b) = both(lf, 1), both(rf, block)
        C = _np(tg.gemm_fp8(A, B, out_dtype=torch.float32))
        # values are the elements rounded to fp32
        off = _bound(a, b, a.shape[1]) + 2.0 ** -22 * (np.abs(a) @ np.abs(b).T)
        assert (np.abs(C - a @ b.T) <= off).all()
    # and against differences: the loss sum(dy * (x W^T)) in the values, along a random direction of x
    (A, a), (B, b) = both(dy, 1), both(W.transpose(0, 1).float(), 128)
    dx = _np(tg.gemm_fp8(A, B, out_dtype=torch.float32))
    d = rng.standard_normal((T, K))
    xv = _np(x)
    diff = (np.sum(a * ((xv + 1e-3 * d) @ b)) - np.sum(a * ((xv - 1e-3 * d) @ b))) / 2e-3
    assert abs(diff - np.sum(dx * d)) <= np.sum((_bound(a, b, N) + 1e-7 * (np.abs(a) @ np.abs(b).T)) * np.abs(d))


# ---------------------------------------------------------------- order
def _ids(rng, T, E, k, kind):
    if kind == "one":
        ids = np.full((T, k), E - 1)
    elif kind == "repeats":
        ids = rng.integers(0, E, (T, k))
    elif kind == "none":
        ids = np.full((T, k), -1)
    else:
        ids = np.argsort(rng.standard_normal((T, E)), axis=1)[:, :k]
        if kind == "away":
            ids = np.where(rng.random((T, k)) < 0.3, rng.choice([-1, E, 2 ** 31 - 1, -2 ** 31], (T, k)), ids)
    return ids.astype(np.int32)


ORDERS = [(1, 8, 2, "plain"), (1, 1, 1, "plain"), (5, 16, 4, "away"), (64, 64, 6, "plain"), (257, 8, 3, "repeats"),
          (1000, 256, 8, "away"), (3, 1024, 16, "plain"), (4099, 64, 8, "plain"), (2500, 1024, 5, "away"),
          (3000, 7, 7, "plain"), (700, 5, 2, "one"), (50, 4, 2, "none"), (40000, 33, 3, "repeats"), (2048, 128, 1, "plain"),
          (20000, 2, 16, "one"), (256, 16, 8, "plain"), (257, 16, 8, "away"), (50000, 1024, 16, "plain"), (3000, 1, 1, "one"),
          (70000, 300, 4, "repeats"), (1025, 3, 2, "none")]


@pytest.mark.parametrize("T,E,k,kind", ORDERS)
def test_sort_gives_the_oracles_order(T, E, k, kind):
    rng = np.random.default_rng(T + E)
    ids = rng.integers(0, E, (T, k)).astype(np.int32) if kind == "repeats" or k > E else _ids(rng, T, E, k, kind)
    position, source, offsets = R.order(ids, E)
    mark(f"moe_sort {T} tokens {E} experts {k} choices {kind}")
    order = tg.moe_sort(_cuda(ids), E)
    torch.cuda.synchronize()
    assert np.array_equal(order.offsets.cpu().numpy(), offsets)
    assert np.array_equal(order.position.cpu().numpy(), position)
    assert np.array_equal(order.source.cpu().numpy(), source)


def test_sort_of_nothing():
    order = tg.moe_sort(torch.empty((0, 3), dtype=torch.int32, device="cuda"), 5)
    assert order.position.shape == (0, 3) and order.source.shape == (0,)
    assert order.offsets.tolist() == [0] * 6


ROWS = [(1, 8, 2, 16, "plain"), (5, 16, 4, 1000, "away"), (33, 4, 2, 1, "plain"), (70, 8, 8, 259, "away"),
        (300, 64, 6, 2048, "plain"), (9, 16, 16, 8192, "plain"), (40, 3, 2, 77, "repeats"), (20, 4, 3, 30, "none"),
        (130, 32, 5, 514, "away"), (6, 4, 2, 2052, "plain"), (6, 8, 5, 4104, "away"), (3, 4, 3, 5, "plain")]


def _order(ids, E):
    return tg.MoeOrder(*(_cuda(a) for a in R.order(ids, E)))


@pytest.mark.parametrize("T,E,k,H,kind", ROWS)
@pytest.mark.parametrize("dtype", ["bf16", "f32", "fp8"])
def test_gather_moves_rows(T, E, k, H, kind, dtype):
    rng = np.random.default_rng(T * H)
    ids = _ids(rng, T, E, k, kind)
    order = _order(ids, E)
    position = order.position.cpu().numpy()
    mark(f"moe_gather {T}x{H} k {k} {dtype} {kind}")
    if dtype == "fp8":
        codes = rng.integers(0, 256, (T, -(-H // 128) * 128), dtype=np.uint8)
        scales = rng.standard_normal((T, -(-H // 128))).astype(np.float32)
        x = _f8(codes, scales, H, 1)
        out = _f8(np.full((T * k, codes.shape[1]), 7, np.uint8), np.full((T * k, scales.shape[1]), 3.0), H, 1)
        r = tg.moe_gather(x, order, out=out)
        assert np.array_equal(_codes(r.codes), R.gather(codes, position, np.full((T * k, codes.shape[1]), 7, np.uint8)))
        assert np.array_equal(r.scales.cpu().numpy(),
                              R.gather(scales, position, np.full((T * k, scales.shape[1]), 3.0, np.float32)))
        return
    x = _held(rng.standard_normal((T, H)), dtype)
    out = torch.full((T * k, H), 3.0, dtype=_dtype(dtype), device="cuda")
    r = tg.moe_gather(_put(x, dtype), order, out=out)
    want = R.gather(x, position, np.full((T * k, H), 3.0))
    assert np.array_equal(_np(r), want), "rows, and those behind the last left as they were"
    if kind == "plain":
        assert np.array_equal(_np(tg.moe_gather(_put(x, dtype), order)), want)


@pytest.mark.parametrize("T,E,k,H,kind", ROWS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_combine_and_its_gradients(T, E, k, H, kind, dtype):
    rng = np.random.default_rng(T + H)
    ids = _ids(rng, T, E, k, kind)
    order = _order(ids, E)
    position = order.position.cpu().numpy()
    x, dy = (_held(rng.standard_normal((n, H)), dtype) for n in (T * k, T))
    w = rng.random((T, k)).astype(np.float32)
    w64 = w.astype(np.float64)
    mark(f"moe_combine {T}x{H} k {k} {dtype} {kind}")
    step = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    for weights, arg in ((w64, _cuda(w)), (np.ones((T, k)), None)):
        y = _np(tg.moe_combine(_put(x, dtype), order, arg))
        want = R.combine(x, position, weights)
        # k products and additions in fp32, one rounding to the type
        size = R.combine(np.abs(x), position, weights)
        off = 2 * k * 2.0 ** -24 * size
        assert (np.abs(y - want) <= off + step * (np.abs(want) + off)).all()
    out = torch.full((T * k, H), 3.0, dtype=_dtype(dtype), device="cuda")
    dx, dw = tg.moe_combine_grad(_put(dy, dtype), _put(x, dtype), order, _cuda(w), out=out)
    assert dx.data_ptr() == out.data_ptr()
    want_dx, want_dw = R.combine_grad(dy, x, position, w64, np.full((T * k, H), 3.0))
    assert (np.abs(_np(dx) - want_dx) <= (step + 2.0 ** -24) * np.abs(want_dx) + 2.0 ** -140).all()
    behind = np.ones(T * k, bool)
    behind[position[position >= 0]] = False
    assert (_np(dx)[behind] == 3.0).all(), "rows behind the last left as they were"
    _, size = R.combine_grad(np.abs(dy), np.abs(x), position, w64, np.zeros((T * k, H)))
    assert (np.abs(_np(dw) - want_dw) <= (H + 2) * 2.0 ** -24 * size).all()
    assert (_np(dw)[position < 0] == 0).all()


def test_combine_gradient_agrees_with_differences():
    rng = np.random.default_rng(3)
    T, E, k, H = 20, 8, 3, 50
    order = _order(_ids(rng, T, E, k, "away"), E)
    x, dy, w = (_cuda(rng.standard_normal(s).astype(np.float32)) for s in ((T * k, H), (T, H), (T, k)))
    dx, dw = tg.moe_combine_grad(dy, x, order, w, out=torch.zeros_like(x))
    for name, grad in (("x", dx), ("w", dw)):
        d = _cuda(rng.choice([-1.0, 1.0], grad.shape).astype(np.float32))
        hi = tg.moe_combine(x + d if name == "x" else x, order, w + d if name == "w" else w)
        lo = tg.moe_combine(x - d if name == "x" else x, order, w - d if name == "w" else w)
        # linear in each: steps of one are as good as small ones
        got = float((dy.double() * (hi.double() - lo.double())).sum()) / 2
        want = float((grad.double() * d.double()).sum())
        size = float((dy.abs().double() * (hi.abs() + lo.abs()).double()).sum()) + float(grad.abs().double().sum())
        assert abs(got - want) <= (2 * k + H + 4) * 2.0 ** -23 * (size + float(dy.abs().sum()) * k * 8)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_of_every_short_width(dtype):
    """Rows of small integers of 1 to 40 elements, and about the widths where other kernels take over, off
    alignment between elements that are not numbers: sums are exact."""
    rng = np.random.default_rng(40)
    T, k, E = 13, 3, 4
    ids = _ids(rng, T, E, k, "away")
    order = tg.moe_sort(_cuda(ids), E)
    position = order.position.cpu().numpy()
    has = position >= 0
    n = int(has.sum())
    w = rng.integers(1, 5, (T, k)).astype(np.float32)

    def between(a):
        buf = torch.full((a.size + 10,), float("nan"), device="cuda", dtype=_dtype(dtype))
        t = buf[5:5 + a.size].view(a.shape)
        t.copy_(_put(a, dtype))
        return t

    for H in (*range(1, 41), 255, 257, 511, 513, 1023, 1025, 1031, 2049, 2055):
        x, dy = rng.integers(-4, 5, (T * k, H)).astype(np.float64), rng.integers(-4, 5, (T, H)).astype(np.float64)
        x[n:] = np.nan                                 # rows behind the last
        rows = np.where(has[..., None], np.nan_to_num(x)[position], 0.0)
        tx, tdy = between(x), between(dy)
        y = tg.moe_combine(tx, order, _cuda(w))
        assert np.array_equal(_np(y), _held((w[..., None] * rows).sum(1), dtype)), H
        dx, dw = tg.moe_combine_grad(tdy, tx, order, _cuda(w), out=torch.full_like(tx, 7.0))
        want = np.full((T * k, H), 7.0)
        want[position[has]] = (w[..., None] * dy[:, None])[has]
        assert np.array_equal(_np(dx), _held(want, dtype)), H
        assert np.array_equal(_np(dw), np.where(has, (dy[:, None] * rows).sum(2), 0.0)), H
        out = torch.full((T * k, H), 7.0, device="cuda", dtype=_dtype(dtype))
        tg.moe_gather(tdy, order, out=out)
        want[position[has]] = np.repeat(dy[:, None], k, 1)[has]
        assert np.array_equal(_np(out), want), H


# ---------------------------------------------------------------- experts
EXPERTS = [(1, 8, 2, 64, 128, "plain"), (5, 16, 4, 100, 200, "away"), (64, 8, 2, 257, 300, "plain"),
           (200, 5, 2, 130, 520, "repeats"), (300, 4, 1, 513, 128, "one"), (30, 64, 6, 96, 384, "plain"),
           (40, 3, 2, 33, 129, "none"), (700, 6, 3, 256, 256, "away"), (1200, 3, 2, 300, 640, "plain"),
           (2, 300, 1, 40, 140, "plain"), (130, 2, 1, 520, 1024, "plain"), (2000, 4, 2, 1200, 260, "away"),
           (1500, 8, 2, 550, 130, "plain"), (900, 70, 3, 130, 200, "away"), (1, 2, 1, 9000, 300, "plain")]


@pytest.mark.parametrize("T,E,k,N,K,kind", EXPERTS)
@pytest.mark.parametrize("block", [1, 128])
def test_expert_products_are_exact_on_integers(T, E, k, N, K, kind, block):
    rng = np.random.default_rng(T + N)
    ids = _ids(rng, T, E, k, kind)
    _, _, offsets = R.order(ids, E)
    n = T * k
    A, a = _integers(rng, n, K, 1)
    B, b = _integers(rng, N, K, block, (E,))
    want = np.full((n, N), 5.0)
    for e in range(E):
        want[offsets[e]:offsets[e + 1]] = a[offsets[e]:offsets[e + 1]] @ b[e].T
    mark(f"moe_gemm_fp8 {T} tokens {E} experts k {k} {N}x{K} block {block} {kind}")
    for dt, name in ((torch.float32, "f32"), (torch.bfloat16, "bf16")):
        out = torch.full((n, N), 5.0, dtype=dt, device="cuda")
        C = tg.moe_gemm_fp8(A, B, _cuda(offsets), out=out)
        torch.cuda.synchronize()
        assert np.array_equal(_np(C), _held(want, name)), "rows, and those behind the last left as they were"


def test_offsets_that_name_other_rows_are_cut():
    rng = np.random.default_rng(4)
    A, a = _integers(rng, 40, 128, 1)
    B, b = _integers(rng, 32, 128, 128, (4,))
    want = np.full((40, 32), 5.0)
    want[0:10], want[30:40] = a[0:10] @ b[0].T, a[30:40] @ b[2].T
    offsets = np.array([-7, 10, 10, 99, 10], np.int32)      # expert 1 has none, 2 has 10.., 3 has none
    want[10:40] = a[10:40] @ b[2].T
    out = torch.full((40, 32), 5.0, device="cuda")
    assert np.array_equal(_np(tg.moe_gemm_fp8(A, B, _cuda(offsets), out=out)), want)


# ---------------------------------------------------------------- together
def _layer(x, logits, up, down, k, E):
    """The experts of a gated layer for any number of tokens, and what its backward pass needs."""
    ids, w = tg.moe_route(logits, k)
    order = tg.moe_sort(ids, E)
    rows = tg.moe_gather(tg.fp8_quantize(x), order)
    gu = tg.moe_gemm_fp8(rows, up, order.offsets, out_dtype=torch.float32)
    g, u = gu.chunk(2, dim=1)
    h = tg.fp8_quantize((g * torch.sigmoid(g) * u).to(torch.bfloat16).contiguous())
    z = tg.moe_gemm_fp8(h, down, order.offsets)
    y = tg.moe_combine(z, order, w)
    dz, dw = tg.moe_combine_grad(x, z, order, w)
    dx = tg.moe_combine(tg.moe_gather(x, order), order)
    return y, dz, dw, dx


def _layer_inputs(T, E, H, I, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.randn((T, H), device="cuda", generator=g).to(torch.bfloat16)
    logits = torch.randn((T, E), device="cuda", generator=g)
    up = torch.randn((E, 2 * I, H), device="cuda", generator=g) / H ** 0.5
    down = torch.randn((E, H, I), device="cuda", generator=g) / I ** 0.5
    return x, logits, up, down


@pytest.mark.parametrize("T", [1, 20, 300])
def test_a_layer_agrees_with_the_layer_for_few_tokens(T):
    E, H, I, k = 8, 256, 200, 3
    x, logits, up, down = _layer_inputs(T, E, H, I, T)
    (qu, vu), (qd, vd) = tg.fp8_quantize(up, 128, values=True), tg.fp8_quantize(down, 128, values=True)
    y, dz, dw, dx = _layer(x, logits, qu, qd, k, E)
    ref, _, _ = tg.moe_layer(x, logits, vu.to(torch.bfloat16).view(E, 2, I, H), vd.to(torch.bfloat16).contiguous(), k)
    # e4m3 rounds a value m 2^e by a uniform step of 2^(e-3): rms 2^-3 / sqrt 12 / m, 0.0255 over m in [1, 2).  x
    # enters gate and up: silu(g) u moves by silu'(g) dg u + silu(g) du, 0.0255 sqrt(1.07 + 1) of its size for g, u
    # around one; then the hidden state's own 0.0255: 0.045 in the norm together, and half again for few elements
    assert float((y.float() - ref.float()).norm()) <= 0.07 * float(ref.float().norm())
    # every token went to k rows and back
    assert torch.equal(dx, (k * x.float()).to(torch.bfloat16))


def test_a_layer_on_two_streams_and_in_two_graphs():
    E, H, I, k = 8, 256, 130, 2
    up, down = (tg.fp8_quantize(w, 128) for w in _layer_inputs(1, E, H, I, 0)[2:])
    ins = [_layer_inputs(T, E, H, I, T)[:2] for T in (3, 150)]

    def run(i):
        return _layer(*ins[i], up, down, k, E)

    want = [[t.clone() for t in run(i)] for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ins]
    got = []
    for i, s in enumerate(streams):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got.append(run(i))
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert all(torch.equal(a, b) for a, b in zip(g, w))
    graphs = []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            r = run(i)
        graphs.append((g, r))
    for turn in range(3):
        for x, logits in ins:
            x.copy_(torch.randn(x.shape, device="cuda"))
            logits.copy_(torch.randn(logits.shape, device="cuda"))
        want = [[t.clone() for t in run(i)] for i in range(2)]
        for s, (g, _) in zip(streams, graphs):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for (_, r), w in zip(graphs, want):
            assert all(torch.equal(a, b) for a, b in zip(r, w)), f"replay {turn}"


def test_products_in_parts_in_two_graphs():
    """The reduction in parts has a workspace for each call: two graphs and eager calls between their replays."""
    rng = np.random.default_rng(12)
    ins = []
    for M, N, K in ((100, 1000, 9000), (70, 300, 5000)):
        assert tg._native.gemm_fp8_workspace_bytes(M, N, K) > 0
        A, a = _integers(rng, M, K, 1)
        B, b = _integers(rng, N, K, 128)
        ins.append((A, B, a @ b.T))
    graphs, streams = [], [torch.cuda.Stream() for _ in ins]
    for A, B, _ in ins:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            C = tg.gemm_fp8(A, B, act="relu", out_dtype=torch.float32)
        graphs.append((g, C))
    for turn in range(3):
        for (g, C), s in zip(graphs, streams):
            C.fill_(-1.0)
        torch.cuda.synchronize()
        for (g, C), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        for A, B, want in ins:
            assert np.array_equal(_np(tg.gemm_fp8(A, B, out_dtype=torch.float32)), want)
        torch.cuda.synchronize()
        for (g, C), (_, _, want) in zip(graphs, ins):
            assert np.array_equal(_np(C), np.maximum(want, 0)), f"replay {turn}"


@pytest.mark.parametrize("n_cu", [1, 7, 2 ** 31 - 1])
def test_products_under_any_description(n_cu):
    rng = np.random.default_rng(13)
    desc = tg.get_device_desc()
    desc.n_cu = n_cu
    tg.set_device_override(desc)
    try:
        for M, N, K in ((100, 1000, 2000), (300, 600, 700), (5, 100, 300)):
            A, a = _integers(rng, M, K, 1)
            B, b = _integers(rng, N, K, 1)
            assert np.array_equal(_np(tg.gemm_fp8(A, B, out_dtype=torch.float32)), a @ b.T)
    finally:
        tg.set_device_override(None)


# ---------------------------------------------------------------- offsets past 32 bits
def _far_matrix(lead, R_, K, block):
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    codes = torch.randint(0x30, 0x48, (*lead, R_, K), dtype=torch.uint8, device="cuda", generator=g)
    scales = torch.full((*lead, -(-R_ // block), K // 128), 0.5, device="cuda")
    return tg.F8(codes.view(E4M3), scales, K, block)


def _values64(codes):
    return R.VALUES[codes.view(torch.uint8).cpu().numpy()]


def test_rows_past_32_bits_of_a_product():
    K, M = 8192, 530000                                # 4.3e9 codes
    A, B = _far_matrix((), M, K, 1), _far_matrix((), 16, K, 1)
    C = tg.gemm_fp8(A, B, out_dtype=torch.float32)
    a, b = _values64(A.codes[-70:]) * 0.5, _values64(B.codes) * 0.5
    assert (np.abs(_np(C[-70:]) - a @ b.T) <= _bound(a, b, K)).all()


def test_experts_past_32_bits():
    E, N, K = 530, 1024, 8192                          # 4.4e9 codes
    B = _far_matrix((E,), N, K, 128)
    for n in (6, 600):
        A = _far_matrix((), n, K, 1)
        offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
        offsets[E] = n                                 # all rows are the last expert's
        C = tg.moe_gemm_fp8(A, B, offsets, out_dtype=torch.float32)
        a, b = _values64(A.codes) * 0.5, _values64(B.codes[-1]) * 0.5
        assert (np.abs(_np(C) - a @ b.T) <= _bound(a, b, K)).all()


def test_rows_past_32_bits_of_copies_and_sums():
    n, H = 600000, 4096                                # 4.9e9 bytes
    rows = torch.empty((n, H), dtype=torch.bfloat16, device="cuda")
    position = torch.tensor([[n - 1, 3], [n - 2, -1]], dtype=torch.int32, device="cuda")
    order = tg.MoeOrder(position, position.view(-1), position.view(-1)[:1])
    x = torch.randn((2, H), device="cuda").to(torch.bfloat16)
    r = tg.moe_gather(x, order, out=rows)
    assert torch.equal(r[n - 1], x[0]) and torch.equal(r[3], x[0]) and torch.equal(r[n - 2], x[1])
    w = torch.tensor([[0.5, 0.25], [2.0, 9.0]], device="cuda")
    y = tg.moe_combine(rows, order, w)
    assert torch.equal(y, (x.float() * torch.tensor([[0.75], [2.0]], device="cuda")).to(torch.bfloat16))
    dx, dw = tg.moe_combine_grad(x, rows, order, w, out=rows.clone())
    assert torch.equal(dx[n - 1], x[0] / 2) and torch.equal(dx[n - 2], x[1] * 2)
    own = (x.double() ** 2).sum(1)
    assert float((dw.double() - torch.stack([own[[0, 0]], own[[1, 1]] * torch.tensor([1.0, 0.0], device="cuda")])).abs().max()) \
        <= (H + 2) * 2.0 ** -24 * float(own.max())


@pytest.mark.parametrize("along", [True, False])
def test_quantize_past_32_bits(along):
    R_, K = (530000, 8192) if along else (8192, 530000)
    x = torch.zeros((R_, K) if along else (K, R_), dtype=torch.bfloat16, device="cuda")
    x[-128:] = torch.randn((128, x.shape[1]), device="cuda").to(torch.bfloat16)
    t = x if along else x.transpose(0, 1)
    q = tg.fp8_quantize(t)
    if along:
        codes, scales = R.quantise(_np(x[-2:]), 1)
        assert np.array_equal(_codes(q.codes[-2:]), codes) and np.array_equal(q.scales[-2:].cpu().numpy(), scales)
    else:
        # the last 80 of 530000 columns, in their own chunk, and the one before
        codes, scales = R.quantise(_np(t[-3:, -80:]), 1)
        assert K % 128 == 80 and np.array_equal(_codes(q.codes[-3:, -128:]), codes)
        assert np.array_equal(q.scales[-3:, -1:].cpu().numpy(), scales)
    assert not bool(q.codes[:1000].view(torch.uint8)[:, :128].any())


def test_every_entry_point_takes_nothing():
    q = tg.fp8_quantize(torch.empty((0, 64), device="cuda"))
    assert q.codes.shape == (0, 128) and q.scales.shape == (0, 1)
    W = tg.fp8_quantize(torch.ones((32, 64), device="cuda"), 128)
    assert tg.gemm_fp8(q, W).shape == (0, 32)
    Ws = tg.fp8_quantize(torch.ones((5, 32, 64), device="cuda"), 128)
    order = tg.moe_sort(torch.empty((0, 2), dtype=torch.int32, device="cuda"), 5)
    assert tg.moe_gemm_fp8(q, Ws, order.offsets).shape == (0, 32)
    x = torch.empty((0, 64), device="cuda")
    assert tg.moe_gather(x, order).shape == (0, 64) and tg.moe_gather(q, order).codes.shape == (0, 128)
    w = torch.empty((0, 2), device="cuda")
    assert tg.moe_combine(x, order, w).shape == (0, 64)
    dx, dw = tg.moe_combine_grad(x, x, order, w)
    assert dx.shape == (0, 64) and dw.shape == (0, 2)
    # tokens whose choices are all elsewhere, and no rows at all
    none = tg.MoeOrder(torch.full((3, 2), -1, dtype=torch.int32, device="cuda"), order.source, order.offsets)
    assert bool((tg.moe_combine(x, none) == 0).all())
    dx, dw = tg.moe_combine_grad(torch.ones((3, 64), device="cuda"), x, none, torch.ones((3, 2), device="cuda"))
    assert bool((dw == 0).all())


def test_refusals_on_the_gpu_leave_the_output():
    A = tg.fp8_quantize(torch.ones((4, 200), device="cuda"))
    B = tg.fp8_quantize(torch.ones((32, 200), device="cuda"), 128)
    out = torch.full((4, 32), 9.0, device="cuda")
    for a, b in ((B, B), (A._replace(K=300), B), (A, A._replace(K=100)), (A, B._replace(scales=B.scales.cpu())),
                 (A._replace(codes=A.codes.view(torch.uint8)), B), (A, B._replace(block=1))):
        with pytest.raises((ValueError, TypeError)):
            tg.gemm_fp8(a, b, out=out)
    for kw in (dict(bias=torch.zeros(31, device="cuda")), dict(act="tanh"), dict(act=7)):
        with pytest.raises((ValueError, KeyError, tg.TileGemmError)):
            tg.gemm_fp8(A, B, out=out, **kw)
    with pytest.raises(ValueError):
        tg.gemm_fp8(A, B, out=out[:3])
    with pytest.raises(ValueError):
        tg.moe_gemm_fp8(A, B, torch.zeros(5, dtype=torch.int32, device="cuda"), out=out)
    with pytest.raises(tg.TileGemmError):
        tg.moe_sort(torch.zeros((2, 1), dtype=torch.int32, device="cuda"), 1025)
    with pytest.raises(ValueError):
        tg.fp8_quantize(torch.zeros((64, 32), device="cuda")[::2])
    order = tg.moe_sort(torch.zeros((4, 1), dtype=torch.int32, device="cuda"), 2)
    x = torch.ones((5, 32), device="cuda")
    with pytest.raises(ValueError):
        tg.moe_gather(x, order, out=out)
    with pytest.raises(ValueError):
        tg.moe_combine_grad(x, out, order, torch.ones((4, 1), device="cuda"))
    assert bool((out == 9.0).all())
