"""What is not a number in 8-bit matrices stays not a number in the products' own rows and columns, whatever the kernel,
the type of the result, the activation and the way of adding up."""
import numpy as np
import pytest

from gpu_util import mark

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
tg = pytest.importorskip("tile_shape_autotuning_amd")

E4M3 = torch.float8_e4m3fn
TYPES = (torch.bfloat16, torch.float32)


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _matrix(R_, K, block, lead=()):
    """Random finite elements as an F8."""
    return tg.fp8_quantize(torch.randn((*lead, R_, K), device="cuda"), block)


def _with(q, code=None, scale=None):
    """q with a code and a scale (their indices) that are NaN."""
    codes, scales = q.codes.view(torch.uint8).clone(), q.scales.clone()
    if code is not None:
        codes[code] = 0xFF
    if scale is not None:
        scales[scale] = float("nan")
    return q._replace(codes=codes.view(E4M3), scales=scales)


def _apply(v, act):
    # an fp32 result without an activation, as elementary operations that keep a NaN
    if act == "relu":
        return torch.where(v <= 0, torch.zeros_like(v), v)
    return v


# a few rows, tiles of each height, reductions in parts
SHAPES = [(4, 150, 384), (64, 300, 260), (65, 150, 384), (200, 300, 260), (100, 300, 9000), (300, 1100, 1400),
          (2050, 4200, 260), (1500, 5000, 130)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("fast", [False, True])
def test_products_keep_what_is_not_a_number(M, N, K, block, fast):
    torch.manual_seed(M)
    A, B = _matrix(M, K, 1), _matrix(N, K, block)
    last = (N - 1) // block                            # the last row of scales
    a = _with(A, (2, 5), (M - 1, (K - 1) // 128))
    b = _with(B, (N // 3, K - 1), (last, 0))
    bad = torch.zeros((M, N), dtype=torch.bool, device="cuda")
    bad[2], bad[M - 1], bad[:, N // 3], bad[:, last * block:] = True, True, True, True
    mark(f"gemm_fp8 NaN {M}x{N}x{K} block {block} fast {fast}")
    for dt in TYPES:
        plain = tg.gemm_fp8(A, B, out_dtype=dt, fast_sums=fast)
        for act in ("none", "relu", "gelu"):
            C = tg.gemm_fp8(a, b, act=act, out_dtype=dt, fast_sums=fast)
            assert torch.equal(torch.isnan(C), bad), (dt, act)
            if act != "gelu":
                assert torch.equal(C[~bad], _apply(plain, act)[~bad]), (dt, act)
        # a bias that is not a number has its column only
        bias = torch.zeros(N, device="cuda")
        bias[N - 2] = float("nan")
        C = tg.gemm_fp8(A, B, bias, act="relu", out_dtype=dt, fast_sums=fast)
        assert bool(torch.isnan(C[:, N - 2]).all()) and int(torch.isnan(C).sum()) == M


@pytest.mark.parametrize("n,N", [(12, 150), (90, 300), (700, 300), (2500, 1100)])
@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("fast", [False, True])
def test_products_of_experts_keep_what_is_not_a_number(n, N, block, fast):
    torch.manual_seed(n)
    A, B = _matrix(n, 300, 1), _matrix(N, 300, block, (3,))
    offsets = torch.tensor([0, n // 3, n // 2, n], dtype=torch.int32, device="cuda")
    last = (N - 1) // block
    a = _with(A, (2, 5), (n - 1, 2))
    b = _with(B, (0, N // 3, 299), (1, last, 0))       # of the first and the second expert, none of the third
    bad = torch.zeros((n, N), dtype=torch.bool, device="cuda")
    bad[2], bad[n - 1], bad[:n // 3, N // 3], bad[n // 3:n // 2, last * block:] = True, True, True, True
    mark(f"moe_gemm_fp8 NaN {n}x{N} block {block} fast {fast}")
    for dt in TYPES:
        plain = tg.moe_gemm_fp8(A, B, offsets, out_dtype=dt, fast_sums=fast)
        C = tg.moe_gemm_fp8(a, b, offsets, out_dtype=dt, fast_sums=fast)
        assert torch.equal(torch.isnan(C), bad) and torch.equal(C[~bad], plain[~bad]), dt


@pytest.mark.parametrize("M", [3, 130])
def test_an_infinite_activation_is_seen_behind_a_relu(M):
    x = torch.ones((M, 200), device="cuda")
    x[1, 7] = float("inf")
    W = tg.fp8_quantize(torch.ones((40, 200), device="cuda"), 128)
    for dt in TYPES:
        C = tg.gemm_fp8(tg.fp8_quantize(x), W, act="relu", out_dtype=dt)
        assert bool(torch.isnan(C[1]).all()) and int(torch.isnan(C).sum()) == 40


def test_relu_gives_no_negative_zeros():
    A = tg.fp8_quantize(-torch.ones((2, 128), device="cuda"))
    A = A._replace(scales=A.scales * 2.0 ** -75)
    B = tg.fp8_quantize(torch.ones((20, 128), device="cuda"))
    B = B._replace(scales=B.scales * 2.0 ** -75)       # the scales' product underflows: sums of -0
    for m in (2, 130):
        q = A._replace(codes=A.codes.view(torch.uint8)[:1].expand(m, 128).contiguous().view(E4M3),
                       scales=A.scales[:1].expand(m, 1).contiguous())
        C = tg.gemm_fp8(q, B, act="relu", out_dtype=torch.float32)
        assert bool((C == 0).all()) and not bool(torch.signbit(C).any())
