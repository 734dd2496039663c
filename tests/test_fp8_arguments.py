"""What the products of 8-bit matrices and the sorted experts refuse beside tests/test_oracle_fp8.py (no GPU)."""
import pytest

from tile_shape_autotuning_amd import _native as N

BUF = 1 << 20                                          # a plausible, aligned address that nothing reads


def _f8(block=1):
    return N.F8Matrix(BUF, BUF, block, 0)


def _gemm(dtype, M=1):
    return N.gemm_fp8_ptr(M, 16, 128, _f8(), _f8(128), None, BUF, dtype, 0, None, 0)


def _experts(dtype, rows=1):
    return N.moe_gemm_fp8_ptr(rows, 4, 16, 128, _f8(), _f8(128), BUF, BUF, dtype)


@pytest.mark.parametrize("call", [_gemm, _experts])
def test_fast_sums_are_a_part_of_the_type(call):
    for dtype in (N.F32, 3, N.F32 | N.FAST_SUMS, 3 | N.FAST_SUMS, N.FAST_SUMS << 1 | N.BF16, -1, N.BF16 - N.FAST_SUMS):
        assert call(dtype) == N.TG_E_INVAL and "C is bf16" in N.last_error()
    for dtype in (N.BF16, N.BF16_F32OUT):
        assert call(dtype, 0) == N.TG_OK and call(dtype | N.FAST_SUMS, 0) == N.TG_OK


def test_gradients_of_a_sum_without_weights_are_refused_by_name():
    torch = pytest.importorskip("torch")
    import tile_shape_autotuning_amd as tg
    x, ids = torch.zeros((2, 64)), torch.zeros((2, 1), dtype=torch.int32)
    order = tg.MoeOrder(ids, ids[:, 0], torch.zeros(5, dtype=torch.int32))
    with pytest.raises(TypeError, match="moe_gather"):
        tg.moe_combine_grad(x, x, order, None)
