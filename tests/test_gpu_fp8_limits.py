"""Products of 8-bit matrices at and past the limits that the header states."""
import pytest

from gpu_util import mark

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
tg = pytest.importorskip("tile_shape_autotuning_amd")


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()


def _zeros(lead, R_, block):
    codes = torch.zeros((*lead, R_, 128), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    return tg.F8(codes, torch.ones((*lead, -(-R_ // block), 1), device="cuda"), 128, block)


def test_more_workgroups_than_a_launch_has_are_refused():
    E, most = 1024, 2 ** 22
    A = _zeros((), E, 1)
    offsets = torch.arange(E + 1, dtype=torch.int32, device="cuda")
    columns = most // (E // 16 + E) * 64               # as many as always fit
    mark(f"moe_gemm_fp8 {E} rows {E} experts {columns}x128")
    C = tg.moe_gemm_fp8(A, _zeros((E,), columns, 128), offsets)
    assert not bool(C.any())
    del C
    # and what does not, before anything is written
    out = torch.full((E, columns + 64), 9.0, dtype=torch.bfloat16, device="cuda")
    B = _zeros((E,), columns + 64, 128)
    with pytest.raises(tg.TileGemmError, match="too many tiles"):
        tg.moe_gemm_fp8(A, B, offsets, out=out)
    assert bool((out == 9.0).all())


def test_gemm_of_as_many_results_as_always_fit():
    M, N = 2 ** 24, 4096                               # 128 GiB of results, none of which an earlier call left
    if torch.cuda.mem_get_info()[0] < 1.1 * 2 * M * N:
        pytest.skip("other programs hold the card's memory")
    A, B = _zeros((), M, 1), _zeros((), N, 128)
    mark(f"gemm_fp8 {M}x{N}x128")
    C = tg.gemm_fp8(A, B, torch.ones(N, device="cuda"))
    assert all(bool((part == 1).all()) for part in C.view(64, -1, N)), "every result is written"
