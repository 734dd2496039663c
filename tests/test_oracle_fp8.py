"""The oracle of 8-bit matrices and sorted experts against closed forms, and what the C ABI refuses (no GPU)."""
import ctypes

import numpy as np
import pytest

from oracle import fp8_ref as R
from tile_shape_autotuning_amd import _native as N


# ---------------------------------------------------------------- oracle
def test_the_codes_values():
    assert R.code_value(0x7E) == 448.0 and R.code_value(0x01) == 2.0 ** -9 and R.code_value(0x08) == 2.0 ** -6
    assert R.code_value(0x38) == 1.0 and R.code_value(0xB9) == -1.125 and np.isnan(R.code_value(0x7F))
    assert (np.diff(R.VALUES[:127]) > 0).all() and R.VALUES[0] == 0.0


def test_the_codes_agree_with_torch():
    torch = pytest.importorskip("torch")
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(t, R.VALUES, equal_nan=True)


def test_nearest_rounds_ties_to_even_and_saturates():
    finite = np.r_[0:127, 128:255]
    assert np.array_equal(R.nearest(R.VALUES[finite]), finite)
    mids = (R.VALUES[1:127] + R.VALUES[:126]) / 2
    lower = np.arange(126)
    assert np.array_equal(R.nearest(mids), np.where(lower % 2 == 0, lower, lower + 1))
    assert np.array_equal(R.nearest(mids * (1 - 2.0 ** -40)), lower)
    assert np.array_equal(R.nearest(-mids * (1 + 2.0 ** -40)), lower + 1 + 128)
    assert R.nearest(1e9) == 0x7E and R.nearest(-449.0) == 0xFE


def test_quantise_keeps_what_it_can_hold():
    x = np.zeros((3, 130))
    x[0, :4] = [448.0, -1.5, 2.0 ** -9, 2.0 ** -12]
    x[1, 129] = 7.0
    codes, s = R.quantise(x, 1)
    assert codes.shape == (3, 256) and s.shape == (3, 2) and s[0, 0] == 1.0 and s[1, 1] == np.float32(7 / 448)
    assert np.array_equal(R.dense(codes, s, 130, 1)[0, :3], x[0, :3]) and codes[0, 3] == 0
    assert not codes[2].any() and not s[2].any() and not codes[:, 130:].any()
    codes, s = R.quantise(x, 128)
    assert s.shape == (1, 2) and s[0, 0] == 1.0


def test_quantise_marks_blocks_that_are_not_finite():
    x = np.ones((2, 200))
    x[1, 3] = np.inf
    codes, s = R.quantise(x, 1)
    assert np.isnan(s[1, 0]) and (codes[1, :128] == 0x7F).all() and np.isfinite(s[0]).all() and s[1, 1] > 0


def test_order_sorts_and_inverts():
    ids = np.array([[2, 0], [-1, 2], [0, 5], [2, 2]], np.int32)
    position, source, offsets = R.order(ids, 3)
    assert offsets.tolist() == [0, 2, 2, 6]
    assert position.tolist() == [[2, 0], [-1, 3], [1, -1], [4, 5]]
    assert source.tolist() == [1, 4, 0, 3, 6, 7, -1, -1]


def test_combine_and_its_gradient_agree_with_differences():
    rng = np.random.default_rng(0)
    position = np.array([[1, 3], [-1, 0], [2, 7]], np.int32)
    x, w, dy = rng.standard_normal((4, 5)), rng.standard_normal((3, 2)), rng.standard_normal((3, 5))
    dx, dw = R.combine_grad(dy, x, position, w, np.zeros_like(x))
    h = 1e-6
    # the sum is linear in each of its inputs: differences are exact but for rounding
    for (i, j) in np.ndindex(x.shape):
        d = np.zeros_like(x)
        d[i, j] = h
        diff = np.sum(dy * (R.combine(x + d, position, w) - R.combine(x - d, position, w))) / (2 * h)
        assert abs(diff - dx[i, j]) < 1e-8
    for (i, j) in np.ndindex(w.shape):
        d = np.zeros_like(w)
        d[i, j] = h
        diff = np.sum(dy * (R.combine(x, position, w + d) - R.combine(x, position, w - d))) / (2 * h)
        assert abs(diff - dw[i, j]) < 1e-8
    # and the gradient of gathering is the combination without weights
    full = np.array([[1, 3], [2, 0]], np.int32)
    t, g = rng.standard_normal((2, 5)), rng.standard_normal((4, 5))
    rows = R.gather(t, full, np.zeros((4, 5)))
    assert np.isclose(np.sum(g * rows), np.sum(R.combine(g, full, np.ones((2, 2))) * t))


# ---------------------------------------------------------------- refusals: no GPU is touched
BUF = 1 << 20                                          # a plausible, aligned address that nothing reads
BIG = (1 << 24) + 1


def _f8(codes=BUF, scales=BUF, block=1):
    return N.F8Matrix(codes, scales, block, 0)


def _quantize(**kw):
    a = dict(count=1, R=16, K=128, block=1, x=BUF, dtype=N.BF16, rows=True, codes=BUF, scales=BUF, values=None)
    a.update(kw)
    return N.fp8_quantize_ptr(*a.values())


@pytest.mark.parametrize("kw", [dict(count=-1), dict(R=-1), dict(K=0), dict(block=2), dict(block=0), dict(dtype=2),
                                dict(x=None), dict(codes=None), dict(codes=BUF + 8), dict(scales=None),
                                dict(scales=BUF + 2), dict(x=BUF + 1), dict(x=BUF + 2, dtype=N.F32),
                                dict(values=BUF + 1)])
def test_quantize_refuses(kw):
    assert _quantize(**kw) == N.TG_E_INVAL and N.last_error()


def test_quantize_limits_and_empty():
    for kw in (dict(R=BIG), dict(K=BIG), dict(count=65536), dict(R=1 << 20, K=1 << 20)):
        assert _quantize(**kw) == N.TG_E_UNSUPPORTED
    assert _quantize(count=0, x=None) == N.TG_OK and _quantize(R=0, x=None, codes=None) == N.TG_OK


def _gemm(**kw):
    a = dict(M=1, N=16, K=128, A=_f8(), B=_f8(block=128), bias=None, C=BUF, dtype=N.BF16, act=0, ws=BUF,
             ws_bytes=1 << 40)
    a.update(kw)
    return N.gemm_fp8_ptr(*a.values())


def _experts(**kw):
    a = dict(rows=1, E=4, N=16, K=128, A=_f8(), B=_f8(block=128), offsets=BUF, C=BUF, dtype=N.BF16)
    a.update(kw)
    return N.moe_gemm_fp8_ptr(*a.values())


BAD = [dict(N=-1), dict(K=0), dict(dtype=N.F32), dict(dtype=3), dict(A=None), dict(B=None), dict(A=_f8(block=128)),
       dict(A=_f8(codes=None)), dict(A=_f8(codes=BUF + 8)), dict(A=_f8(scales=BUF + 2)), dict(B=_f8(scales=None)),
       dict(B=_f8(block=64)), dict(B=_f8(codes=BUF + 4)), dict(C=None), dict(C=BUF + 1),
       dict(C=BUF + 2, dtype=N.BF16_F32OUT)]


@pytest.mark.parametrize("kw", BAD + [dict(M=-1), dict(act=3), dict(act=-1), dict(bias=BUF + 2)])
def test_gemm_refuses(kw):
    assert _gemm(**kw) == N.TG_E_INVAL and N.last_error()


@pytest.mark.parametrize("kw", BAD + [dict(rows=-1), dict(E=0), dict(offsets=None), dict(offsets=BUF + 2)])
def test_expert_products_refuse(kw):
    assert _experts(**kw) == N.TG_E_INVAL and N.last_error()


def test_product_limits_and_empty():
    for kw in (dict(M=BIG), dict(N=BIG), dict(K=(1 << 22) + 1)):
        assert _gemm(**kw) == N.TG_E_UNSUPPORTED
    for kw in (dict(rows=BIG), dict(N=BIG), dict(K=(1 << 22) + 1), dict(E=1025)):
        assert _experts(**kw) == N.TG_E_UNSUPPORTED
    assert _gemm(M=0, A=None, C=None) == N.TG_OK and _gemm(N=0, B=None) == N.TG_OK
    assert _experts(rows=0, A=None, C=None) == N.TG_OK and _experts(N=0, B=None) == N.TG_OK
    n = ctypes.c_size_t()
    assert N.lib().tg_gemm_fp8_workspace_bytes(1, 1, 0, ctypes.byref(n)) == N.TG_E_INVAL
    assert N.lib().tg_gemm_fp8_workspace_bytes(1, 1, BIG, ctypes.byref(n)) == N.TG_E_INVAL
    assert N.lib().tg_gemm_fp8_workspace_bytes(1, 1, 1, None) == N.TG_E_INVAL


def _sort(**kw):
    a = dict(T=4, E=8, k=2, ids=BUF, position=BUF, source=BUF, offsets=BUF, ws=BUF, ws_bytes=1 << 40)
    a.update(kw)
    return N.moe_sort_ptr(*a.values())


@pytest.mark.parametrize("kw", [dict(T=-1), dict(E=0), dict(k=0), dict(ids=None), dict(position=None),
                                dict(source=None), dict(offsets=None), dict(ids=BUF + 2), dict(offsets=BUF + 1)])
def test_sort_refuses(kw):
    assert _sort(**kw) == N.TG_E_INVAL and N.last_error()


def test_sort_limits():
    # many pairs: counts of blocks of experts, in the workspace
    need = N.moe_sort_workspace_bytes(4096, 64, 8)
    assert need > 0 and N.moe_sort_workspace_bytes(16, 64, 8) == 0 and N.moe_sort_workspace_bytes(0, 1, 1) == 0
    for kw in (dict(ws=None), dict(ws=BUF + 8), dict(ws_bytes=need - 1)):
        assert _sort(T=4096, E=64, k=8, **kw) == N.TG_E_INVAL
    for kw in (dict(T=BIG), dict(E=1025), dict(k=17)):
        assert _sort(**kw) == N.TG_E_UNSUPPORTED
    n = ctypes.c_size_t()
    assert N.lib().tg_moe_sort_workspace_bytes(-1, 1, 1, ctypes.byref(n)) == N.TG_E_INVAL
    assert N.lib().tg_moe_sort_workspace_bytes(1, 1, 1, None) == N.TG_E_INVAL


def _gather(**kw):
    a = dict(T=4, k=2, rows=8, position=BUF, bytes=16, x=BUF, out=BUF, bytes2=0, x2=None, out2=None)
    a.update(kw)
    return N.moe_gather_ptr(*a.values())


def _combine(**kw):
    a = dict(T=4, k=2, rows=8, H=16, x=BUF, dtype=N.BF16, position=BUF, weights=None, y=BUF)
    a.update(kw)
    return N.moe_combine_ptr(*a.values())


def _grad(**kw):
    a = dict(T=4, k=2, rows=8, H=16, dy=BUF, x=BUF, dtype=N.BF16, position=BUF, weights=BUF, dx=BUF, dw=BUF)
    a.update(kw)
    return N.moe_combine_grad_ptr(*a.values())


ROWS = [dict(T=-1), dict(k=0), dict(rows=-1), dict(position=None), dict(position=BUF + 2), dict(x=None)]


@pytest.mark.parametrize("kw", ROWS + [dict(bytes=0), dict(bytes2=-1), dict(out=None), dict(bytes2=4),
                                       dict(bytes2=4, x2=BUF)])
def test_gather_refuses(kw):
    assert _gather(**kw) == N.TG_E_INVAL and N.last_error()


@pytest.mark.parametrize("kw", ROWS + [dict(H=0), dict(dtype=2), dict(y=None), dict(y=BUF + 1), dict(x=BUF + 1),
                                       dict(x=BUF + 2, dtype=N.F32), dict(weights=BUF + 2)])
def test_combine_refuses(kw):
    assert _combine(**kw) == N.TG_E_INVAL and N.last_error()


@pytest.mark.parametrize("kw", ROWS + [dict(H=0), dict(dtype=2), dict(dy=None), dict(dx=None), dict(dw=None),
                                       dict(weights=None), dict(dw=BUF + 2), dict(dx=BUF + 1),
                                       dict(dy=BUF + 2, dtype=N.F32)])
def test_combine_grad_refuses(kw):
    assert _grad(**kw) == N.TG_E_INVAL and N.last_error()


@pytest.mark.parametrize("call", [_gather, _combine, _grad])
def test_row_limits_and_empty(call):
    for kw in (dict(T=BIG), dict(k=17), dict(rows=1 << 31)):
        assert call(**kw) == N.TG_E_UNSUPPORTED
    wide = [dict(bytes=BIG), dict(bytes2=BIG)] if call is _gather else [dict(H=BIG)]
    for kw in wide:
        assert call(**kw) == N.TG_E_UNSUPPORTED
    assert call(T=0, position=None, x=None) == N.TG_OK


# ---------------------------------------------------------------- what the binding refuses
def test_python_refuses_cpu_tensors_types_and_shapes():
    torch = pytest.importorskip("torch")
    import tile_shape_autotuning_amd as tg
    bf = torch.zeros((2, 64), dtype=torch.bfloat16)
    for call in (lambda: tg.fp8_quantize(bf), lambda: tg.fp8_quantize(bf, 64), lambda: tg.fp8_quantize(bf[0])):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        tg.fp8_quantize(bf.double())
    f8 = tg.F8(torch.zeros((2, 128)).to(torch.float8_e4m3fn), torch.zeros((2, 1)), 64, 1)
    with pytest.raises(ValueError, match="GPU"):
        tg.gemm_fp8(f8, f8)
    for bad in (None, bf, (1, 2, 3)):
        with pytest.raises(TypeError, match="A must be an F8"):
            tg.gemm_fp8(bad, f8)
    for kw, word in ((dict(block=128), "block"), (dict(block=2), "block"), (dict(K=200), "codes"), (dict(K=0), "K"),
                     (dict(codes=torch.zeros((2, 128))), "codes"), (dict(scales=torch.zeros((2, 2))), "scales"),
                     (dict(scales=torch.zeros((2, 1), dtype=torch.float64)), "scales")):
        with pytest.raises(ValueError, match=word):
            tg.gemm_fp8(f8._replace(**kw), f8)
    ids = torch.zeros((2, 1), dtype=torch.int32)
    with pytest.raises(ValueError):
        tg.moe_sort(ids, 4)
    with pytest.raises(TypeError):
        tg.moe_sort(ids.long(), 4)
    order = tg.MoeOrder(ids, ids[:, 0], torch.zeros(5, dtype=torch.int32))
    with pytest.raises(ValueError):
        tg.moe_gather(bf, order)
    with pytest.raises(TypeError):
        tg.moe_gather(bf.double(), order)
    with pytest.raises(ValueError):
        tg.moe_combine(bf, order)
    with pytest.raises(TypeError):
        tg.moe_combine_grad(bf.half(), bf, order, torch.ones((2, 1)))
