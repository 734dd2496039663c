"""The oracle of 4-bit weights and expert layers against closed forms, and the
refusals of the C ABI that need no GPU (a call with a bad argument is refused
before the library looks for a device)."""
import ctypes

import numpy as np
import pytest

from oracle import experts_ref as R
from tile_shape_autotuning_amd import _native as N


@pytest.mark.parametrize("K,n", [(1, 1), (128, 16), (130, 17), (300, 5)])
def test_pack_and_unpack_are_inverse(K, n):
    codes = np.random.default_rng(K).integers(0, 16, (K, n))
    assert np.array_equal(R.unpack(R.pack(codes), K, n), codes)


def test_the_words_of_one_element():
    codes = np.zeros((256, 32), np.int64)
    codes[128 + 64 + 16 + 5, 16 + 3] = 9             # chunk 1, step 2, lane group 2, row 5 of eight
    words = R.pack(codes)
    assert words[1, 1, 2 * 16 + 3, 2] == 9 << (4 * (2 + 4)) and np.count_nonzero(words) == 1


def test_quantisation_closed_forms():
    W = np.outer(np.arange(-7, 8), [1.0, 0.25])      # exactly the symmetric grid
    codes, s, z, v = R.quantize(W, 32, False, True)
    assert np.array_equal(v, W) and np.array_equal(s[0], [1.0, 0.25]) and np.all(z == 8)
    W = np.arange(0, 16, dtype=float)[:, None] - 5.0
    codes, s, z, v = R.quantize(W, 32, True, False)
    assert np.array_equal(codes[:, 0], np.arange(16)) and z[0, 0] == 5 and np.array_equal(v, W)
    # quotients in the middle go to the even neighbour, groups are independent, a zero group stays zero
    W = np.zeros((96, 1))
    W[:4, 0] = [7.0, 0.5, 1.5, -2.5]
    W[32, 0] = -14.0
    codes, s, z, v = R.quantize(W, 32, False, False)
    assert list(v[:4, 0]) == [7.0, 0.0, 2.0, -2.0] and list(s[:, 0]) == [1.0, 2.0, 0.0] and np.all(codes[64:] == 8)


def test_routing_closed_forms():
    ids, w = R.route([[0.0, np.log(3.0), 0.0, np.log(4.0)]], 2, False)
    assert ids.tolist() == [[3, 1]] and np.allclose(w, [[4 / 9, 3 / 9]])
    ids, w = R.route([[1.0, 1.0, 1.0]], 2, True)
    assert ids.tolist() == [[0, 1]] and np.allclose(w, 0.5)
    ids, w = R.route([[-np.inf, -np.inf]], 1, True)
    assert ids.tolist() == [[0]] and w[0, 0] == 0.0


def test_mlp_closed_form():
    # one-hot rows: expert e maps x = c one_hot(0) to silu(c g) (c u) d in column 1
    gate, up, down = np.zeros((2, 2, 1)), np.zeros((2, 2, 1)), np.zeros((2, 1, 2))
    gate[:, 0, 0], up[:, 0, 0], down[:, 0, 1] = [1.0, 2.0], [3.0, 5.0], [7.0, 11.0]
    x = np.array([[2.0, 0.0]])
    y, _ = R.mlp(x, np.array([[1, 0, -1, 2]]), np.array([[0.5, 0.25, 9.0, 9.0]]), gate, up, down, "silu")
    silu = lambda v: v / (1 + np.exp(-v))            # noqa: E731
    assert np.allclose(y, [[0.0, 0.5 * silu(4.0) * 10.0 * 11.0 + 0.25 * silu(2.0) * 6.0 * 7.0]])


# ---------------------------------------------------------------- refusals: no GPU is touched
BUF = 1 << 20                                          # a plausible, aligned address that nothing reads


def _w4(group=128, scale=N.BF16, data=BUF, scales=BUF, fmt=N.W_W4):
    return N.Weight(fmt, group, scale, 0, data, scales, None)


def _quantize(**kw):
    a = dict(count=1, K=128, N=16, group=128, W=BUF, dtype=N.BF16, rows=True, scale=N.BF16, words=BUF, scales=BUF,
             zeros=None, values=None)
    a.update(kw)
    return N.w4_quantize_ptr(*a.values())


@pytest.mark.parametrize("kw", [dict(count=-1), dict(K=0), dict(N=0), dict(group=96), dict(group=16), dict(group=0),
                                dict(dtype=2), dict(scale=2), dict(W=None), dict(words=None), dict(words=BUF + 4),
                                dict(scales=None), dict(W=BUF + 1), dict(values=BUF + 1)])
def test_quantize_refuses(kw):
    assert _quantize(**kw) == N.TG_E_INVAL and N.last_error()


def test_quantize_limits():
    assert _quantize(K=(1 << 21) + 1) == N.TG_E_UNSUPPORTED
    assert _quantize(count=65536) == N.TG_E_UNSUPPORTED
    assert _quantize(count=0, words=None, scales=None, W=None) == N.TG_OK


def _gemm(**kw):
    a = dict(M=1, N=16, K=128, A=BUF, w=_w4(), bias=None, C=BUF, dtype=N.BF16, act=0)
    a.update(kw)
    return N.gemm_w4_ptr(*a.values())


@pytest.mark.parametrize("kw", [dict(M=-1), dict(N=-1), dict(K=0), dict(A=None), dict(C=None), dict(A=BUF + 1),
                                dict(C=BUF + 1), dict(C=BUF + 2, dtype=N.BF16_F32OUT), dict(bias=BUF + 2),
                                dict(dtype=N.F32), dict(act=3), dict(act=-1), dict(w=None), dict(w=_w4(group=48)),
                                dict(w=_w4(scale=2)), dict(w=_w4(data=None)), dict(w=_w4(data=BUF + 8)),
                                dict(w=_w4(scales=None)), dict(w=_w4(fmt=N.W_BF16)), dict(w=_w4(fmt=7))])
def test_gemm_w4_refuses(kw):
    assert _gemm(**kw) == N.TG_E_INVAL and N.last_error()


def test_gemm_w4_limits_and_empty():
    assert _gemm(K=(1 << 21) + 1) == N.TG_E_UNSUPPORTED
    assert _gemm(M=(1 << 20) + 1) == N.TG_E_UNSUPPORTED
    assert _gemm(M=0, A=None, C=None) == N.TG_OK and _gemm(N=0) == N.TG_OK


def _route(**kw):
    a = dict(T=1, E=8, k=2, logits=BUF, dtype=N.F32, renorm=True, ids=BUF, weights=BUF)
    a.update(kw)
    return N.moe_route_ptr(*a.values())


@pytest.mark.parametrize("kw", [dict(T=-1), dict(E=0), dict(k=0), dict(k=9), dict(logits=None), dict(ids=None),
                                dict(weights=None), dict(dtype=2), dict(logits=BUF + 2), dict(ids=BUF + 2)])
def test_route_refuses(kw):
    assert _route(**kw) == N.TG_E_INVAL and N.last_error()


def test_route_limits_and_empty():
    assert _route(E=1025) == N.TG_E_UNSUPPORTED and _route(E=64, k=17) == N.TG_E_UNSUPPORTED
    assert _route(T=(1 << 24) + 1) == N.TG_E_UNSUPPORTED
    assert _route(T=0, logits=None) == N.TG_OK


def _mlp(layer=False, **kw):
    a = dict(T=1, H=64, I=64, E=8, k=2, x=BUF, ids=BUF, weights=BUF, up=_w4(), down=_w4(), y=BUF, gate=0, ws=BUF,
             ws_bytes=1 << 16, logits=BUF)
    a.update(kw)
    if layer:
        return N.moe_layer_ptr(a["T"], a["H"], a["I"], a["E"], a["k"], a["x"], a["logits"], N.F32, True, a["up"],
                               a["down"], a["y"], a["ids"], a["weights"], a["gate"], a["ws"], a["ws_bytes"])
    a.pop("logits")
    return N.moe_mlp_ptr(*a.values())


@pytest.mark.parametrize("layer", [False, True])
@pytest.mark.parametrize("kw", [dict(T=-1), dict(H=0), dict(I=0), dict(E=0), dict(k=0), dict(k=9), dict(x=None),
                                dict(x=BUF + 1), dict(y=None), dict(ids=None), dict(weights=BUF + 2), dict(gate=2),
                                dict(up=None), dict(down=_w4(group=40)), dict(down=_w4(data=BUF + 2, fmt=N.W_BF16)),
                                dict(ws=None), dict(ws=BUF + 8), dict(ws_bytes=2 * 128 * 4 - 1)])
def test_mlp_refuses(layer, kw):
    assert _mlp(layer, **kw) == N.TG_E_INVAL and N.last_error()


@pytest.mark.parametrize("layer", [False, True])
def test_mlp_limits_and_empty(layer):
    for kw in (dict(H=65537), dict(I=65537), dict(E=1025), dict(E=64, k=17)):
        assert _mlp(layer, **kw) == N.TG_E_UNSUPPORTED
    assert _mlp(layer, T=0, x=None, y=None, ws=None) == N.TG_OK


def test_workspace_is_for_one_pass_of_tokens():
    assert N.moe_workspace_bytes(3, 10, 17, 4) == 3 * 4 * (32 + 10) * 4
    assert N.moe_workspace_bytes(1000, 10, 17, 4) == N.moe_workspace_bytes(64, 10, 17, 4)
    n = ctypes.c_size_t()
    assert N.lib().tg_moe_workspace_bytes(1, 1, 0, 1, ctypes.byref(n)) == N.TG_E_INVAL
    assert N.lib().tg_moe_workspace_bytes(1, 1, 1, 1, None) == N.TG_E_INVAL


def test_python_refuses_cpu_tensors_and_shapes():
    torch = pytest.importorskip("torch")
    import tile_shape_autotuning_amd as tg
    A = torch.zeros((2, 64), dtype=torch.bfloat16)
    w = tg.W4(torch.zeros((1, 1, 64, 4), dtype=torch.int32), torch.zeros((1, 1, 16)), None, 64, 16, 64)
    with pytest.raises(ValueError):
        tg.gemm_w4(A, w)
    with pytest.raises(ValueError):
        tg.w4_quantize(A)
    with pytest.raises(ValueError):
        tg.moe_route(torch.zeros((2, 4)), 2)
    with pytest.raises(TypeError):
        tg.moe_route(torch.zeros((2, 4), dtype=torch.float64), 2)
    ids, wt = torch.zeros((2, 1), dtype=torch.int32), torch.zeros((2, 1))
    with pytest.raises(ValueError):
        tg.moe_mlp(A, ids, wt, w, w)
    with pytest.raises(TypeError):
        tg.moe_mlp(A, ids.long(), wt, w, w)
