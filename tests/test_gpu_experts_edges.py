"""4-bit weights and expert layers where they can go wrong: the hidden state's
precision, hot experts, rows near overflow, gates far from zero, groups that
are not finite.  The fp64 oracle and the helpers are those of test_gpu_experts.
"""
import numpy as np
import pytest

from oracle import experts_ref as R

from gpu_util import mark
from test_gpu_experts import _bf16, _choices, _cuda, _experts, _gpu, _np, _w4, tg, torch    # noqa: F401

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- the hidden state
def _lone_neurons(rng, T, E, I):
    """Integer experts of which one hidden neuron in 128 is not zero: x [T, 2], gate and up [E, 2, I, 2] and the
    neurons.  Gates are near 700 (gate(g) = g in fp32, SiLU and GELU), hidden values 700^2 - s^2, s <= 12: integers
    of 19 bits whose differences bf16 holds."""
    x = np.stack([np.full(T, 175.0), rng.integers(1, 4, T)], 1)
    up = np.zeros((E, 2, I, 2))
    at = np.array([c + int(rng.integers(min(128, I - c))) for c in range(0, I, 128)])
    up[:, 0, :, 0] = 4.0
    up[:, 0, :, 1] = rng.integers(-4, 5, (E, I))
    up[:, 1, at, 0] = 4.0
    up[:, 1, at, 1] = -up[:, 0, at, 1]
    return x, up, at


def _pair_columns(rng, E, I, H, at):
    """[E, I, H]: each column takes one of the neurons with 1, 2 or 3 and another with the opposite."""
    d = np.zeros((E, I, H))
    for e in range(E):
        for n in range(H):
            i, j = rng.choice(at, 2, replace=False)
            a = rng.integers(1, 4)
            d[e, i, n], d[e, j, n] = a, -a
    return d


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("kind,group,zero", [("bf16", 0, False), ("w4", 128, False), ("w4", 64, True),
                                             ("w4", 32, True)])
@pytest.mark.parametrize("T,E,I", [(3, 2, 520), (2, 2, 2600), (40, 2, 520), (40, 2, 1300), (40, 2, 2600), (3, 2, 301)])
def test_hidden_values_keep_24_bits(T, E, I, kind, group, zero, act):
    # h <= 700^2 < 2^24 / 31, alone in its chunk: every sum, the 4-bit product's constant parts (31 h, 24 h)
    # included, is an integer below 2^24 and exact in fp32, so y is the difference of two h, rounded once to bf16
    rng = np.random.default_rng(I + T + group)
    H = 48
    x, up, at = _lone_neurons(rng, T, E, I)
    d = _pair_columns(rng, E, I, H, at)
    x = np.concatenate([x, np.zeros((T, H - 2))], 1)
    up = np.concatenate([up, np.zeros((E, 2, I, H - 2))], 3)
    ids = np.tile(np.arange(E, dtype=np.int32), (T, 1))
    ids[:, 1] = -1                                     # one expert a token: its sums stand alone
    ids[::2, 0] = 1
    if T > 16:
        assert T * ids.shape[1] > 8 * E                # two row tiles
    w = np.ones(ids.shape, np.float32)
    if kind == "bf16":
        down = _bf16(d.transpose(0, 2, 1))
    else:
        P, G = -(-H // 16), -(-I // group)
        z = rng.integers(4, 12, (E, P, G, 16), dtype=np.uint8) if zero else None
        words = []
        for e in range(E):
            zk = np.full((I, H), 8) if z is None else \
                z[e].transpose(1, 0, 2).reshape(G, P * 16)[:, :H].repeat(group, 0)[:I].astype(int)
            words.append(R.pack(d[e].astype(int) + zk))
        down = tg.W4(_cuda(np.stack(words)), torch.ones((E, P, G, 16), device="cuda"), _cuda(z) if zero else None,
                     I, H, group)
    mark(f"hidden values T{T} E{E} I{I} {kind} g{group} {act}")
    y = tg.moe_mlp(_bf16(x), _cuda(ids), _cuda(w), _bf16(up), down, gate=act)
    torch.cuda.synchronize()
    h = np.einsum("th,eih->tei", x, up[:, 0]) * np.einsum("th,eih->tei", x, up[:, 1])
    ref = np.stack([h[t, ids[t, 0]] @ d[ids[t, 0]] for t in range(T)])
    assert np.abs(h).max() * 31 < 2 ** 24
    assert np.array_equal(_np(y), R.round_bf16(ref))


@pytest.mark.parametrize("kind", ["bf16", "w4"])
def test_infinite_hidden_values_stay_infinite(kind):
    # bf16 experts: an infinite hidden value meets the formula's infinities, and NaN only where it meets a zero weight
    x = torch.ones((3, 16), device="cuda", dtype=torch.bfloat16)
    x[1] = 3e38                                        # gate 3e38 * 16 overflows
    up = torch.ones((1, 2, 8, 16), device="cuda", dtype=torch.bfloat16)
    up[0, 1, 1:] = 0.0                                 # neuron 0 alone is infinite; 0 * inf gives NaN elsewhere
    up[0, 0, 1:] = 0.0
    down = torch.zeros((1, 16, 8), device="cuda", dtype=torch.bfloat16)
    down[0, :, 0] = torch.tensor([1.0, -2.0] * 8, device="cuda")
    if kind == "w4":
        with_codes = tg.w4_quantize(down.transpose(1, 2), 32)
        y = tg.moe_mlp(x, torch.zeros((3, 1), dtype=torch.int32, device="cuda"), torch.ones((3, 1), device="cuda"), up,
                       with_codes)
        assert bool(torch.isnan(y[1]).all()) and bool(torch.isfinite(y[[0, 2]]).all())
        return
    y = tg.moe_mlp(x, torch.zeros((3, 1), dtype=torch.int32, device="cuda"), torch.ones((3, 1), device="cuda"), up, down)
    inf = float("inf")
    assert y[1].tolist() == [inf, -inf] * 8 and bool(torch.isfinite(y[[0, 2]]).all())


@pytest.mark.parametrize("T,E,k,H,I,kind,group,zero", [(64, 8, 2, 512, 640, "bf16", 0, False),
                                                       (64, 8, 2, 512, 640, "w4", 64, True),
                                                       (48, 32, 4, 512, 2304, "w4", 128, False)])
def test_outputs_round_once(T, E, k, H, I, kind, group, zero):
    # How many bf16 outputs may differ from the rounded exact ones: a sum off by d is rounded otherwise with
    # probability d / step.  d in units of the root of the sum of the squares of its terms: at most 48 fp32
    # additions one after the other (three parts of 4 fragments, two chunks a wave, eight waves, k pairs), off by
    # 2^-24 on average where sums are truncated, of partial sums up to the root (4 bits: the constant parts'
    # 24 against 7.5 of a code's own on average, 3.2 times, and a chunk at a time): 3e-6, 9e-6.  A hidden state in
    # one bf16 would be off by 1e-3.
    rng = np.random.default_rng(T + H + group)
    x = R.round_bf16(rng.standard_normal((T, H)))
    if kind == "bf16":
        u = R.round_bf16(rng.standard_normal((E, 2, I, H)) / np.sqrt(H))
        d = R.round_bf16(rng.standard_normal((E, H, I)) / np.sqrt(I))
        up, down = _bf16(u), _bf16(d)
        g, u, d = u[:, 0].transpose(0, 2, 1), u[:, 1].transpose(0, 2, 1), d.transpose(0, 2, 1)
    else:
        up, u = _w4(rng, (E, 2), H, I, group, zero, "f32", powers=(0.3 / np.sqrt(H), 0.2 / np.sqrt(H)))
        down, d = _w4(rng, (E,), I, H, group, zero, "f32", powers=(0.3 / np.sqrt(I), 0.2 / np.sqrt(I)))
        g, u = u[:, 0], u[:, 1]
    ids, w = _choices(rng, T, E, k)
    ref, root = np.zeros((T, H)), np.zeros((T, H))
    for t in range(T):
        for j in range(k):
            e = ids[t, j]
            h = w[t, j] * R.act(x[t] @ g[e], "silu") * (x[t] @ u[e])
            ref[t] += h @ d[e]
            root[t] += (h * h) @ (d[e] * d[e])
    mark(f"outputs round once T{T} E{E} k{k} {H}x{I} {kind}")
    y = _np(tg.moe_mlp(_bf16(x), _cuda(ids), _cuda(w), up, down))
    step = 2.0 ** (np.floor(np.log2(np.abs(ref))) - 7)
    off = (3e-6 if kind == "bf16" else 9e-6) * np.sqrt(root)
    allowed = float(np.minimum(off / step, 1.0).sum())
    assert np.all(np.abs(y - ref) <= 0.5 * step + off + 2.0 ** -8 * off), "one rounding, and what the sums are off by"
    assert int((y != R.round_bf16(ref)).sum()) <= allowed + 3 * np.sqrt(allowed), (allowed, y.size)


def test_silu_far_from_zero():
    # A neuron with gate g and one that takes its value away again, to 16 bits of it: y is what is left, 2^-17 of the
    # value or less, so its rounding to bf16 hides nothing.  SiLU in fp32: exp to a unit (2^-23), a sum and a quotient
    # to half of one each; the three parts of h and their sums another; u = 2^p and gate(64) = 64 are exact.
    g = R.round_bf16(-np.concatenate([np.linspace(18.0, 86.5, 40), [0.5, 1.0, 4.0, -3.0, -11.0, -30.0, 17.0, 87.0]]))
    n = len(g)
    value = g / (1.0 + np.exp(-g))
    u = 2.0 ** -np.floor(np.log2(np.abs(value)))
    take = -value * u / 64.0
    hi = R.round_bf16(take)
    mid = R.round_bf16(take - hi)
    up, down = np.zeros((1, 2, 2 * n, 16)), np.zeros((1, n, 2 * n))
    up[0, 0, 0::2, 0], up[0, 1, 0::2, 0] = g, u
    up[0, 0, 1::2, 0], up[0, 1, 1::2, 0], up[0, 1, 1::2, 1] = 64.0, hi, mid
    down[0, np.arange(n), 2 * np.arange(n)] = down[0, np.arange(n), 2 * np.arange(n) + 1] = 1.0
    for c in range(0, n, 16):                          # as many outputs as inputs a call
        y = tg.moe_mlp(torch.ones((1, 16), dtype=torch.bfloat16, device="cuda"), _cuda(np.zeros((1, 1), np.int32)),
                       torch.ones((1, 1), device="cuda"), _bf16(up), _bf16(down[:, c:c + 16]))
        ref = (value * u + 64.0 * (hi + mid))[c:c + 16]
        bound = 2.0 ** -8 * np.abs(ref) + (2.0 ** -23 + 3 * 2.0 ** -24) * np.abs(value * u)[c:c + 16]
        assert np.all(np.abs(_np(y)[0] - ref) <= bound), np.abs(_np(y)[0] - ref) / bound


# ---------------------------------------------------------------- arguments
def test_what_is_no_w4_is_refused_by_name():
    x = torch.ones((4, 64), dtype=torch.bfloat16, device="cuda")
    ids, w = torch.zeros((4, 1), dtype=torch.int32, device="cuda"), torch.ones((4, 1), device="cuda")
    up = torch.zeros((2, 2, 8, 64), dtype=torch.bfloat16, device="cuda")
    q, _ = _w4(np.random.default_rng(0), (), 64, 32, 32, False, "bf16")
    for bad in (None, torch.zeros((64, 32), dtype=torch.bfloat16, device="cuda"), q[:5]):
        with pytest.raises(TypeError, match="B must be a W4"):
            tg.gemm_w4(x, bad)
    for bad in (None, q, q[:5]):
        with pytest.raises(TypeError, match="gate_up must be"):
            tg.moe_mlp(x, ids, w, bad, torch.zeros((2, 64, 8), dtype=torch.bfloat16, device="cuda"))
    for bad in (None, q[:5]):
        with pytest.raises(TypeError, match="down must be"):
            tg.moe_mlp(x, ids, w, up, bad)


def test_a_group_longer_than_the_matrix_is_one_group():
    rng = np.random.default_rng(41)
    W = torch.from_numpy(rng.standard_normal((300, 40)).astype(np.float32)).cuda()
    A = torch.from_numpy(rng.integers(-4, 5, (70, 300)).astype(np.float32)).cuda().to(torch.bfloat16)
    want, values = tg.w4_quantize(W, 384, zero_point=True, values=True)
    for group in (2 ** 21, 2 ** 31 - 128):
        q, v = tg.w4_quantize(W, group, zero_point=True, values=True)
        assert torch.equal(q.words, want.words) and torch.equal(q.scales, want.scales) and torch.equal(v, values)
        for M in (1, 40, 70):
            assert torch.equal(tg.gemm_w4(A[:M], q), tg.gemm_w4(A[:M], want))


# ---------------------------------------------------------------- hot experts
def _skewed(rng, T, E, k, hot):
    """Every token names expert `hot` first, the others are spread over the rest."""
    rest = np.array([e for e in range(E) if e != hot])
    ids = np.stack([np.concatenate([[hot], rng.permutation(rest)[:k - 1]]) for _ in range(T)]).astype(np.int32)
    for row in ids:
        rng.shuffle(row)
    return ids, (rng.integers(1, 9, (T, k)) / 8.0).astype(np.float32)


def _check_close(y, x, ids, w, g, u, d, act):
    """Against the oracle in norms, token by token: g and u are exact, h is off by 2^-22 (exp, sum, quotient, product),
    the last sums by at most 48 + 4 blocks of fp32 additions of partial sums up to the root of their terms' squares (in
    4 bits 3.2 times that, see test_outputs_round_once), and one rounding to bf16 of half a step, 2^-8 of the value."""
    ref, root, d2 = np.zeros(y.shape), np.zeros(y.shape), d * d
    for t in range(len(x)):
        for j in range(ids.shape[1]):
            if 0 <= ids[t, j] < len(g):
                e = ids[t, j]
                h = w[t, j].astype(np.float64) * R.act(x[t] @ g[e], act) * (x[t] @ u[e])
                ref[t] += h @ d[e]
                root[t] += (h * h) @ d2[e]
    size = np.sqrt(root.sum(1))
    off = np.linalg.norm(_np(y) - ref, axis=1)
    assert np.all(off <= 2.0 ** -8 * np.linalg.norm(ref, axis=1) + 1e-5 * size), off / size


# (T, E, k, H, I, kind): whether there is one row tile (T k <= 8 E), and how many panels and blocks a workgroup has
HOT = [(64, 64, 2, 256, 128, "bf16"), (64, 64, 2, 256, 128, "w4"),
       # several blocks of both reductions, several panels a workgroup
       (40, 48, 2, 2200, 2100, "w4"), (33, 40, 2, 2200, 2304, "bf16"),
       # one panel a workgroup, one expert: next block's rows on their way with its words
       (20, 64, 1, 4104, 64, "w4"), (20, 64, 1, 4104, 64, "bf16"), (20, 64, 1, 64, 4104, "w4"),
       (20, 64, 1, 64, 4104, "bf16"),
       # two row tiles, more than 32 rows, several blocks
       (64, 2, 2, 2200, 1300, "w4"), (50, 3, 2, 2200, 1300, "bf16"), (64, 8, 8, 136, 72, "w4"),
       # the element-load forms
       (64, 64, 2, 1101, 1277, "bf16"), (40, 2, 2, 1101, 1277, "bf16"), (40, 48, 2, 1101, 1277, "w4")]


@pytest.mark.parametrize("T,E,k,H,I,kind", HOT)
def test_a_hot_expert_takes_several_passes(T, E, k, H, I, kind):
    rng = np.random.default_rng(T + H + I)
    some = E if E * H * I < 2 ** 24 else 3             # distinct experts; the others repeat them
    up, down, g, u, d = _experts(rng, some, H, I, kind)
    pick = np.arange(E) % some
    at = torch.from_numpy(pick).cuda()
    if kind == "w4":
        up, down = (tg.W4(q.words[at], q.scales[at], q.zeros[at], *q[3:]) for q in (up, down))
    else:
        up, down = up[at], down[at]
    x = rng.integers(-2, 3, (T, H)).astype(np.float64)
    ids, w = _skewed(rng, T, E, k, E // 3)
    mark(f"hot expert T{T} E{E} k{k} H{H} I{I} {kind} row tiles {1 if T <= 16 or T * k <= 8 * E else 2}")
    y = tg.moe_mlp(_bf16(x), _cuda(ids), _cuda(w), up, down)
    again = tg.moe_mlp(_bf16(x), _cuda(ids), _cuda(w), up, down)
    torch.cuda.synchronize()
    assert torch.equal(y, again)
    _check_close(y, x, pick[ids], w, g, u, d, "silu")


# ---------------------------------------------------------------- the range of 4-bit products
@pytest.mark.parametrize("M", [1, 20, 40, 130])
@pytest.mark.parametrize("group,zero", [(128, False), (128, True), (64, False), (64, True), (32, True), (32, False)])
def test_gemm_w4_up_to_the_end_of_its_range(M, group, zero):
    # integers times 2^114: sums of |A| over 128 k up to 128 * 4 * 2^114 = 2^123, the largest held; a power of two
    # changes no rounding, so exact integers stay exact
    rng = np.random.default_rng(M + group)
    K, N, far = 712, 72, 2.0 ** 114
    A = rng.integers(-4, 5, (M, K)).astype(np.float64)
    A[0], A[M // 2] = 4.0, -4.0
    q, W = _w4(rng, (), K, N, group, zero, "f32", powers=(0.5 / far, 1.0 / far, 2.0 / far))
    C = tg.gemm_w4(_bf16(A * far), q, out_dtype=torch.float32)
    assert np.array_equal(_np(C), (A * far) @ W)


@pytest.mark.parametrize("T", [3, 40])
@pytest.mark.parametrize("group,zero", [(128, False), (64, True), (32, True)])
def test_4_bit_experts_up_to_the_end_of_their_range(T, group, zero):
    # x and the hidden state times a power of two, the weights' scales divided by it: the same bits
    rng = np.random.default_rng(T + group)
    E, k, H, I, far = 2, 2, 200, 136, 2.0 ** 114
    up, down, g, u, d = _experts(rng, E, H, I, "w4", group, zero, "f32")
    x = rng.integers(-4, 5, (T, H)).astype(np.float64)
    x[0] = 4.0
    ids, w = _choices(rng, T, E, k)
    want = tg.moe_mlp(_bf16(x), _cuda(ids), _cuda(w), up, down)
    y = tg.moe_mlp(_bf16(x * far), _cuda(ids), _cuda(w), up._replace(scales=up.scales / far), down)
    assert torch.equal(y, want)
    h = np.max(np.abs(np.stack([R.act(x @ g[e], "silu") * (x @ u[e]) for e in range(E)])).sum(2))
    far = 2.0 ** (122 - np.ceil(np.log2(h)))           # times weights up to 1: half of the range
    y = tg.moe_mlp(_bf16(x), _cuda(ids), _cuda((w * far).astype(np.float32)), up,
                   down._replace(scales=down.scales / np.float32(far)))
    assert torch.equal(y, want) and bool(torch.isfinite(y).all())


# ---------------------------------------------------------------- quantisation
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("scale", ["f32", "bf16"])
def test_a_range_that_overflows_gives_nan_in_products_too(scale, dtype):
    W = torch.ones((160, 3), device="cuda")
    W[3, 0], W[4, 0] = 3e38, -3e38                     # hi - lo overflows fp32
    W[3, 1] = 3e38                                     # large, but no overflow
    if dtype == "bf16":
        W = W.to(torch.bfloat16)
    q, v = tg.w4_quantize(W, 64, zero_point=True, scale_dtype=torch.float32 if scale == "f32" else None, values=True)
    nan = torch.isnan(v).cpu()
    assert bool(nan[:64, 0].all()) and int(nan.sum()) == 64
    assert int(torch.isnan(q.scales).sum()) == 1 and not bool(torch.isinf(q.scales).any())
    A = torch.randn((70, 160), device="cuda").to(torch.bfloat16) * 2.0 ** -10      # S times 2e37 is in range
    for M in (1, 20, 70):
        C = tg.gemm_w4(A[:M], q, out_dtype=torch.float32)
        assert bool(torch.isnan(C[:, 0]).all()) and bool(torch.isfinite(C[:, 1:]).all())
    # symmetric: no overflow, the largest magnitude is a code
    s, v = tg.w4_quantize(W, 64, values=True)
    assert bool(torch.isfinite(s.scales).all()) and bool(torch.isfinite(v).all())


# ---------------------------------------------------------------- shares of the work
@pytest.mark.parametrize("cus", [1, 7, 304, 2 ** 31 - 1])
def test_shares_follow_the_device_description(cus):
    # More or fewer panels a workgroup: blocks of the reduction meet wave by wave or, with one panel, at the end, so
    # the same products are added in another order.  Either order is off by at most 136 additions in a group and
    # one a chunk or block, 2^-23 each of terms of up to 63 scales (test_gemm_w4_on_random_rows), before the
    # rounding to bf16, whose results are then a step (2^-7) apart at most.  g and u come in one block: the same bits.
    rng = np.random.default_rng(cus % 1000)
    q, W = _w4(rng, (), 2200, 700, 64, True, "bf16")
    up, down, g, u, d = _experts(rng, 5, 264, 2200, "w4")
    x = torch.randn((200, 2200), device="cuda").to(torch.bfloat16)
    rows = torch.randn((30, 264), device="cuda").to(torch.bfloat16)
    choice, share = _choices(rng, 30, 5, 2)
    ids, w = _cuda(choice), _cuda(share)

    def everything():
        return [tg.gemm_w4(x[:M], q) for M in (3, 30, 60, 200)] + \
            [tg.moe_mlp(rows[:T], ids[:T], w[:T], up, down) for T in (2, 30)]

    want = everything()
    desc = tg.get_device_desc()
    desc.n_cu = cus
    tg.set_device_override(desc)
    try:
        got = everything()
    finally:
        tg.set_device_override(None)
    size = np.abs(_np(x)) @ np.full((2200, 700), 63.0 * 2.0)
    _, terms = R.mlp(_np(rows), choice, share.astype(np.float64), g, u, d, "silu")
    terms *= np.max(np.abs(d)) / np.mean(np.abs(d)) * 63.0 * 1.01
    for a, b in zip(got, want):
        a, b = _np(a), _np(b)
        most = 2 * (136 + 18 + 18) * 2.0 ** -23 * (size if a.shape[1] == 700 else terms)[:len(a)]
        assert np.all(np.abs(a - b) <= 2.0 ** -7 * np.maximum(np.abs(a), np.abs(b)) + most)
    for a, b in zip(got[:4], want[:4]):
        assert np.linalg.norm(_np(a) - _np(b)) <= 2.0 ** -8 * np.linalg.norm(_np(b))


# ---------------------------------------------------------------- what the documents allow
@pytest.mark.parametrize("kind", ["bf16", "w4"])
@pytest.mark.parametrize("T", [3, 40])
def test_rows_off_alignment_an_output_given_and_what_is_around_it(T, kind):
    rng = np.random.default_rng(T)
    E, k, H, I = 2, 2, 264, 136
    up, down, *_ = _experts(rng, E, H, I, kind)
    x = _bf16(rng.integers(-2, 3, (T, H)))
    ids, w = (_cuda(a) for a in _choices(rng, T, E, k))
    want = tg.moe_mlp(x, ids, w, up, down)
    store = torch.full(((T + 2) * H + 1,), 7.0, dtype=torch.bfloat16, device="cuda")
    off = torch.empty(T * H + 1, dtype=torch.bfloat16, device="cuda")[1:].view(T, H)
    off.copy_(x)
    out = store[H + 1:(T + 1) * H + 1].view(T, H)
    got = tg.moe_mlp(off, ids, w, up, down, out=out)
    assert got is out and bool((store[:H + 1] == 7.0).all()) and bool((store[(T + 1) * H + 1:] == 7.0).all())
    # the same sums in the same order (one block of either reduction)
    assert torch.equal(out, want)
    logits = torch.randn((T, E), device="cuda")
    y, i, s = tg.moe_layer(off, logits, up, down, k, out=out)
    assert y is out and torch.equal(y, tg.moe_mlp(x, i, s, up, down))


def test_a_layer_with_masked_rows():
    rng = np.random.default_rng(2)
    up, down, *_ = _experts(rng, 6, 64, 48, "w4")
    x = torch.randn((5, 64), device="cuda").to(torch.bfloat16)
    logits = torch.randn((5, 6), device="cuda")
    clean, *_ = tg.moe_layer(x, logits, up, down, 2)
    logits[1] = -float("inf")                          # nothing is left
    logits[3] = torch.finfo(torch.float32).min         # all alike
    logits[4, 2] = float("nan")
    y, ids, w = tg.moe_layer(x, logits, up, down, 2)
    assert not bool(y[1].any()) and ids[1].tolist() == [0, 1] and w[1].tolist() == [0.0, 0.0]
    assert ids[3].tolist() == [0, 1] and w[3].tolist() == [0.5, 0.5] and bool(torch.isfinite(y[3]).all())
    assert ids[4].tolist()[0] == 2 and bool(torch.isnan(y[4]).all())
    assert torch.equal(y[[0, 2]], clean[[0, 2]])


@pytest.mark.parametrize("T,E,k,H,I,kind", [(64, 1024, 16, 16, 16, "bf16"), (2, 1, 1, 65536, 16, "bf16"),
                                            (20, 1, 1, 65536, 16, "w4"), (2, 1, 1, 16, 65536, "w4"),
                                            (20, 1, 1, 16, 65536, "bf16")])
def test_experts_at_their_limits(T, E, k, H, I, kind):
    rng = np.random.default_rng(H + I)
    up, down, g, u, d = _experts(rng, E, H, I, kind, 128, False)
    x = np.zeros((T, H))
    x[:, rng.choice(H, 64, replace=H < 64)] = rng.integers(-2, 3, (T, 64))
    x[:, -1] = 1.0
    ids, w = _choices(rng, T, E, k)
    mark(f"experts at their limits T{T} E{E} k{k} H{H} I{I} {kind}")
    y = tg.moe_mlp(_bf16(x), _cuda(ids), _cuda(w), up, down)
    torch.cuda.synchronize()
    # up to 32 blocks of two chunks one after the other: 4 + 32 more additions than _check_close counts, as 32 of its 48
    # are the k pairs and waves of larger layers
    _check_close(y, x, ids, w, g, u, d, "silu")


@pytest.mark.parametrize("M,N,K", [(1, 16, 2 ** 21), (70, 16, 2 ** 21), (3, 2 ** 21, 32), (2 ** 20, 16, 40)])
def test_gemm_w4_at_its_limits(M, N, K):
    rng = np.random.default_rng(M + N)
    P, C, G = -(-N // 16), -(-K // 128), -(-K // 128)
    words = torch.randint(-2 ** 31, 2 ** 31, (P, C, 64, 4), dtype=torch.int32, device="cuda")
    q = tg.W4(words, torch.ones((P, G, 16), device="cuda"), None, K, N, 128)
    # at most 32 of a row's elements are not zero: integers, exact
    at = np.unique(np.concatenate([rng.choice(K, 30), [0, K - 1]]))
    A = torch.zeros((M, K), dtype=torch.bfloat16, device="cuda")
    some = torch.from_numpy(rng.integers(-4, 5, (M, len(at))).astype(np.float32)).cuda()
    cols = torch.from_numpy(at).cuda()
    A[:, cols] = some.to(torch.bfloat16)
    mark(f"gemm_w4 at its limits {M}x{N}x{K}")
    C_ = tg.gemm_w4(A, q, out_dtype=torch.float32)
    n = torch.arange(N, device="cuda")
    ref = torch.zeros((M, N), device="cuda")
    for i, k in enumerate(at.tolist()):
        word = words[n // 16, k // 128, 16 * (k % 32 // 8) + n % 16, k % 128 // 32]
        code = (word >> (4 * (k % 8 // 2 + 4 * (k % 2)))) & 15
        ref += some[:, i:i + 1] * (code.float() - 8.0)
    assert torch.equal(C_, ref)


def test_route_and_quantize_at_their_limits():
    T = 2 ** 24
    logits = torch.randn((T, 2), device="cuda").to(torch.bfloat16)
    ids, w = tg.moe_route(logits, 1, renorm=True)
    assert torch.equal(ids[:, 0], (logits[:, 1] > logits[:, 0]).to(torch.int32)) and bool((w == 1.0).all())
    for K, N in ((2 ** 21, 3), (3, 2 ** 21)):
        W = (torch.randint(-7, 8, (K, N), device="cuda")).float()
        W[::32] = 7.0                                  # every group's scale is 1: the codes hold W
        q, v = tg.w4_quantize(W, 32, values=True)
        assert torch.equal(v, W) and bool((q.scales[:, :, :3] == 1.0).all())
