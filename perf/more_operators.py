"""Cases for the operators of 8-bit products and of expert layers on many tokens.

Five operators, each in a plain form of elementary torch operations (fp32, fp64
where 32 bits lose what matters) and, with `own` set, as calls of
tile_shape_autotuning_amd:

  quantize   [.., R, K] -> e4m3 codes with an fp32 scale for each 128 elements
             of a row, or for each block of 128 x 128
  gemm       C = act(A . B^T + bias) of two such matrices
  experts    the same for rows sorted by expert, each expert with its own B
  dispatch   (token, expert) pairs sorted by expert, the tokens' rows brought
             into that order
  combine    y[t] = sum_j weight[t, j] * row of the pair (t, j), and its gradient

Storage of 8-bit matrices, R rows x K columns: codes float8_e4m3fn
[.., R, 128 ceil(K / 128)], zero past K; scales fp32 [.., R, ceil(K / 128)]
(block 1) or [.., ceil(R / 128), ceil(K / 128)] (block 128).  An element is
code * scale.
"""
import math

import torch

own = False

LISTED = [
    # one token's hidden state on its way into an 8-bit projection: latency
    dict(name="quantize 1x4096", op="quantize", E=1, R=1, K=4096, block=1, dtype="bf16", along=True),
    # a training step's activations for the weight gradient: rows are channels, so blocks run down the columns
    dict(name="quantize 4096x8192 across", op="quantize", E=1, R=4096, K=8192, block=1, dtype="bf16", along=False),
    # one token through a square projection: the latency of a decode step
    dict(name="gemm 1x4096x4096", op="gemm", M=1, N=4096, K=4096, block=128, out="bf16", bias=False, act="none"),
    # a decode batch through a wide feed-forward projection: the weights' stream from HBM
    dict(name="gemm 16x28672x8192", op="gemm", M=16, N=28672, K=8192, block=128, out="bf16", bias=False, act="none"),
    # nothing divides anything; fp32 output, fused bias and GELU
    dict(name="gemm 333x1001x777", op="gemm", M=333, N=1001, K=777, block=1, out="f32", bias=True, act="gelu"),
    # a large square: bound by the matrix cores
    dict(name="gemm 8192x8192x8192", op="gemm", M=8192, N=8192, K=8192, block=128, out="bf16", bias=False, act="none"),
    # a decode batch over many small experts, gate and up together
    dict(name="experts 64x2816x2048", op="experts", T=64, E=64, k=6, N=2816, K=2048, block=128, out="bf16", skew=0.5,
         away=0.0),
    # a prompt over the same kind of experts, some chosen much more often than others
    dict(name="experts 4096x2048x2048", op="experts", T=4096, E=64, k=8, N=2048, K=2048, block=128, out="bf16",
         skew=1.0, away=0.0),
    # a handful of tokens with an odd width, some of their choices on another rank
    dict(name="dispatch 5x1000", op="dispatch", T=5, E=16, k=4, H=1000, dtype="bf16", skew=0.5, away=0.25),
    # a long prompt over many experts, quantised before it is copied
    dict(name="dispatch 16384x2048 fp8", op="dispatch", T=16384, E=256, k=8, H=2048, dtype="fp8", skew=1.0, away=0.0),
    # one token's experts meet again
    dict(name="combine 1x2048", op="combine", T=1, E=64, k=6, H=2048, dtype="bf16", skew=0.5, away=0.0, grad=False),
    # a training step: the sum, and the gradients of the rows and of the weights
    dict(name="combine 8192x4096 step", op="combine", T=8192, E=64, k=8, H=4096, dtype="bf16", skew=1.0, away=0.0,
         grad=True),
]


def listed():
    return [dict(c) for c in LISTED]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return int(max(lo, min(hi, round(v / step) * step)))


def draw(rng):
    op = rng.choice(["quantize", "gemm", "gemm", "experts", "experts", "dispatch", "combine"])
    step = rng.choice([1, 8, 128])
    block = rng.choice([1, 128, 128])
    if op == "quantize":
        while True:
            E, R, K = _log(rng, 1, 16), _log(rng, 1, 16384), _log(rng, 64, 16384, step)
            if E * R * K <= 2 ** 26:
                break
        return dict(op=op, E=E, R=R, K=K, block=block, dtype=rng.choice(["bf16", "f32"]), along=rng.random() < 0.6)
    if op == "gemm":
        while True:
            M, N, K = _log(rng, 1, 8192), _log(rng, 64, 28672, step), _log(rng, 64, 16384, step)
            if M * N * K <= 2 ** 38 and N * K <= 2 ** 28:
                break
        return dict(op=op, M=M, N=N, K=K, block=block, out=rng.choice(["bf16", "f32"]), bias=rng.random() < 0.5,
                    act=rng.choice(["none", "relu", "gelu"]))
    T, E = _log(rng, 1, 8192), _log(rng, 4, 256)
    k = rng.randint(1, min(8, E))
    c = dict(op=op, T=T, E=E, k=k, skew=rng.choice([0.0, 0.5, 1.0]), away=rng.choice([0.0, 0.0, 0.25]))
    if op == "experts":
        while True:
            N, K = _log(rng, 128, 8192, step), _log(rng, 128, 8192, step)
            if E * N * K <= 2 ** 29 and T * k * N * K <= 2 ** 37:
                break
        c.update(N=N, K=K, block=block, out=rng.choice(["bf16", "f32"]))
        return c
    while True:
        H = _log(rng, 64, 8192, step)
        if T * k * H <= 2 ** 28:
            break
    if op == "dispatch":
        c.update(H=H, dtype=rng.choice(["bf16", "f32", "fp8"]))
    else:
        c.update(H=H, dtype=rng.choice(["bf16", "f32"]), grad=rng.random() < 0.5)
    return c


DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _ceil(a, b):
    return -(-a // b)


def _spread(t, n, dim):
    """Each element of `dim` 128 times, the first n of them."""
    return t.repeat_interleave(128, dim=dim).narrow(dim, 0, n)


def _stored(gen, lead, R, K, block):
    """Random matrices in storage form: columns of different size, as channels of activations and weights are."""
    C, P = _ceil(K, 128), _ceil(R, block)
    x = torch.randn((*lead, R, K), device="cuda", generator=gen)
    x *= torch.exp(0.5 * torch.randn(K, device="cuda", generator=gen))
    x = torch.nn.functional.pad(x, (0, C * 128 - K, 0, P * block - R)).view(-1, P, block, C, 128)
    scales = x.abs().amax(dim=(2, 4)) / 448.0
    codes = (x / scales.view(-1, P, 1, C, 1)).clamp_(-448.0, 448.0).to(torch.float8_e4m3fn)
    codes = codes.view(-1, P * block, C * 128)[:, :R].contiguous()
    return codes.view(*lead, R, C * 128), scales.view(*lead, P, C), K, block


def _choices(gen, c):
    """Each token's experts: the k largest of logits that favour some experts over others, a part of them elsewhere."""
    T, E, k = c["T"], c["E"], c["k"]
    logits = torch.randn((T, E), device="cuda", generator=gen)
    logits += c["skew"] * torch.randn(E, device="cuda", generator=gen)
    top, ids = torch.sort(logits, dim=1, descending=True, stable=True)
    ids = ids[:, :k].to(torch.int32)
    gone = torch.rand((T, k), device="cuda", generator=gen) < c["away"]
    return torch.where(gone, torch.full_like(ids, -1), ids).contiguous(), torch.softmax(top[:, :k], dim=1).contiguous()


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))

    def normal(*shape):
        return torch.randn(shape, device="cuda", generator=gen)

    s = {"case": c}
    if c["op"] == "quantize":
        shape = (c["E"], c["R"], c["K"]) if c["along"] else (c["E"], c["K"], c["R"])
        x = normal(*shape) * torch.exp(0.5 * normal(c["E"], 1, shape[2]))
        x = x.to(DTYPES[c["dtype"]])
        s["x"] = x if c["along"] else x.transpose(1, 2)
    elif c["op"] == "gemm":
        s["A"] = _stored(gen, (), c["M"], c["K"], 1)
        s["B"] = _stored(gen, (), c["N"], c["K"], c["block"])
        s["bias"] = normal(c["N"]) if c["bias"] else None
    else:
        ids, weights = _choices(gen, c)
        n = ids.numel()
        if c["op"] == "dispatch":
            s["ids"] = ids
            if c["dtype"] == "fp8":
                s["x"] = _stored(gen, (), c["T"], c["H"], 1)
                s["out"] = (torch.zeros((n, s["x"][0].shape[1]), device="cuda").to(torch.float8_e4m3fn),
                            torch.zeros((n, s["x"][1].shape[1]), device="cuda"), c["H"], 1)
            else:
                s["x"] = normal(c["T"], c["H"]).to(DTYPES[c["dtype"]])
                s["out"] = torch.zeros((n, c["H"]), dtype=DTYPES[c["dtype"]], device="cuda")
            return s
        s["order"] = _plain_sort(ids, c["E"])
        if c["op"] == "experts":
            s["A"] = _stored(gen, (), n, c["K"], 1)
            s["B"] = _stored(gen, (c["E"],), c["N"], c["K"], c["block"])
            s["out"] = torch.zeros((n, c["N"]), dtype=DTYPES[c["out"]], device="cuda")
        else:
            s["weights"] = weights
            s["rows"] = normal(n, c["H"]).to(DTYPES[c["dtype"]])
            if c["grad"]:
                s["dy"] = normal(c["T"], c["H"]).to(DTYPES[c["dtype"]])
                s["drows"] = torch.zeros((n, c["H"]), dtype=DTYPES[c["dtype"]], device="cuda")
    return s


# ---------------------------------------------------------------- plain forms
def _act(v, act):
    if act == "relu":
        return torch.clamp_min(v, 0.0)
    if act == "gelu":
        return 0.5 * v * (1.0 + torch.erf(v * math.sqrt(0.5)))
    return v


def _e4m3(q):
    """The nearest of the type's values, ties to the even one, up to 448; fp64 in, fp64 out."""
    a = q.abs()
    step = torch.exp2(torch.clamp_min(torch.floor(torch.log2(torch.clamp_min(a, 2.0 ** -20))), -6.0) - 3.0)
    return torch.copysign(torch.clamp_max(torch.round(a / step) * step, 448.0), q)


def _dense(m):
    """Storage form -> fp32 [.., R, 128 ceil(K / 128)]."""
    codes, scales, K, block = m
    scales = _spread(scales, codes.shape[-1], -1)
    if block == 128:
        scales = _spread(scales, codes.shape[-2], -2)
    return codes.float() * scales


def _plain_quantize(s):
    c, x = s["case"], s["x"]
    E, R, K, block = c["E"], c["R"], c["K"], c["block"]
    C, P = _ceil(K, 128), _ceil(R, block)
    x = torch.nn.functional.pad(x.float(), (0, C * 128 - K, 0, P * block - R)).view(E, P, block, C, 128)
    scales = (x.abs().amax(dim=(2, 4)).double() / 448.0).float()
    unit = torch.where(scales == 0, torch.ones_like(scales), scales).double().view(E, P, 1, C, 1)
    codes = _e4m3(x.double() / unit).float()
    values = (codes * scales.view(E, P, 1, C, 1)).view(E, P * block, C * 128)[:, :R, :K]
    codes = codes.view(E, P * block, C * 128)[:, :R].to(torch.float8_e4m3fn)
    return {"codes": codes, "scales": scales, "values": values.to(DTYPES[c["dtype"]])}


def _plain_gemm(s):
    v = torch.matmul(_dense(s["A"]), _dense(s["B"]).transpose(0, 1))
    if s["bias"] is not None:
        v = v + s["bias"]
    return _act(v, s["case"]["act"]).to(DTYPES[s["case"]["out"]])


def _plain_experts(s):
    A, out = _dense(s["A"]), s["out"]
    codes, scales, K, block = s["B"]
    ends = s["order"][2].tolist()
    for e in range(s["case"]["E"]):
        if ends[e] < ends[e + 1]:
            B = _dense((codes[e], scales[e], K, block))
            out[ends[e]:ends[e + 1]] = torch.matmul(A[ends[e]:ends[e + 1]], B.transpose(0, 1)).to(out.dtype)
    return out


def _plain_sort(ids, E):
    """(position [T, k], source [T k], offsets [E + 1]): pairs by expert, in the order of their numbers within one;
    pairs elsewhere have position -1, and rows behind the last pair source -1."""
    flat = ids.reshape(-1).long()
    n = flat.numel()
    here = (flat >= 0) & (flat < E)
    _, source = torch.sort(torch.where(here, flat, torch.full_like(flat, E)), stable=True)
    counts = torch.zeros(E + 1, dtype=torch.long, device=ids.device)
    counts.scatter_add_(0, torch.where(here, flat + 1, torch.zeros_like(flat)), here.long())
    offsets = torch.cumsum(counts, 0)
    rank = torch.arange(n, device=ids.device)
    position = torch.empty_like(flat).scatter_(0, source, rank)
    position = torch.where(here, position, torch.full_like(position, -1)).view(ids.shape)
    source = torch.where(rank < offsets[E], source, torch.full_like(source, -1))
    return position.to(torch.int32), source.to(torch.int32), offsets.to(torch.int32)


def _plain_gather(x, source, k, out):
    at = (torch.clamp_min(source, 0) // k).long()
    keep = (source >= 0).unsqueeze(1)
    if x.element_size() == 1:                          # codes are moved, not computed with
        out = out.view(torch.uint8)
        return torch.where(keep, x.view(torch.uint8)[at], out).view(torch.float8_e4m3fn)
    return torch.where(keep, x[at], out)


def _plain_dispatch(s):
    c = s["case"]
    position, source, offsets = _plain_sort(s["ids"], c["E"])
    if c["dtype"] == "fp8":
        rows = tuple(_plain_gather(s["x"][i], source, c["k"], s["out"][i]) for i in (0, 1))
    else:
        rows = _plain_gather(s["x"], source, c["k"], s["out"])
    return position, source, offsets, rows


def _plain_combine(s):
    c, rows, position = s["case"], s["rows"], s["order"][0]
    T, k, H = c["T"], c["k"], c["H"]
    here = (position >= 0).unsqueeze(-1)
    at = torch.clamp_min(position, 0).long()
    w = torch.where(here, s["weights"].unsqueeze(-1), torch.zeros((), device=rows.device))
    y = torch.zeros((T, H), device=rows.device)
    for j in range(k):
        y = y + w[:, j] * rows[at[:, j]].float()
    y = y.to(rows.dtype)
    if not c["grad"]:
        return y
    dy, drows = s["dy"].float(), s["drows"]
    dw = torch.empty((T, k), device=rows.device)
    for j in range(k):
        dw[:, j] = torch.where(here[:, j, 0], (dy * rows[at[:, j]].float()).sum(dim=1), torch.zeros_like(dw[:, j]))
    source = s["order"][1]
    pair = torch.clamp_min(source, 0).long()
    d = (dy[pair // k] * s["weights"].reshape(-1)[pair].unsqueeze(1)).to(rows.dtype)
    return y, torch.where((source >= 0).unsqueeze(1), d, drows), dw


def run(state):
    c = state["case"]
    op = c["op"]
    if own:
        import tile_shape_autotuning_amd as tg
        if op == "quantize":
            q, values = tg.fp8_quantize(state["x"], c["block"], values=True)
            return {"codes": q.codes, "scales": q.scales, "values": values}
        if op == "gemm":
            return tg.gemm_fp8(state["A"], state["B"], state["bias"], act=c["act"], out_dtype=DTYPES[c["out"]])
        if op == "experts":
            return tg.moe_gemm_fp8(state["A"], state["B"], state["order"][2], out=state["out"])
        if op == "dispatch":
            order = tg.moe_sort(state["ids"], c["E"])
            rows = tg.moe_gather(state["x"], order, out=state["out"])
            return order.position, order.source, order.offsets, tuple(rows[:2]) if c["dtype"] == "fp8" else rows
        y = tg.moe_combine(state["rows"], state["order"], state["weights"])
        if not c["grad"]:
            return y
        return (y,) + tuple(tg.moe_combine_grad(state["dy"], state["rows"], state["order"], state["weights"],
                                                out=state["drows"]))
    if op == "quantize":
        return _plain_quantize(state)
    if op == "gemm":
        return _plain_gemm(state)
    if op == "experts":
        return _plain_experts(state)
    if op == "dispatch":
        return _plain_dispatch(state)
    return _plain_combine(state)


# ---------------------------------------------------------------- what a pass cannot do without
def _stored_bytes(R, K, block):
    return float(R * K + 4 * _ceil(R, block) * _ceil(K, 128))


def work(case):
    c = case
    size = {"bf16": 2, "f32": 4}
    if c["op"] == "quantize":
        n = c["E"] * c["R"] * c["K"]
        return {"bytes": 2 * size[c["dtype"]] * n + c["E"] * _stored_bytes(c["R"], c["K"], c["block"]),
                "flops": 3.0 * n}
    if c["op"] == "gemm":
        M, N, K = c["M"], c["N"], c["K"]
        b = _stored_bytes(M, K, 1) + _stored_bytes(N, K, c["block"]) + size[c["out"]] * M * N
        return {"bytes": b + (4 * N if c["bias"] else 0), "flops": 2.0 * M * N * K}
    stays = 1.0 - c["away"]
    T, E, k = c["T"], c["E"], c["k"]
    n = stays * T * k
    if c["op"] == "experts":
        N, K = c["N"], c["K"]
        active = E * (1.0 - (1.0 - stays * k / E) ** T)          # experts that T tokens choose on average
        b = n / (T * k) * (_stored_bytes(T * k, K, 1) + size[c["out"]] * T * k * N)
        return {"bytes": b + active * _stored_bytes(N, K, c["block"]) + 4 * (E + 1), "flops": 2.0 * n * N * K}
    H = c["H"]
    if c["op"] == "dispatch":
        row = _stored_bytes(1, H, 1) if c["dtype"] == "fp8" else size[c["dtype"]] * H
        return {"bytes": row * (T + n) + 12.0 * T * k + 4 * (E + 1), "flops": float(T * k)}
    b = size[c["dtype"]] * H * (n + T) + 8.0 * T * k
    if c["grad"]:
        b += size[c["dtype"]] * H * (n + T) + 4.0 * T * k
    return {"bytes": b, "flops": (5.0 if c["grad"] else 2.0) * n * H}


# ---------------------------------------------------------------- the definition, in 64 bits
def _nearest_code(q):
    """Values of the nearest codes, from the list of all of them."""
    table = torch.arange(127, dtype=torch.uint8, device=q.device).view(torch.float8_e4m3fn).double()
    middle = (table[1:] + table[:-1]) / 2
    a = q.abs()
    low = torch.bucketize(a, middle)                   # how many middles lie below
    tie = (low < 126) & (a == middle[low.clamp_max(125)]) & (low % 2 == 1)
    return torch.where(q < 0, -1.0, 1.0) * table[low + tie.long()]


def _matrix64(m, at=()):
    codes, scales, K, block = m
    r = torch.arange(codes.shape[-2], device=codes.device).view(-1, 1) // block
    k = torch.arange(K, device=codes.device).view(1, -1) // 128
    return codes[at][:, :K].double() * scales[at][r, k].double()


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "quantize":
        E, R, K, block = c["E"], c["R"], c["K"], c["block"]
        C, P = _ceil(K, 128), _ceil(R, block)
        codes = torch.zeros((E, R, C * 128), dtype=torch.float64, device="cuda")
        scales = torch.empty((E, P, C), dtype=torch.float64, device="cuda")
        values = torch.empty((E, R, K), dtype=torch.float64, device="cuda")
        r = torch.arange(R, device="cuda") // block
        for i in range(C):
            x = s["x"][:, :, i * 128:(i + 1) * 128].double()
            top = torch.zeros((E, P), dtype=torch.float64, device="cuda")
            top = top.scatter_reduce(1, r.expand(E, R), x.abs().amax(dim=2), "amax")
            step = (top / 448.0).float().double()
            scales[:, :, i] = step
            unit = torch.where(step > 0, step, torch.ones_like(step))[:, r].unsqueeze(2)
            code = _nearest_code(x / unit)
            codes[:, :, i * 128:i * 128 + x.shape[2]] = code
            values[:, :, i * 128:i * 128 + x.shape[2]] = code * step[:, r].unsqueeze(2)
        return {"codes": codes, "scales": scales, "values": values}
    if c["op"] == "gemm":
        v = _matrix64(s["A"]) @ _matrix64(s["B"]).t()
        if s["bias"] is not None:
            v += s["bias"].double()
        if c["act"] == "relu":
            return torch.where(v > 0, v, torch.zeros_like(v))
        if c["act"] == "gelu":
            return v * torch.special.erfc(-v / math.sqrt(2.0)) / 2.0
        return v
    T, k = c["T"], c["k"]
    if c["op"] == "experts":
        ends = s["order"][2].tolist()
        A, y = _matrix64(s["A"]), torch.zeros((T * k, c["N"]), dtype=torch.float64, device="cuda")
        for e in range(c["E"]):
            if ends[e] < ends[e + 1]:
                y[ends[e]:ends[e + 1]] = A[ends[e]:ends[e + 1]] @ _matrix64(s["B"], e).t()
        return y
    if c["op"] == "dispatch":
        # expert after expert; whole numbers are compared with the plain form's
        pairs = torch.cat([torch.nonzero(s["ids"].flatten() == e).flatten() for e in range(c["E"])])
        parts = [(a.double(), torch.zeros(b.shape, dtype=torch.float64, device="cuda"))
                 for a, b in (zip(s["x"][:2], s["out"][:2]) if c["dtype"] == "fp8" else [(s["x"], s["out"])])]
        for a, rows in parts:
            rows[:pairs.numel()] = a[pairs // k]
        rows = tuple(r for _, r in parts) if c["dtype"] == "fp8" else parts[0][1]
        return None, None, None, rows
    position, rows = s["order"][0].long(), s["rows"]
    y = torch.zeros((T, c["H"]), dtype=torch.float64, device="cuda")
    dw = torch.zeros((T, k), dtype=torch.float64, device="cuda")
    drows = torch.zeros((T * k, c["H"]), dtype=torch.float64, device="cuda")
    for j in range(k):
        t = torch.nonzero(position[:, j] >= 0).flatten()
        p = position[t, j]
        w = s["weights"][t, j].double().unsqueeze(1)
        y[t] += w * rows[p].double()
        if c["grad"]:
            dy = s["dy"][t].double()
            dw[t, j] = (dy * rows[p].double()).sum(dim=1)
            drows[p] = w * dy
    return (y, drows, dw) if c["grad"] else y
