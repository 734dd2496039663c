"""Cases for the operators that work on expert layers and 4-bit weights.

Five operators of a decoder's feed-forward path, each in a plain form of
elementary torch operations (fp32, fp64 where 32 bits lose what matters) and,
with `own` set, as calls of tile_shape_autotuning_amd:

  quantize   weights [.., K, N] -> 4-bit codes with a scale (and a zero point)
             for each group of rows of a column
  gemm       C = act(A . W + bias) on such weights
  route      softmax over the experts' logits, the k largest of each token
  mlp        y[t] = sum_j weight[t, j] * expert ids[t, j] (x[t]), gated experts,
             bf16 or 4-bit
  layer      mlp with the routing taken from the logits in the same call

Storage of 4-bit weights, K rows x N columns: panels of 16 columns and chunks
of 128 rows, words [ceil(N/16), ceil(K/128), 64, 4] int32.  Word (p, c, l, t)
holds column 16 p + l % 16, rows 128 c + 32 t + 8 (l // 16) + 0..7; its nibbles
0..3 hold the even rows 0, 2, 4, 6 and its nibbles 4..7 the odd rows 1, 3, 5, 7.
Scales (bf16 or fp32) and zero points (uint8; absent: 8) are
[ceil(N/16), ceil(K/group), 16].  A weight is scale * (code - zero point).
"""
import math

import torch

own = False

# One entry per operator at the ends and in the middle of its range.
LISTED = [
    # one token through a square projection: the latency of a decode step
    dict(name="gemm 1x4096x4096", op="gemm", M=1, N=4096, K=4096, group=128, zero=False, scale="bf16", out="bf16",
         bias=False, act="none"),
    # a decode batch through a wide feed-forward projection: the weights' stream from HBM
    dict(name="gemm 16x28672x8192", op="gemm", M=16, N=28672, K=8192, group=128, zero=True, scale="bf16", out="bf16",
         bias=False, act="none"),
    # nothing divides anything: odd K and N, small groups, fp32 scales and output, fused bias and GELU
    dict(name="gemm 48x1001x777", op="gemm", M=48, N=1001, K=777, group=32, zero=True, scale="f32", out="f32",
         bias=True, act="gelu"),
    # a prompt: enough rows to be bound by the matrix cores
    dict(name="gemm 2048x4096x4096", op="gemm", M=2048, N=4096, K=4096, group=128, zero=False, scale="bf16",
         out="bf16", bias=False, act="none"),
    # a projection's weights, as stored for the product
    dict(name="quantize 4096x4096", op="quantize", E=1, K=4096, N=4096, group=128, zero=False, scale="bf16",
         dtype="bf16", rows_first=True),
    # a stack of experts kept as output rows x input columns in fp32, with zero points
    dict(name="quantize 16x2048x1408", op="quantize", E=16, K=2048, N=1408, group=64, zero=True, scale="f32",
         dtype="f32", rows_first=False),
    # one token's routing
    dict(name="route 1x64", op="route", T=1, E=64, k=6, renorm=True, dtype="f32"),
    # a long prompt's routing
    dict(name="route 16384x256", op="route", T=16384, E=256, k=8, renorm=False, dtype="bf16"),
    # a handful of tokens with odd widths, some of their choices on another rank
    dict(name="mlp 5x1000x1242 bf16", op="mlp", T=5, E=16, k=4, H=1000, I=1242, w="bf16", group=0, zero=False,
         scale="bf16", gate="gelu", away=0.25),
    # a decode batch over many small experts in 4 bits
    dict(name="mlp 64x2048x1408 w4", op="mlp", T=64, E=64, k=6, H=2048, I=1408, w="w4", group=64, zero=True,
         scale="bf16", gate="silu", away=0.0),
    # one token through two of eight large experts: the weights' stream from HBM
    dict(name="layer 1x4096x14336 bf16", op="layer", T=1, E=8, k=2, H=4096, I=14336, w="bf16", group=0, zero=False,
         scale="bf16", gate="silu", renorm=True),
    # a small decode batch over many experts in 4 bits, from the logits
    dict(name="layer 16x2048x1024 w4", op="layer", T=16, E=64, k=8, H=2048, I=1024, w="w4", group=128, zero=False,
         scale="bf16", gate="silu", renorm=True),
]


def listed():
    return [dict(c) for c in LISTED]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return int(max(lo, min(hi, round(v / step) * step)))


def draw(rng):
    op = rng.choice(["gemm", "gemm", "quantize", "route", "mlp", "layer"])
    group = rng.choice([32, 64, 128, 256, 1024])
    zero = rng.random() < 0.5
    scale = rng.choice(["bf16", "f32"])
    step = rng.choice([1, 8, 64])
    if op == "gemm":
        while True:
            M, N, K = _log(rng, 1, 2048), _log(rng, 64, 28672, step), _log(rng, 64, 8192, step)
            if M * N * K <= 2048 * 4096 * 4096:
                break
        return dict(op=op, M=M, N=N, K=K, group=group, zero=zero, scale=scale, out=rng.choice(["bf16", "f32"]),
                    bias=rng.random() < 0.5, act=rng.choice(["none", "relu", "gelu"]))
    if op == "quantize":
        while True:
            E, K, N = _log(rng, 1, 16), _log(rng, 64, 8192, step), _log(rng, 64, 8192, step)
            if E * K * N <= 16 * 2048 * 1408:
                break
        return dict(op=op, E=E, K=K, N=N, group=group, zero=zero, scale=scale, dtype=rng.choice(["bf16", "f32"]),
                    rows_first=rng.random() < 0.5)
    if op == "route":
        E = _log(rng, 8, 512)
        return dict(op=op, T=_log(rng, 1, 8192), E=E, k=rng.randint(1, 8), renorm=rng.random() < 0.5,
                    dtype=rng.choice(["bf16", "f32"]))
    while True:
        T, E = _log(rng, 1, 96), _log(rng, 8, 128)
        k = rng.randint(1, min(8, E))
        H, I = _log(rng, 256, 4096, step), _log(rng, 128, 14336, step)
        w = rng.choice(["bf16", "w4"])
        size = 2 if w == "bf16" else 0.5
        if min(E, T * k) * H * I * size <= 2 * 4096 * 14336 * 2 and E * H * I <= 8 * 4096 * 14336:
            break
    c = dict(op=op, T=T, E=E, k=k, H=H, I=I, w=w, group=group if w == "w4" else 0, zero=zero and w == "w4",
             scale=scale, gate=rng.choice(["silu", "gelu"]))
    if op == "mlp":
        c["away"] = rng.choice([0.0, 0.25])
    else:
        c["renorm"] = rng.random() < 0.5
    return c


DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _ceil(a, b):
    return -(-a // b)


def _packed(gen, lead, K, N, group, zero, scale):
    """Random 4-bit weights in storage form whose products with unit rows are of order one: every code, zero points
    in the middle of their range, scales of one sign that differ from group to group."""
    P, C, G = _ceil(N, 16), _ceil(K, 128), _ceil(K, group)
    words = torch.randint(-2 ** 31, 2 ** 31, (*lead, P, C, 64, 4), dtype=torch.int32, device="cuda", generator=gen)
    scales = (0.5 + torch.rand((*lead, P, G, 16), device="cuda", generator=gen)) / (4.8 * math.sqrt(K))
    zeros = None
    if zero:
        zeros = torch.randint(5, 11, (*lead, P, G, 16), dtype=torch.uint8, device="cuda", generator=gen)
    return words, scales.to(DTYPES[scale]), zeros, K, N, group


def _experts(gen, c):
    E, H, I = c["E"], c["H"], c["I"]
    if c["w"] == "w4":
        return (_packed(gen, (E, 2), H, I, c["group"], c["zero"], c["scale"]),
                _packed(gen, (E,), I, H, c["group"], c["zero"], c["scale"]))
    up = torch.empty((E, 2, I, H), dtype=torch.bfloat16, device="cuda").normal_(0.0, 1 / math.sqrt(H), generator=gen)
    down = torch.empty((E, H, I), dtype=torch.bfloat16, device="cuda").normal_(0.0, 1 / math.sqrt(I), generator=gen)
    return up, down


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))

    def normal(*shape):
        return torch.randn(shape, device="cuda", generator=gen)

    s = {"case": c}
    if c["op"] == "gemm":
        s["A"] = normal(c["M"], c["K"]).to(torch.bfloat16)
        s["B"] = _packed(gen, (), c["K"], c["N"], c["group"], c["zero"], c["scale"])
        s["bias"] = normal(c["N"]) if c["bias"] else None
    elif c["op"] == "quantize":
        # weights of a trained layer: rows of different scales, a shifted mean where zero points are of use
        shape = (c["E"], c["K"], c["N"]) if c["rows_first"] else (c["E"], c["N"], c["K"])
        W = normal(*shape) * (0.02 * (0.5 + torch.rand((c["E"], 1, 1), device="cuda", generator=gen)))
        W = (W + (0.01 if c["zero"] else 0.0)).to(DTYPES[c["dtype"]])
        s["W"] = W if c["rows_first"] else W.transpose(1, 2)
    elif c["op"] == "route":
        s["logits"] = (2.0 * normal(c["T"], c["E"])).to(DTYPES[c["dtype"]])
    else:
        s["x"] = normal(c["T"], c["H"]).to(torch.bfloat16)
        s["up"], s["down"] = _experts(gen, c)
        logits = 2.0 * normal(c["T"], c["E"])
        if c["op"] == "layer":
            s["logits"] = logits
        else:
            p, ids = torch.sort(logits, dim=1, descending=True, stable=True)
            ids = ids[:, :c["k"]].to(torch.int32)
            away = torch.rand(ids.shape, device="cuda", generator=gen) < c["away"]
            s["ids"] = torch.where(away, torch.full_like(ids, -1), ids).contiguous()
            s["weights"] = torch.softmax(p[:, :c["k"]], dim=1).contiguous()
    return s


# ---------------------------------------------------------------- plain forms
def _act(v, act):
    if act == "relu":
        return torch.clamp_min(v, 0.0)
    if act == "gelu":
        return 0.5 * v * (1.0 + torch.erf(v * math.sqrt(0.5)))
    if act == "silu":
        return v / (1.0 + torch.exp(-v))
    return v


def _per_group(t, N):
    """[.., P, G, 16] -> [.., G, N]"""
    t = t.transpose(-3, -2)
    return t.reshape(*t.shape[:-2], -1)[..., :N]


def _dense(packed):
    """Storage form -> fp32 [.., K, N]"""
    words, scales, zeros, K, N, group = packed
    lead, (P, C) = words.shape[:-4], words.shape[-4:-2]
    r = torch.arange(8, dtype=torch.int32, device=words.device)
    q = (words.unsqueeze(-1) >> (r % 2 * 16 + r // 2 * 4)) & 15
    n = len(lead)
    q = q.view(*lead, P, C, 4, 16, 4, 8).permute(*range(n), n + 1, n + 4, n + 2, n + 5, n, n + 3)
    q = q.reshape(*lead, C * 128, P * 16)[..., :K, :N].float()
    s = _per_group(scales, N).float().repeat_interleave(group, dim=-2)[..., :K, :]
    if zeros is None:
        return (q - 8.0) * s
    return (q - _per_group(zeros, N).float().repeat_interleave(group, dim=-2)[..., :K, :]) * s


def _plain_gemm(s):
    c = s["case"]
    v = torch.matmul(s["A"].float(), _dense(s["B"]))
    if s["bias"] is not None:
        v = v + s["bias"]
    return _act(v, c["act"]).to(DTYPES[c["out"]])


def _plain_quantize(s):
    c, W = s["case"], s["W"].float()
    E, K, N, group = c["E"], c["K"], c["N"], c["group"]
    P, C, G = _ceil(N, 16), _ceil(K, 128), _ceil(K, group)
    Wg = torch.nn.functional.pad(W, (0, 0, 0, G * group - K)).view(E, G, group, N)
    if c["zero"]:
        lo, hi = Wg.amin(dim=2), Wg.amax(dim=2)        # a group's range always holds zero
        lo, hi = torch.clamp_max(lo, 0.0), torch.clamp_min(hi, 0.0)
        scale = ((hi - lo).double() / 15.0).float().to(DTYPES[c["scale"]])
        sd = torch.where(scale == 0, torch.ones_like(scale), scale).double()
        z = torch.round(-lo.double() / sd).clamp(0, 15)
    else:
        scale = (Wg.abs().amax(dim=2).double() / 7.0).float().to(DTYPES[c["scale"]])
        sd = torch.where(scale == 0, torch.ones_like(scale), scale).double()
        z = torch.full_like(sd, 8.0)
    q = (torch.round(Wg.double() / sd.unsqueeze(2)) + z.unsqueeze(2)).clamp(0, 15)
    values = ((q - z.unsqueeze(2)).float() * scale.float().unsqueeze(2)).view(E, G * group, N)[:, :K]
    q = q.view(E, G * group, N)[:, :K].to(torch.int64)
    q = torch.nn.functional.pad(q, (0, P * 16 - N, 0, C * 128 - K)).view(E, C, 4, 4, 8, P, 16)
    r = torch.arange(8, dtype=torch.int64, device=q.device)
    shift = (r % 2 * 16 + r // 2 * 4).view(8, 1, 1)
    words = (q << shift).sum(dim=4).permute(0, 4, 1, 3, 5, 2).reshape(E, P, C, 64, 4).to(torch.int32)

    def stored(t):
        t = torch.nn.functional.pad(t, (0, P * 16 - N)).view(E, G, P, 16)
        return t.transpose(1, 2).contiguous()

    out = {"words": words, "scales": stored(scale), "values": values.to(DTYPES[c["dtype"]])}
    if c["zero"]:
        out["zeros"] = stored(z).to(torch.uint8)
    return out


def _plain_route(logits, k, renorm):
    v, ids = torch.sort(logits.float(), dim=1, descending=True, stable=True)
    p = torch.exp(v - v[:, :1])
    top = p[:, :k]
    total = top.sum(dim=1, keepdim=True) if renorm else p.sum(dim=1, keepdim=True)
    return ids[:, :k].to(torch.int32), top / total


def _plain_mlp(s, ids, weights):
    c = s["case"]
    T, E, k, H, I = c["T"], c["E"], c["k"], c["H"], c["I"]
    x = s["x"].float()
    here = ids >= 0
    at = torch.where(here, ids, torch.zeros_like(ids)).to(torch.int64)
    w = torch.where(here, weights, torch.zeros_like(weights))
    if T * k < E:                                      # few choices: each with its own copy of its expert
        pick = at.reshape(-1)
        if c["w"] == "w4":
            up = tuple(t[pick] if t is not None else None for t in s["up"][:3]) + s["up"][3:]
            down = tuple(t[pick] if t is not None else None for t in s["down"][:3]) + s["down"][3:]
            up, down = _dense(up).transpose(-1, -2), _dense(down).transpose(-1, -2)
        else:
            up, down = s["up"][pick].float(), s["down"][pick].float()
        xp = x.unsqueeze(1).expand(T, k, H).reshape(T * k, 1, H)
        gu = (up * xp.unsqueeze(1)).sum(dim=-1)        # [T k, 2, I]
        h = _act(gu[:, 0], c["gate"]) * gu[:, 1]
        y = (down * h.unsqueeze(1)).sum(dim=-1).view(T, k, H)
        return (y * w.unsqueeze(-1)).sum(dim=1).to(torch.bfloat16)
    if c["w"] == "w4":
        up, down = _dense(s["up"]).transpose(-1, -2), _dense(s["down"])
    else:
        up, down = s["up"].float(), s["down"].float().transpose(1, 2)
    gu = torch.matmul(x, up.reshape(E * 2 * I, H).transpose(0, 1)).view(T, E, 2, I)
    share = torch.zeros((T, E), device=x.device).scatter_add_(1, at, w)
    h = _act(gu[:, :, 0], c["gate"]) * gu[:, :, 1] * share.unsqueeze(-1)
    return torch.matmul(h.reshape(T, E * I), down.reshape(E * I, H)).to(torch.bfloat16)


def run(state):
    c = state["case"]
    op = c["op"]
    if own:
        import tile_shape_autotuning_amd as tg
        if op == "gemm":
            return tg.gemm_w4(state["A"], state["B"], state["bias"], act=c["act"], out_dtype=DTYPES[c["out"]])
        if op == "quantize":
            q, values = tg.w4_quantize(state["W"], c["group"], zero_point=c["zero"], scale_dtype=DTYPES[c["scale"]],
                                       values=True)
            out = {"words": q.words, "scales": q.scales, "values": values}
            if c["zero"]:
                out["zeros"] = q.zeros
            return out
        if op == "route":
            return tg.moe_route(state["logits"], c["k"], renorm=c["renorm"])
        if op == "mlp":
            return tg.moe_mlp(state["x"], state["ids"], state["weights"], state["up"], state["down"], gate=c["gate"])
        return tg.moe_layer(state["x"], state["logits"], state["up"], state["down"], c["k"], renorm=c["renorm"],
                            gate=c["gate"])
    if op == "gemm":
        return _plain_gemm(state)
    if op == "quantize":
        return _plain_quantize(state)
    if op == "route":
        return _plain_route(state["logits"], c["k"], c["renorm"])
    if op == "mlp":
        return _plain_mlp(state, state["ids"], state["weights"])
    ids, weights = _plain_route(state["logits"], c["k"], c["renorm"])
    return _plain_mlp(state, ids, weights), ids, weights


# ---------------------------------------------------------------- what a pass cannot do without
def _weight_bytes(K, N, w, group, zero, scale):
    if w == "bf16":
        return 2.0 * K * N
    per_group = {"bf16": 2, "f32": 4}[scale] + (1 if zero else 0)
    return 0.5 * K * N + per_group * _ceil(K, group) * N


def work(case):
    c = case
    size = {"bf16": 2, "f32": 4}
    if c["op"] == "gemm":
        M, N, K = c["M"], c["N"], c["K"]
        b = 2 * M * K + _weight_bytes(K, N, "w4", c["group"], c["zero"], c["scale"]) + size[c["out"]] * M * N
        return {"bytes": b + (4 * N if c["bias"] else 0), "flops": 2.0 * M * N * K}
    if c["op"] == "quantize":
        n = c["E"] * c["K"] * c["N"]
        b = 2 * size[c["dtype"]] * n + c["E"] * _weight_bytes(c["K"], c["N"], "w4", c["group"], c["zero"], c["scale"])
        return {"bytes": b, "flops": 4.0 * n}
    route = c["T"] * c["E"] * (size[c["dtype"]] if c["op"] == "route" else 4) + 8 * c["T"] * c["k"] \
        if c["op"] != "mlp" else 8 * c["T"] * c["k"]
    if c["op"] == "route":
        return {"bytes": route, "flops": 4.0 * c["T"] * c["E"]}
    # the experts that T tokens choose on average, each once
    stays = 1.0 - c.get("away", 0.0)
    active = c["E"] * (1.0 - (1.0 - stays * c["k"] / c["E"]) ** c["T"])
    H, I = c["H"], c["I"]
    per = 2 * _weight_bytes(H, I, c["w"], c["group"], c["zero"], c["scale"]) + \
        _weight_bytes(I, H, c["w"], c["group"], c["zero"], c["scale"])
    return {"bytes": active * per + 4 * c["T"] * H + route, "flops": 6.0 * stays * c["T"] * c["k"] * H * I}


# ---------------------------------------------------------------- the definition, in 64 bits
def _codes64(words, K, N):
    """Codes [K, N] of one matrix, word by word of each row of eight: element (k, n) is looked up where it is stored."""
    k = torch.arange(K, device=words.device).view(K, 1)
    n = torch.arange(N, device=words.device).view(1, N)
    word = words.long()[n // 16, k // 128, (k % 32) // 8 * 16 + n % 16, k % 128 // 32]
    nibble = k % 8 // 2 + 4 * (k % 2)
    return torch.remainder(torch.div(torch.remainder(word, 2 ** 32), 16 ** nibble, rounding_mode="floor"), 16)


def _matrix64(packed, at):
    """Matrix `at` (an index of the leading dimensions) in fp64, [K, N]."""
    words, scales, zeros, K, N, group = packed
    q = _codes64(words[at], K, N).double()
    g = torch.arange(K, device=q.device).view(K, 1) // group
    n = torch.arange(N, device=q.device).view(1, N)
    z = zeros[at][n // 16, g, n % 16].double() if zeros is not None else 8.0
    return scales[at][n // 16, g, n % 16].double() * (q - z)


def _act64(v, act):
    if act == "relu":
        return torch.where(v > 0, v, torch.zeros_like(v))
    if act == "gelu":
        return v * torch.special.erfc(-v / math.sqrt(2.0)) / 2.0
    if act == "silu":
        return v * torch.sigmoid(v)
    return v


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "gemm":
        v = s["A"].double() @ _matrix64(s["B"], ())
        return _act64(v if s["bias"] is None else v + s["bias"].double(), c["act"])
    if c["op"] == "quantize":
        # scales and the values of the codes, group by group; whole numbers are compared with the plain form's
        P, G = _ceil(c["N"], 16), _ceil(c["K"], c["group"])
        scales = torch.zeros((c["E"], P * 16, G), dtype=torch.float64, device="cuda")
        values = torch.empty((c["E"], c["K"], c["N"]), dtype=torch.float64, device="cuda")
        for g in range(G):
            W = s["W"][:, g * c["group"]:(g + 1) * c["group"]].double()
            zero = torch.zeros_like(W[:, 0])
            top, low = torch.maximum(W.amax(1), zero), torch.minimum(W.amin(1), zero)
            if c["zero"]:
                step = (top - low).float().double() / 15.0
            else:
                step = torch.maximum(top, -low) / 7.0
            step = step.float().to(DTYPES[c["scale"]]).double()
            unit = torch.where(step > 0, step, zero + 1.0)
            z = torch.round(-low / unit).clamp(0, 15) if c["zero"] else zero + 8.0
            code = (torch.round(W / unit[:, None]) + z[:, None]).clamp(0, 15)
            values[:, g * c["group"]:(g + 1) * c["group"]] = (code - z[:, None]) * step[:, None]
            scales[:, :c["N"], g] = step
        out = {"words": None, "scales": scales.view(c["E"], P, 16, G).transpose(2, 3), "values": values}
        if c["zero"]:
            out["zeros"] = None
        return out
    if c["op"] != "mlp":
        v = s["logits"].double()
        order = torch.argsort(v, dim=1, descending=True, stable=True)[:, :c["k"]]
        p = torch.softmax(v, dim=1).gather(1, order)
        weights = p / p.sum(1, keepdim=True) if c["renorm"] else p
        if c["op"] == "route":
            return None, weights
        ids = order
    else:
        ids, weights = s["ids"].long(), s["weights"].double()
    x = s["x"].double()
    y = torch.zeros((c["T"], c["H"]), dtype=torch.float64, device="cuda")
    for e in sorted(set(ids.flatten().tolist()) - {-1}):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if c["w"] == "w4":
            g, u, d = _matrix64(s["up"], (e, 0)), _matrix64(s["up"], (e, 1)), _matrix64(s["down"], (e,))
        else:
            g, u, d = s["up"][e, 0].double().t(), s["up"][e, 1].double().t(), s["down"][e].double().t()
        xe = x[t]
        y.index_add_(0, t, ((_act64(xe @ g, c["gate"]) * (xe @ u)) @ d) * weights[t, j].unsqueeze(1))
    return y if c["op"] == "mlp" else (y, None, weights)
