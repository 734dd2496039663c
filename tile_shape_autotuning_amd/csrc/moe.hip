// Mixture-of-experts feed-forward layer for a few tokens:
//   y[t] = sum_j w[t, j] * Wd[e] . (gate(Wg[e] x[t]) * (Wu[e] x[t])),  e = ids[t, j]
// with bf16 weights stored [out][in], or 4-bit weights (w4.hpp).
//
// A few tokens choose a few rows for each expert: the work is the stream of the
// chosen experts' weights, each read once for 16 rows, or 32 where experts have
// more than 8 on average (moe.hpp).  Three kernels:
//   1. gate and up (moe_up.hip): a workgroup takes a share of one chosen
//      expert's panels of 16 columns, gate and up together, gathers that
//      expert's tokens as the rows of its MFMA tiles (panel_stream.hpp) and
//      writes w * gate(g) * u of each to the workspace, in fp32: the layer
//      rounds to fewer bits once, at y;
//   2. down (moe_down.hip): the same over the down projection's panels, whose
//      rows are those fp32 as three bf16 each, all of their 24 bits; fp32 sums
//      of each pair of token and expert to the workspace;
//   3. the sum of each token's pairs, in the order of its choices.
// No atomics: the same call gives the same bits.
//
// Which experts are chosen, and by whom, every workgroup works out itself from
// ids (moe.hpp): a bit for each expert, the i-th set bit is the i-th chosen one.
// An id outside [0, E) adds nothing; an expert named twice by a token counts
// with the sum of both weights.
//
// Bound by the stream: two of eight bf16 experts of 4096 x 14336 for one token
// 82 + 54 + 5 us, 5.8 and 4.4 TB/s in the first two; 64 tokens over 64 experts
// of 2048 x 1408 in 4 bits 52 + 45 + 5 us, 3.9 and 2.2 TB/s (in the second, the
// third part of the hidden state takes 6 us, the expanding and the other two
// products 8, the meeting of the sums 5, and 11 chunks leave two of eight waves
// without a load).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <string>

#include "moe.hpp"

namespace tg {

// ---------------------------------------------------------------- routing
struct RouteParams {
    const void* logits;
    int32_t* ids;
    float* weights;
    int64_t T;
    int E, k, bf16, renorm;
};

// Order-preserving image of a float: NaN above everything, -0 equal to +0.
__device__ __forceinline__ unsigned order_key(float v)
{
    if (v != v)
        return 0xFFFFFFFFu;
    const unsigned b = __float_as_uint(v + 0.0f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ float logit_of(unsigned key)
{
    return key & 0x80000000u ? __uint_as_float(key & 0x7FFFFFFFu) : __uint_as_float(~key);
}

// Lane 63 combines all lanes through the data-parallel primitives (six
// instructions; shuffles through LDS took the routing of 16384 x 256 from 12 to
// 18 us): shifts within rows of 16, then each row's last lane to the next.
template <int CTRL, int ROWS>
__device__ __forceinline__ unsigned moved(unsigned v)
{
    return (unsigned)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xf, false);
}

__device__ __forceinline__ unsigned wave_max(unsigned v)
{
    v = max(v, moved<0x111, 0xf>(v));
    v = max(v, moved<0x112, 0xf>(v));
    v = max(v, moved<0x114, 0xf>(v));
    v = max(v, moved<0x118, 0xf>(v));
    v = max(v, moved<0x142, 0xa>(v));
    v = max(v, moved<0x143, 0xc>(v));
    return (unsigned)__builtin_amdgcn_readlane((int)v, 63);
}

__device__ __forceinline__ float wave_sum(float v)
{
    auto add = [&](unsigned o) { v += __uint_as_float(o); };
    add(moved<0x111, 0xf>(__float_as_uint(v)));
    add(moved<0x112, 0xf>(__float_as_uint(v)));
    add(moved<0x114, 0xf>(__float_as_uint(v)));
    add(moved<0x118, 0xf>(__float_as_uint(v)));
    add(moved<0x142, 0xa>(__float_as_uint(v)));
    add(moved<0x143, 0xc>(__float_as_uint(v)));
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}

// One wave routes one token; lane l holds experts l, l + 64, ...  The k largest
// logits come out one by one (ties: the lowest index); weights are fp32.  A
// row without a finite logit (all -inf) gives experts 0..k-1 with weight 0.
template <int V>
__device__ __forceinline__ void route_token(const RouteParams& p, int64_t t, int lane, int32_t* ids, float* weights)
{
    float v[V];
    unsigned key[V];
    unsigned best = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = lane + 64 * i;
        v[i] = -INFINITY;
        key[i] = 0;                                    // below every logit, NaN included
        if (e < p.E) {
            const int64_t at = t * p.E + e;
            v[i] = p.bf16 ? __uint_as_float((unsigned)static_cast<const unsigned short*>(p.logits)[at] << 16)
                          : static_cast<const float*>(p.logits)[at];
            key[i] = order_key(v[i]);
        }
        best = max(best, key[i]);
    }
    best = wave_max(best);
    const float top = logit_of(best);
    float all = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i)
        all += lane + 64 * i < p.E ? expf(v[i] - top) : 0.0f;
    all = wave_sum(all);
    const bool empty = top == -INFINITY;
    unsigned mine = 0;                                 // lane j keeps the j-th choice
    int mine_id = 0;
    for (int j = 0; j < p.k; ++j) {
        unsigned m = 0;
#pragma unroll
        for (int i = 0; i < V; ++i)
            m = max(m, key[i]);
        m = wave_max(m);
        int id = 0x7FFFFFFF;                           // lowest index that holds the maximum
#pragma unroll
        for (int i = V - 1; i >= 0; --i) {
            const unsigned long long hit = __ballot(key[i] == m);
            if (hit)
                id = 64 * i + __ffsll((long long)hit) - 1;
        }
#pragma unroll
        for (int i = 0; i < V; ++i)
            key[i] = id == lane + 64 * i ? 0u : key[i];
        if (lane == j) {
            mine = m;
            mine_id = id;
        }
    }
    // the key gives the logit back (a zero's sign apart)
    const float e = lane < p.k && !empty ? expf(logit_of(mine) - top) : 0.0f;
    const float sum = p.renorm ? wave_sum(e) : all;
    if (lane < p.k) {
        ids[lane] = mine_id;
        weights[lane] = empty ? 0.0f : e / sum;
    }
}

template <int V>
__global__ void __launch_bounds__(256) moe_route_kernel(RouteParams p)
{
    const int lane = threadIdx.x & 63;
    const int64_t t = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (t < p.T)
        route_token<V>(p, t, lane, p.ids + t * p.k, p.weights + t * p.k);
}

static int launch_route(const RouteParams& p, hipStream_t s)
{
    const dim3 grid((unsigned)ceil_div(p.T, 4)), block(256);
    const int v = (int)ceil_div(p.E, 64);
    if (v <= 1)
        hipLaunchKernelGGL(moe_route_kernel<1>, grid, block, 0, s, p);
    else if (v <= 2)
        hipLaunchKernelGGL(moe_route_kernel<2>, grid, block, 0, s, p);
    else if (v <= 4)
        hipLaunchKernelGGL(moe_route_kernel<4>, grid, block, 0, s, p);
    else if (v <= 8)
        hipLaunchKernelGGL(moe_route_kernel<8>, grid, block, 0, s, p);
    else
        hipLaunchKernelGGL(moe_route_kernel<16>, grid, block, 0, s, p);
    return launched("moe_route launch");
}

// ---------------------------------------------------------------- experts
// y[t] = sum of the token's pairs, in the order of its choices.  Pairs that the
// other kernels left out (no such expert, an expert's second mention) are
// skipped here by the same rule.
__global__ void __launch_bounds__(256) moe_sum_kernel(MoeParams p)
{
    const int t = blockIdx.y, col = blockIdx.x * 256 + threadIdx.x;
    const int32_t* ids = p.ids + t * p.k;
    if (col >= p.H)
        return;
    float v = 0.0f;
    for (int j = 0; j < p.k; ++j) {
        bool first = ids[j] >= 0 && ids[j] < p.E;
        for (int i = 0; i < j; ++i)
            first = first && ids[i] != ids[j];
        if (first)
            v += p.yp[((int64_t)t * p.k + j) * p.H + col];
    }
    p.y[(int64_t)t * p.H + col] = f32_to_bf16_rne(v);
}

static int launch_pass(const MoeParams& p, const tg_weight& up, const tg_weight& down, hipStream_t s)
{
    int st = launch_up(p, up, s);
    if (st != TG_OK || (st = launch_down(p, down, s)) != TG_OK)
        return st;
    hipLaunchKernelGGL(moe_sum_kernel, dim3((unsigned)ceil_div(p.H, 256), (unsigned)p.T), dim3(256), 0, s, p);
    return launched("moe sum launch");
}

static ExpertStack stack_of(const tg_weight& w, int64_t K, int64_t N)
{
    ExpertStack s{};
    s.panels = (int)ceil_div(N, 16);
    if (w.format == TG_W_W4) {
        s.w4 = view_w4(w, K);
        s.words = (int64_t)s.panels * s.w4.chunks * 64;
        s.scales = (int64_t)s.panels * s.w4.groups * 16;
    } else {
        s.bf16 = static_cast<const unsigned short*>(w.data);
    }
    return s;
}

static int check_route(int64_t T, int64_t E, int k)
{
    if (T < 0 || E < 1 || k < 1 || k > E)
        return set_error(TG_E_INVAL, "T must be >= 0, 1 <= k <= E");
    if (E > kMaxExperts || k > kMaxChoices || T > (int64_t)1 << 24)
        return set_error(TG_E_UNSUPPORTED, "at most 1024 experts, 16 choices and 2^24 tokens");
    return TG_OK;
}

static int check_logits(const void* logits, int logits_dtype, const int32_t* ids, const float* weights)
{
    if (logits_dtype != TG_F32 && logits_dtype != TG_BF16)
        return set_error(TG_E_INVAL, "logits are fp32 or bf16");
    if (!logits || !ids || !weights || ((uintptr_t)logits & (logits_dtype == TG_F32 ? 3u : 1u)) ||
        (((uintptr_t)ids | (uintptr_t)weights) & 3u))
        return set_error(TG_E_INVAL, "logits, ids and weights must be given, aligned to their elements");
    return TG_OK;
}

// h, then yp
static size_t workspace_of(int64_t T, int64_t H, int64_t I, int k)
{
    return (size_t)std::min<int64_t>(T, kTokens) * (size_t)k * (size_t)(ceil_div(I, 16) * 16 + H) * 4;
}

// everything but the choices
static int check_mlp(int64_t T, int64_t H, int64_t I, int64_t E, int k, const void* x, const tg_weight* up,
                     const tg_weight* down, void* y, int gate, void* ws, size_t ws_bytes)
{
    int st = check_route(T, E, k);
    if (st != TG_OK)
        return st;
    if (H < 1 || I < 1)
        return set_error(TG_E_INVAL, "H and I must be >= 1");
    if (H > 65536 || I > 65536)
        return set_error(TG_E_UNSUPPORTED, "H and I are at most 65536");
    if (gate != TG_GATE_SILU && gate != TG_GATE_GELU)
        return set_error(TG_E_INVAL, "unknown gate activation");
    if (T == 0)
        return TG_OK;
    if ((st = check_weight(up, "gate_up")) != TG_OK || (st = check_weight(down, "down")) != TG_OK)
        return st;
    if (!x || !y || (((uintptr_t)x | (uintptr_t)y) & 1u))
        return set_error(TG_E_INVAL, "x and y must be given, aligned to their elements");
    if (!ws || ((uintptr_t)ws & 15u) || ws_bytes < workspace_of(T, H, I, k))
        return set_error(TG_E_INVAL, "the workspace must be 16-byte aligned and hold tg_moe_workspace_bytes() bytes");
    return TG_OK;
}

static MoeParams params_of(int64_t H, int64_t I, int64_t E, int k, const tg_weight* up, const tg_weight* down, int gate,
                           void* ws)
{
    MoeParams p{};
    p.h = static_cast<float*>(ws);
    p.up = stack_of(*up, H, I);
    p.down = stack_of(*down, I, H);
    p.stride = ceil_div(I, 16) * 16;
    p.E = (int)E;
    p.k = k;
    p.H = (int)H;
    p.I = (int)I;
    p.gelu = gate == TG_GATE_GELU;
    return p;
}

static int run_mlp(MoeParams p, int64_t T, const void* x, const int32_t* ids, const float* weights, void* y,
                   const tg_weight* up, const tg_weight* down)
{
    // passes share the workspace: the stream orders them
    for (int64_t t = 0; t < T; t += kTokens) {
        p.T = (int)std::min<int64_t>(kTokens, T - t);
        p.yp = p.h + (int64_t)p.T * p.k * p.stride;
        p.x = static_cast<const unsigned short*>(x) + t * p.H;
        p.ids = ids + t * p.k;
        p.weights = weights + t * p.k;
        p.y = static_cast<unsigned short*>(y) + t * p.H;
        const int st = launch_pass(p, *up, *down, current_stream());
        if (st != TG_OK)
            return st;
    }
    return TG_OK;
}

static RouteParams route_of(int64_t T, int64_t E, int k, const void* logits, int dtype, int renorm, int32_t* ids,
                            float* weights)
{
    RouteParams r{};
    r.logits = logits;
    r.ids = ids;
    r.weights = weights;
    r.T = T;
    r.E = (int)E;
    r.k = k;
    r.bf16 = dtype == TG_BF16;
    r.renorm = renorm != 0;
    return r;
}

}  // namespace tg

using namespace tg;

extern "C" {

int tg_moe_route(int64_t T, int64_t E, int k, const void* logits, int dtype, int renorm, int32_t* ids, float* weights)
{
    int st = check_route(T, E, k);
    if (st != TG_OK || T == 0)
        return st;
    if ((st = check_logits(logits, dtype, ids, weights)) != TG_OK)
        return st;
    if (!have_device())
        return set_error(TG_E_UNSUPPORTED, "no HIP device");
    return launch_route(route_of(T, E, k, logits, dtype, renorm, ids, weights), current_stream());
}

int tg_moe_workspace_bytes(int64_t T, int64_t H, int64_t I, int k, size_t* bytes)
{
    if (!bytes || T < 0 || H < 1 || H > 65536 || I < 1 || I > 65536 || k < 1 || k > kMaxChoices)
        return set_error(TG_E_INVAL, "bad size, or bytes is NULL");
    *bytes = workspace_of(T, H, I, k);
    return TG_OK;
}

int tg_moe_mlp(int64_t T, int64_t H, int64_t I, int64_t E, int k, const void* x, const int32_t* ids,
               const float* weights, const tg_weight* gate_up, const tg_weight* down, void* y, int gate,
               void* workspace, size_t workspace_bytes)
{
    const int st = check_mlp(T, H, I, E, k, x, gate_up, down, y, gate, workspace, workspace_bytes);
    if (st != TG_OK || T == 0)
        return st;
    if (!ids || !weights || (((uintptr_t)ids | (uintptr_t)weights) & 3u))
        return set_error(TG_E_INVAL, "ids and weights must be given, 4-byte aligned");
    if (!have_device())
        return set_error(TG_E_UNSUPPORTED, "no HIP device");
    return run_mlp(params_of(H, I, E, k, gate_up, down, gate, workspace), T, x, ids, weights, y, gate_up, down);
}

int tg_moe_layer(int64_t T, int64_t H, int64_t I, int64_t E, int k, const void* x, const void* logits,
                 int logits_dtype, int renorm, const tg_weight* gate_up, const tg_weight* down, void* y, int32_t* ids,
                 float* weights, int gate, void* workspace, size_t workspace_bytes)
{
    int st = check_mlp(T, H, I, E, k, x, gate_up, down, y, gate, workspace, workspace_bytes);
    if (st != TG_OK || T == 0)
        return st;
    if ((st = check_logits(logits, logits_dtype, ids, weights)) != TG_OK)
        return st;
    if (!have_device())
        return set_error(TG_E_UNSUPPORTED, "no HIP device");
    st = launch_route(route_of(T, E, k, logits, logits_dtype, renorm, ids, weights), current_stream());
    if (st != TG_OK)
        return st;
    return run_mlp(params_of(H, I, E, k, gate_up, down, gate, workspace), T, x, ids, weights, y, gate_up, down);
}

}  // extern "C"
