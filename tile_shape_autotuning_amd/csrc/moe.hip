// Mixture-of-experts feed-forward layer for a few tokens:
//   y[t] = sum_j w[t, j] * Wd[e] . (gate(Wg[e] x[t]) * (Wu[e] x[t])),  e = ids[t, j]
// with bf16 weights stored [out][in], or 4-bit weights (w4.hpp).
//
// A few tokens choose a few rows for each expert: the work is the stream of the
// chosen experts' weights, each read once.  Two kernels:
//   1. gate and up: a workgroup owns 16 columns of one chosen expert's gate and
//      up matrices, gathers that expert's tokens as the rows of its MFMA tiles
//      and writes w * gate(g) * u of each to the workspace, as the sum of two
//      bf16 (16 bits of mantissa, so that the layer rounds once, at y);
//   2. down: a workgroup owns 16 columns of y and runs through the chosen
//      experts one after the other, as one product whose reduction is the
//      experts' hidden widths end to end, cut evenly among its waves.  A wave
//      adds an expert's rows into its own fp32 tile of tokens in LDS; the
//      waves' tiles are added in wave order.  No atomics: the same call gives
//      the same bits.
// Which experts are chosen, and by whom, every workgroup works out itself from
// ids: a bit for each expert, the i-th set bit is the i-th chosen one.  An id
// outside [0, E) adds nothing; an expert named twice by a token counts with
// the sum of both weights.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <string>
#include <type_traits>

#include "panel_stream.hpp"
#include "w4.hpp"
#include "w4_host.hpp"

namespace tg {

static constexpr int kMaxExperts = 1024, kMaxChoices = 16;
static constexpr int kTokens = 64;                     // tokens of one pass: a lane each
static constexpr int kExpertWords = kMaxExperts / 32;

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

__device__ __forceinline__ unsigned wave_max(unsigned v)
{
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1)
        v = max(v, (unsigned)__shfl_xor((int)v, off));
    return v;
}

__device__ __forceinline__ float wave_sum(float v)
{
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1)
        v += __shfl_xor(v, off);
    return v;
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
    const float top = best & 0x80000000u ? __uint_as_float(best & 0x7FFFFFFFu) : __uint_as_float(~best);
    float all = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i)
        all += lane + 64 * i < p.E ? expf(v[i] - top) : 0.0f;
    all = wave_sum(all);
    const bool empty = top == -INFINITY;
    float mine = 0.0f, chosen = 0.0f;                  // lane j keeps the j-th choice
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
        float l = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if (id == lane + 64 * i) {
                l = v[i];
                key[i] = 0;
            }
        }
        l = __shfl(l, id & 63);
        const float e = empty ? 0.0f : expf(l - top);
        chosen += e;
        if (lane == j) {
            mine = e;
            mine_id = id;
        }
    }
    if (lane < p.k) {
        ids[lane] = mine_id;
        weights[lane] = empty ? 0.0f : mine / (p.renorm ? chosen : all);
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
// A stack of matrices [K -> N], one for each expert or two.
struct ExpertStack {
    const unsigned short* bf16;                        // [.., N, K]
    W4View w4;                                         // matrix 0 of the stack
    int64_t words, scales;                             // elements of w4.words / w4.scales from one matrix to the next
    int N, K, panels;
};

__device__ __forceinline__ W4View matrix(const ExpertStack& s, int64_t i)
{
    W4View v = s.w4;
    v.words += i * s.words;
    v.scales = static_cast<const char*>(v.scales) + i * s.scales * (v.scale_f32 ? 4 : 2);
    if (v.zeros)
        v.zeros += i * s.scales;
    return v;
}

struct MoeParams {
    const unsigned short* x;                           // [T][H]
    const int32_t* ids;                                // [T][k]
    const float* weights;
    unsigned* h;                                       // [T k][stride], two bf16: high half + low half
    float* yp;                                         // [T k][H], each pair's part of y
    unsigned short* y;                                 // [T][H]
    ExpertStack up, down;
    int64_t stride;                                    // I rounded up to 16
    int T, E, k, H, I, gelu;
    int up_per, up_blocks, down_per, down_blocks;      // panels a workgroup, blocks of the reduction
};

// The tokens that chose expert e, one a lane: lane r holds the r-th one's pair
// index t k + j (its first choice of e) and the sum of its weights for e.
// Returns how many.
__device__ __forceinline__ int rows_of(const int* ids, const float* weights, int T, int k, int e, int lane, int& pair,
                                       float& weight)
{
    int first = -1;
    float w = 0.0f;
    if (lane < T)
        for (int j = k - 1; j >= 0; --j)
            if (ids[lane * k + j] == e) {
                first = lane * k + j;
                if (weights)
                    w += weights[first];
            }
    const unsigned long long has = __ballot(first >= 0);
    const int rank = __popcll(has & ((1ull << lane) - 1));
    // lanes without a row send theirs past the rows
    const int to = 4 * (first >= 0 ? rank : __popcll(has) + (lane - rank));
    pair = __builtin_amdgcn_ds_permute(to, first);
    weight = __int_as_float(__builtin_amdgcn_ds_permute(to, __float_as_int(w)));
    return __popcll(has);
}

// Marks the chosen experts (all threads), copies ids to LDS; ends in a barrier.
__device__ __forceinline__ void mark_experts(const int32_t* ids, int n, int E, int* copy, unsigned* bits)
{
    for (int i = threadIdx.x; i < kExpertWords; i += blockDim.x)
        bits[i] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
        const int e = ids[i];
        copy[i] = e;
        if (e >= 0 && e < E)
            atomicOr(&bits[e >> 5], 1u << (e & 31));
    }
    __syncthreads();
}

// The chosen experts as a wave sees them: lane i < 32 holds bits of experts
// 32 i .. 32 i + 31 and how many are chosen up to there.
struct Chosen {
    unsigned word;
    int upto, count;
    __device__ __forceinline__ Chosen(const unsigned* bits, int lane)
    {
        word = lane < kExpertWords ? bits[lane] : 0u;
        upto = __popc(word);
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
            const int o = __shfl_up(upto, off);
            if (lane >= off)
                upto += o;
        }
        count = __builtin_amdgcn_readlane(upto, 63);
    }
    // i-th chosen expert, i < count
    __device__ __forceinline__ int expert(int i) const
    {
        const int at = __ffsll((long long)__ballot(upto > i)) - 1;
        unsigned w = __builtin_amdgcn_readlane(word, at);
        int skip = i - (__builtin_amdgcn_readlane(upto, at) - __popc(w));
        for (; skip > 0; --skip)
            w &= w - 1;
        return at * 32 + __ffs((int)w) - 1;
    }
};

__device__ __forceinline__ float gated(float g, float u, int gelu)
{
    return (gelu ? gelu_erf(g) : g / (1.0f + __expf(-g))) * u;
}

// The wave's share of a workgroup's work on one chosen expert: a stream of the
// expert's panels past MT x 16 of its rows (panel_stream.hpp).
struct Share {
    int expert, rows, pair;                            // lane r: the r-th row's pair
    float weight;
};

// False if there is no `slot`-th chosen expert.
__device__ __forceinline__ bool share_of(const MoeParams& p, int slot, int* ids, unsigned* bits, const float* weights,
                                         int lane, Share& s)
{
    mark_experts(p.ids, p.T * p.k, p.E, ids, bits);
    const Chosen chosen(bits, lane);
    if (slot >= chosen.count)
        return false;
    s.expert = chosen.expert(slot);
    s.rows = rows_of(ids, weights, p.T, p.k, s.expert, lane, s.pair, s.weight);
    return true;
}

template <bool W4F, bool ZERO, int MT, int W, int CW, int GS, bool VEC>
__global__ void __launch_bounds__(64 * W) moe_up_kernel(MoeParams p)
{
    using S = PanelStream<W4F, ZERO, MT, 2, 1, W, CW, GS, 32>;
    __shared__ f32x4_t red[S::RED], mid[S::MID];
    __shared__ int ids[kTokens * kMaxChoices];
    __shared__ unsigned bits[kExpertWords];
    extern __shared__ f32x4_t part[];                  // [p.per][MT][2][64] if there is more than one block
    S s(red, mid, p.up.w4.scale_f32);
    const int lane = s.lane, l16 = lane & 15, kq = lane >> 4;
    Share e;
    if (!share_of(p, blockIdx.y, ids, bits, p.weights, lane, e))
        return;
    const int panel0 = blockIdx.x * p.up_per;
    const int n = min(p.up_per, p.up.panels - panel0);
    const int chunks = (p.H + 127) / 128;
    W4View v[2];
    const unsigned short* wb[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        if constexpr (W4F)
            v[j] = matrix(p.up, 2 * (int64_t)e.expert + j);
        else
            wb[j] = p.up.bf16 + (2 * (int64_t)e.expert + j) * p.I * p.H;
    }

    for (int r0 = 0; r0 < e.rows; r0 += 16 * MT) {
        auto rows = [&](int block) {
            const int c0 = (block * W + s.wave) * CW;
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const int r = r0 + 16 * m + l16;
                const unsigned short* x = p.x + (int64_t)(__shfl(e.pair, r & 63) / p.k) * p.H;
#pragma unroll
                for (int i = 0; i < CW; ++i) {
#pragma unroll
                    for (int t = 0; t < 4; ++t)
                        s.a[i][m][0][t] = splat4(0);
                    if (r < e.rows && c0 + i < chunks)
                        load_chunk(s.a[i][m][0], x, c0 + i, kq, p.H);
                }
            }
        };
        auto load = [&](int block, int index, typename S::Words& b, bool some) {
            const int c0 = (block * W + s.wave) * CW;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                if constexpr (W4F)
                    s.load_w4(b, j, v[j], panel0 + index, c0, some);
                else
                    s.template load_bf16<VEC>(b, j, wb[j], p.I, p.H, panel0 + index, c0, some);
            }
        };
        auto done = [&](int block, int index, int m, f32x4_t (&sum)[2]) {
            f32x4_t* held = part + (index * MT + m) * 128 + lane;
            if (block > 0) {
                sum[0] += held[0];
                sum[1] += held[64];
            }
            if (block + 1 < p.up_blocks) {
                held[0] = sum[0];
                held[64] = sum[1];
                return;
            }
            const int at = fresh(lane), col = (panel0 + index) * 16 + (at & 15);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = r0 + 16 * m + (at >> 4) * 4 + r;
                const int to = __shfl(e.pair, row & 63);
                const float w = __shfl(e.weight, row & 63);
                if (row >= e.rows)
                    continue;
                // columns past I stay zero for the second kernel
                const float hv = col < p.I ? w * gated(sum[0][r], sum[1][r], p.gelu) : 0.0f;
                const unsigned short hi = f32_to_bf16_rne(hv);
                const float rest = hv - __uint_as_float((unsigned)hi << 16);
                // an infinity or NaN stays one: its rest is no number
                const unsigned short lo = (hi & 0x7F80u) != 0x7F80u ? f32_to_bf16_rne(rest) : (unsigned short)0;
                p.h[(int64_t)to * p.stride + col] = (unsigned)hi << 16 | lo;
            }
        };
        s.run(p.up_blocks, n, rows, load, done);
    }
}

template <bool W4F, bool ZERO, int MT, int W, int CW, int GS, bool VEC>
__global__ void __launch_bounds__(64 * W) moe_down_kernel(MoeParams p)
{
    using S = PanelStream<W4F, ZERO, MT, 1, 2, W, CW, GS, 32>;
    __shared__ f32x4_t red[S::RED], mid[S::MID];
    __shared__ int ids[kTokens * kMaxChoices];
    __shared__ unsigned bits[kExpertWords];
    extern __shared__ f32x4_t part[];                  // [p.per][MT][64] if there is more than one block
    S s(red, mid, p.down.w4.scale_f32);
    const int lane = s.lane, l16 = lane & 15, kq = lane >> 4;
    Share e;
    if (!share_of(p, blockIdx.y, ids, bits, nullptr, lane, e))
        return;
    const int panel0 = blockIdx.x * p.down_per;
    const int n = min(p.down_per, p.down.panels - panel0);
    W4View v;
    const unsigned short* wb = nullptr;
    if constexpr (W4F)
        v = matrix(p.down, e.expert);
    else
        wb = p.down.bf16 + (int64_t)e.expert * p.H * p.I;

    for (int r0 = 0; r0 < e.rows; r0 += 16 * MT) {
        auto rows = [&](int block) {
            const int c0 = (block * W + s.wave) * CW;
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const int r = r0 + 16 * m + l16;
                const unsigned* h = p.h + (int64_t)__shfl(e.pair, r & 63) * p.stride;
#pragma unroll
                for (int i = 0; i < CW; ++i)
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
                        const int64_t k = (int64_t)(c0 + i) * 128 + 32 * t + 8 * kq;
                        u32x4_t h0 = splat4(0), h1 = splat4(0);
                        if (r < e.rows && k < p.stride) {
                            h0 = *reinterpret_cast<const u32x4_t*>(h + k);
                            h1 = *reinterpret_cast<const u32x4_t*>(h + k + 4);
                        }
#pragma unroll
                        for (int d = 0; d < 4; ++d) {
                            const unsigned x0 = d < 2 ? h0[2 * d] : h1[2 * d - 4];
                            const unsigned x1 = d < 2 ? h0[2 * d + 1] : h1[2 * d - 3];
                            s.a[i][m][0][t][d] = __builtin_amdgcn_perm(x1, x0, 0x07060302u);
                            s.a[i][m][1][t][d] = __builtin_amdgcn_perm(x1, x0, 0x05040100u);
                        }
                    }
            }
        };
        auto load = [&](int block, int index, typename S::Words& b, bool some) {
            const int c0 = (block * W + s.wave) * CW;
            if constexpr (W4F)
                s.load_w4(b, 0, v, panel0 + index, c0, some);
            else
                s.template load_bf16<VEC>(b, 0, wb, p.H, p.I, panel0 + index, c0, some);
        };
        auto done = [&](int block, int index, int m, f32x4_t (&sum)[1]) {
            f32x4_t* held = part + (index * MT + m) * 64 + lane;
            if (block > 0)
                sum[0] += *held;
            if (block + 1 < p.down_blocks) {
                *held = sum[0];
                return;
            }
            const int at = fresh(lane), col = (panel0 + index) * 16 + (at & 15);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = r0 + 16 * m + (at >> 4) * 4 + r;
                const int from = __shfl(e.pair, row & 63);
                if (row < e.rows && col < p.H)
                    p.yp[(int64_t)from * p.H + col] = sum[0][r];
            }
        };
        s.run(p.down_blocks, n, rows, load, done);
    }
}

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

// Panels of a workgroup: two workgroups a compute unit over all chosen experts
// (at most), as far as the sums of the reduction's earlier blocks find room in
// LDS beside the `used` bytes.
static int panels_per(int panels, int slots, int blocks, size_t used, size_t panel_bytes)
{
    int64_t per = std::max<int64_t>(1, (int64_t)panels * slots / (2 * kCus));
    if (blocks > 1)
        per = std::min<int64_t>(per, (int64_t)((kLdsBytes - used) / panel_bytes));
    return (int)std::min<int64_t>(per, panels);
}

template <bool W4F, bool ZERO, int MT, int CW, int GS, bool VEC>
static void run_up(MoeParams p, hipStream_t s)
{
    constexpr int W = 8;
    using S = PanelStream<W4F, ZERO, MT, 2, 1, W, CW, GS, 32>;
    constexpr size_t used = (S::RED + S::MID) * 16 + (kTokens * kMaxChoices + kExpertWords) * 4;
    static_assert(used + MT * 2048 <= kLdsBytes, "LDS");
    const int slots = std::min(p.E, p.T * p.k);
    p.up_blocks = (int)ceil_div(ceil_div(p.H, 128), W * CW);
    p.up_per = panels_per(p.up.panels, slots, p.up_blocks, used, MT * 2048);
    const size_t lds = p.up_blocks > 1 ? (size_t)p.up_per * MT * 2048 : 0;
    const dim3 grid((unsigned)ceil_div(p.up.panels, p.up_per), (unsigned)slots);
    hipLaunchKernelGGL((moe_up_kernel<W4F, ZERO, MT, W, CW, GS, VEC>), grid, dim3(64 * W), lds, s, p);
}

template <bool W4F, bool ZERO, int MT, int CW, int GS, bool VEC>
static void run_down(MoeParams p, hipStream_t s)
{
    constexpr int W = 8;
    using S = PanelStream<W4F, ZERO, MT, 1, 2, W, CW, GS, 32>;
    constexpr size_t used = (S::RED + S::MID) * 16 + (kTokens * kMaxChoices + kExpertWords) * 4;
    static_assert(used + MT * 1024 <= kLdsBytes, "LDS");
    const int slots = std::min(p.E, p.T * p.k);
    p.down_blocks = (int)ceil_div(ceil_div(p.I, 128), W * CW);
    p.down_per = panels_per(p.down.panels, slots, p.down_blocks, used, MT * 1024);
    const size_t lds = p.down_blocks > 1 ? (size_t)p.down_per * MT * 1024 : 0;
    const dim3 grid((unsigned)ceil_div(p.down.panels, p.down_per), (unsigned)slots);
    hipLaunchKernelGGL((moe_down_kernel<W4F, ZERO, MT, W, CW, GS, VEC>), grid, dim3(64 * W), lds, s, p);
}

// Picks the instantiation for a weight: f.template go<W4F, ZERO, MT, CW, GS, VEC>(p, s).
template <class F>
static void dispatch(const tg_weight& w, int T, int64_t K, const MoeParams& p, hipStream_t s)
{
    const bool many = T > 16;
    if (w.format == TG_W_W4) {
        const bool two = K > 1024;                     // chunks a wave
        auto pick = [&](auto zero, auto gs) {
            constexpr bool Z = decltype(zero)::value;
            constexpr int G = decltype(gs)::value;
            if (many)
                two ? F::template go<true, Z, 2, 2, G, true>(p, s) : F::template go<true, Z, 2, 1, G, true>(p, s);
            else
                two ? F::template go<true, Z, 1, 2, G, true>(p, s) : F::template go<true, Z, 1, 1, G, true>(p, s);
        };
        using One = std::integral_constant<int, 1>;
        using Four = std::integral_constant<int, 4>;
        if (w.zeros)
            w.group >= 128 ? pick(std::true_type{}, Four{}) : pick(std::true_type{}, One{});
        else
            w.group >= 128 ? pick(std::false_type{}, Four{}) : pick(std::false_type{}, One{});
    } else if (K % 8 == 0) {
        many ? F::template go<false, false, 2, 1, 4, true>(p, s) : F::template go<false, false, 1, 1, 4, true>(p, s);
    } else {
        many ? F::template go<false, false, 2, 1, 4, false>(p, s) : F::template go<false, false, 1, 1, 4, false>(p, s);
    }
}

struct Up {
    template <bool W4F, bool ZERO, int MT, int CW, int GS, bool VEC>
    static void go(const MoeParams& p, hipStream_t s) { run_up<W4F, ZERO, MT, CW, GS, VEC>(p, s); }
};
struct Down {
    template <bool W4F, bool ZERO, int MT, int CW, int GS, bool VEC>
    static void go(const MoeParams& p, hipStream_t s) { run_down<W4F, ZERO, MT, CW, GS, VEC>(p, s); }
};

static int launch_pass(const MoeParams& p, const tg_weight& up, const tg_weight& down, hipStream_t s)
{
    dispatch<Up>(up, p.T, p.H, p, s);
    int st = launched("moe gate and up launch");
    if (st != TG_OK)
        return st;
    dispatch<Down>(down, p.T, p.I, p, s);
    if ((st = launched("moe down launch")) != TG_OK)
        return st;
    hipLaunchKernelGGL(moe_sum_kernel, dim3((unsigned)ceil_div(p.H, 256), (unsigned)p.T), dim3(256), 0, s, p);
    return launched("moe sum launch");
}

static ExpertStack stack_of(const tg_weight& w, int64_t K, int64_t N)
{
    ExpertStack s{};
    s.N = (int)N;
    s.K = (int)K;
    s.panels = (int)ceil_div(N, 16);
    if (w.format == TG_W_W4) {
        s.w4 = view_w4(w, K, N, 0);
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
    if ((st = check_weight(up, H, I, "gate_up")) != TG_OK || (st = check_weight(down, I, H, "down")) != TG_OK)
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
    p.h = static_cast<unsigned*>(ws);
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
        p.yp = reinterpret_cast<float*>(p.h + (int64_t)p.T * p.k * p.stride);
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
