// What the kernels of the expert layer share (moe.hip has the overview): the
// call's parameters, how a workgroup finds its expert and that expert's tokens,
// and how the work is divided.
#pragma once

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "panel_stream.hpp"
#include "w4_host.hpp"

namespace tg {

constexpr int kMaxExperts = 1024, kMaxChoices = 16;
constexpr int kTokens = 64;                     // tokens of one pass: a lane each
constexpr int kExpertWords = kMaxExperts / 32;

// A stack of matrices [K -> N], one for each expert or two.
struct ExpertStack {
    const unsigned short* bf16;                        // [.., N, K]
    W4View w4;                                         // matrix 0 of the stack
    int64_t words, scales;                             // elements of w4.words / w4.scales from one matrix to the next
    int panels;
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
    float* h;                                          // [T k][stride]
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

// Steps whose words are held or on their way: 4-bit words are small (gate and up
// of 64 experts of 2048 x 1408: 49 us with four, 52 with two).
template <bool W4F>
constexpr int kDepth = W4F ? 4 : 2;

// Panels of a workgroup, so that the workgroups of all the experts that T
// tokens choose on average run at once, `resident` on a compute unit: one
// round of equal shares (of two and a third rounds the last third idles: gate
// and up of two 4096 x 14336 experts 99 us instead of 84).  `used`,
// `panel_bytes`: LDS, and what a panel holds there between blocks of the
// reduction.
inline int panels_per(int panels, const MoeParams& p, int resident, int blocks, size_t used, size_t panel_bytes)
{
    const double miss = 1.0 - (double)p.k / p.E;
    const double chosen = std::min<double>((double)p.T * p.k, p.E * (1.0 - std::pow(miss, p.T)));
    const double each = (double)compute_units() * resident / std::max(1.0, chosen);
    int64_t per = ceil_div(panels, std::max(1, (int)std::min<double>(each, panels)));
    if (blocks > 1)
        per = std::min<int64_t>(per, (int64_t)((kLdsBytes - used) / panel_bytes));
    return (int)std::min<int64_t>(per, panels_in_reach((std::max(p.H, p.I) + 127) / 128));
}

// Workgroups of a kernel that a compute unit holds.
template <class Kernel>
inline int resident_on_cu(Kernel kernel, int threads)
{
    int n = 0;
    if (hipOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, 0) != hipSuccess) {
        (void)hipGetLastError();
        return 1;
    }
    return std::max(n, 1);
}

// F::go<W4F, ZERO, MT, CW, GS, VEC>(p, s) for a weight whose reduction has K
// rows; `vec`: what is read along it comes in aligned 16 bytes.  Two row tiles
// where an expert has more than 8 rows on average: with fewer, more than 16
// are rare, and their panels stream by once more for each 16.  Two chunks a
// wave where eight waves have them (F::kMany with two row tiles).  (16 waves of
// one chunk: the same within 5 % where there are 16 chunks, 33 us instead of 20
// where there are 8.)
template <class F>
static void by_weight(const tg_weight& w, int64_t K, bool vec, const MoeParams& p, hipStream_t s)
{
    const bool many = p.T > 16 && p.T * p.k > 8 * p.E, two = K > 1024;
    auto rest = [&](auto w4f, auto zero, auto gs, auto v) {
        constexpr bool Q = decltype(w4f)::value, Z = decltype(zero)::value, V = decltype(v)::value;
        constexpr int G = decltype(gs)::value;
        if constexpr (V) {
            if (two) {
                many ? F::template go<Q, Z, 2, F::kMany, G, V>(p, s) : F::template go<Q, Z, 1, 2, G, V>(p, s);
                return;
            }
        }
        many ? F::template go<Q, Z, 2, 1, G, V>(p, s) : F::template go<Q, Z, 1, 1, G, V>(p, s);
    };
    using One = std::integral_constant<int, 1>;
    using Two = std::integral_constant<int, 2>;
    using Four = std::integral_constant<int, 4>;
    auto by_vec = [&](auto w4f, auto zero, auto gs) {
        vec ? rest(w4f, zero, gs, std::true_type{}) : rest(w4f, zero, gs, std::false_type{});
    };
    auto by_group = [&](auto zero) {
        w.group >= 128 ? by_vec(std::true_type{}, zero, Four{})
                       : w.group == 64 ? by_vec(std::true_type{}, zero, Two{}) : by_vec(std::true_type{}, zero, One{});
    };
    if (w.format == TG_W_W4)
        w.zeros ? by_group(std::true_type{}) : by_group(std::false_type{});
    else
        by_vec(std::false_type{}, std::false_type{}, Four{});
}

int launch_up(const MoeParams& p, const tg_weight& w, hipStream_t s);       // moe_up.hip
int launch_down(const MoeParams& p, const tg_weight& w, hipStream_t s);     // moe_down.hip

}  // namespace tg
