// Tokens in the order of their experts, and back: the sort of (token, choice)
// pairs, the copy of rows into that order, the weighted sum that brings them
// back, and its gradients.  Everything here is bound by memory, but for the
// sort's latency.  The same call gives the same bits: the only atomics are counts
// of pairs in LDS, whole numbers whose order does not matter.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <string>

#include "kernels/common.hpp"
#include "row_piece.hpp"
#include "w4_host.hpp"

namespace tg {

constexpr int kOrderExperts = 1024, kOrderChoices = 16;
constexpr int64_t kUnits = (int64_t)1 << 31;           // pieces of all rows of a call
constexpr int64_t kOrderTokens = (int64_t)1 << 24, kOrderWidth = (int64_t)1 << 24;

static unsigned grid_of(int64_t n) { return (unsigned)std::min<int64_t>(n, 1 << 20); }

// ---------------------------------------------------------------- sort
// Few pairs: a workgroup takes one expert, counts the pairs of the experts before
// it, then walks the pairs in order and numbers its own.  The last workgroup
// takes the pairs without an expert, and the rows behind the last one.
__global__ void __launch_bounds__(256) moe_sort_few_kernel(const int32_t* ids, int n, int E, int32_t* position,
                                                           int32_t* source, int32_t* offsets)
{
    __shared__ int part[4];
    const int e = blockIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int before = 0;
    for (int i = threadIdx.x; i < n; i += 256)
        before += ids[i] >= 0 && ids[i] < e;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1)
        before += __shfl_xor(before, off);
    if (lane == 0)
        part[wave] = before;
    __syncthreads();
    int at = part[0] + part[1] + part[2] + part[3];
    if (threadIdx.x == 0)
        offsets[e] = at;
    if (e == E) {
        for (int i = threadIdx.x; i < n; i += 256) {
            if (ids[i] < 0 || ids[i] >= E)
                position[i] = -1;
            if (i >= at)
                source[i] = -1;
        }
        return;
    }
    for (int i0 = 0; i0 < n; i0 += 256) {
        const int i = i0 + threadIdx.x;
        const bool mine = i < n && ids[i] == e;
        const unsigned long long has = __ballot(mine);
        __syncthreads();
        if (lane == 0)
            part[wave] = __popcll(has);
        __syncthreads();
        int to = at + __popcll(has & ((1ull << lane) - 1));
        for (int w = 0; w < wave; ++w)
            to += part[w];
        if (mine) {
            position[i] = to;
            source[to] = i;
        }
        at += part[0] + part[1] + part[2] + part[3];
    }
}

// Many pairs: blocks of `per` pairs are counted by expert, then every block adds
// up the counts of all blocks (for the experts' first rows) and of those before
// it, and numbers its own pairs, 64 of a wave at a time.
struct SortParams {
    const int32_t* ids;
    int32_t *position, *source, *offsets, *counts;     // counts: [blocks][E]
    int n, E, per, blocks;
};

constexpr int kSortThreads = 1024, kSortWaves = kSortThreads / 64;

__global__ void __launch_bounds__(kSortThreads) moe_count_kernel(SortParams p)
{
    __shared__ int count[kOrderExperts];
    for (int e = threadIdx.x; e < p.E; e += kSortThreads)
        count[e] = 0;
    __syncthreads();
    const int first = blockIdx.x * p.per, last = min(p.n, first + p.per);
    for (int i = first + threadIdx.x; i < last; i += kSortThreads) {
        const int e = p.ids[i];
        if ((unsigned)e < (unsigned)p.E)
            atomicAdd(&count[e], 1);                   // sums of ones: any order
    }
    __syncthreads();
    for (int e = threadIdx.x; e < p.E; e += kSortThreads)
        p.counts[blockIdx.x * p.E + e] = count[e];
}

__global__ void __launch_bounds__(kSortThreads) moe_place_kernel(SortParams p)
{
    extern __shared__ int next[];                      // [waves][E]: the row of a wave's next pair of an expert
    __shared__ int sums[2][kSortThreads];              // all pairs of an expert, and those of the blocks before
    __shared__ int part[kSortWaves];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int first = blockIdx.x * p.per, last = min(p.n, first + p.per);
    const int each = p.per / kSortWaves, from = first + wave * each, to = min(last, from + each);
    for (int i = tid; i < kSortWaves * p.E; i += kSortThreads)
        next[i] = 0;
    sums[0][tid] = sums[1][tid] = 0;
    __syncthreads();
    for (int i = from + lane; i < to; i += 64) {
        const int e = p.ids[i];
        if ((unsigned)e < (unsigned)p.E)
            atomicAdd(&next[wave * p.E + e], 1);
    }
    // several threads an expert, where there are fewer experts than threads, take blocks in turn
    const int turns = kSortThreads / p.E;
    if (tid < turns * p.E) {
        const int e = tid % p.E;
        int all = 0, before = 0;
#pragma unroll 8
        for (int b = tid / p.E; b < p.blocks; b += turns) {
            const int c = p.counts[b * p.E + e];
            all += c;
            before += b < (int)blockIdx.x ? c : 0;
        }
        atomicAdd(&sums[0][e], all);
        atomicAdd(&sums[1][e], before);
    }
    __syncthreads();
    // rows before this expert's: a sum over the experts before it
    const int all = sums[0][tid];
    int upto = all;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const int o = __shfl_up(upto, off);
        upto += lane >= off ? o : 0;
    }
    if (lane == 63)
        part[wave] = upto;
    __syncthreads();
    int rows = 0;
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) {
        upto += w < wave ? part[w] : 0;
        rows += part[w];
    }
    if (tid < p.E) {
        if (blockIdx.x == 0)
            p.offsets[tid] = upto - all;
        int at = upto - all + sums[1][tid];
        for (int w = 0; w < kSortWaves; ++w) {
            const int c = next[w * p.E + tid];
            next[w * p.E + tid] = at;
            at += c;
        }
    }
    if (blockIdx.x == 0 && tid == 0)
        p.offsets[p.E] = rows;
    for (int i = max(first, rows) + tid; i < last; i += kSortThreads)
        p.source[i] = -1;
    __syncthreads();
    for (int i0 = from; i0 < to; i0 += 64) {
        const int i = i0 + lane;
        const int e = i < to ? p.ids[i] : -1;
        const bool has = (unsigned)e < (unsigned)p.E;
        // lanes with the same expert
        unsigned long long same = __ballot(has);
        for (int bit = 1; bit < p.E; bit <<= 1) {
            const unsigned long long set = __ballot(has && (e & bit));
            same &= e & bit ? set : ~set;
        }
        const int rank = __popcll(same & ((1ull << lane) - 1));
        const int r = has ? next[wave * p.E + e] + rank : -1;
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");      // all lanes have read
        if (has && (same >> lane) == 1)                // the last of them
            next[wave * p.E + e] = r + 1;
        if (i < to)
            p.position[i] = r;
        if (has)
            p.source[r] = i;
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
}

// Pairs up to which the sort is one launch of E + 1 workgroups that all walk the
// pairs (2048 pairs of 64 experts: 9.7 us, more host time than kernel; two
// launches 13.0), and how more are cut: every block reads the counts of all.
constexpr int kSortFew = 2048, kSortBlocks = 64;
static void sort_blocks(int64_t n, int& per, int& blocks)
{
    per = (int)std::max<int64_t>(kSortThreads, ceil_div(ceil_div(n, kSortBlocks), kSortThreads) * kSortThreads);
    blocks = (int)ceil_div(n, per);
}

// ---------------------------------------------------------------- rows into order
struct GatherParams {
    const int32_t* position;
    int64_t T, rows;
    int k, pieces;
    const char* x[2];
    char* out[2];
    int64_t bytes[2];
};

constexpr int kPiece = 4;                              // 16-byte loads of a lane

// A wave reads a piece of a token's row once and writes it to each of the
// token's rows: `at` holds them, a lane each, -1 for none.
__device__ __forceinline__ void gather_piece(const char* x, char* out, int64_t bytes, int64_t t, int64_t piece, int k,
                                             int at, int lane)
{
    const int64_t items = bytes / 16, first = piece * 64 * kPiece + lane;
    const char* from = x + t * bytes;
    u32x4_t v[kPiece] = {};
    // lanes past the row read its last 16 bytes: a branch for them would wait for each load
#pragma unroll
    for (int q = 0; q < kPiece; ++q)
        if (piece * 64 * kPiece + 64 * q < items)
            v[q] = reinterpret_cast<const u32x4_any*>(from)[min(first + 64 * q, items - 1)];
    // what is left of the row after its whole 16 bytes
    const int rest = (int)(bytes & 15);
    const bool ends = rest && (piece + 1) * 64 * kPiece >= items && lane < rest;
    const char tail = ends ? from[items * 16 + lane] : (char)0;
#pragma unroll
    for (int q = 0; q < kPiece; ++q)
        __asm__ __volatile__("" : "+v"(v[q]));
    for (int j = 0; j < k; ++j) {
        const int r = __builtin_amdgcn_readlane(at, j);
        if (r < 0)
            continue;
        char* to = out + (int64_t)r * bytes;
#pragma unroll
        for (int q = 0; q < kPiece; ++q)
            if (first + 64 * q < items)
                reinterpret_cast<u32x4_any*>(to)[first + 64 * q] = v[q];
        if (ends)
            to[items * 16 + lane] = tail;
    }
}

// A token's rows for lanes j < k, -1 outside the rows.  Lanes are read (readlane)
// where the whole wave runs: the compiler may compute what a lane gives where it is
// used, so under a divergent branch inactive lanes would give anything.
__device__ __forceinline__ int position_of(const int32_t* position, int64_t t, int k, int64_t rows, int lane)
{
    const int at = lane < k ? position[t * k + lane] : -1;
    return at < rows ? at : -1;
}

__global__ void __launch_bounds__(256) moe_gather_kernel(GatherParams p)
{
    const int lane = threadIdx.x & 63;
    const unsigned units = (unsigned)(p.T * p.pieces);
    for (unsigned u = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); u < units; u += gridDim.x * 4) {
        const int64_t t = u / (unsigned)p.pieces, piece = u - t * p.pieces;
        const int at = position_of(p.position, t, p.k, p.rows, lane);
        gather_piece(p.x[0], p.out[0], p.bytes[0], t, piece, p.k, at, lane);
        if (piece == 0 && p.bytes[1] > 0)
            for (int64_t q = 0; q * 1024 * kPiece < p.bytes[1]; ++q)
                gather_piece(p.x[1], p.out[1], p.bytes[1], t, q, p.k, at, lane);
    }
}

// ---------------------------------------------------------------- rows back
struct CombineParams {
    const void *x, *dy;
    const int32_t* position;
    const float* weights;
    void *y, *dx;
    float* dweights;
    int64_t T, rows, H;
    int k, pieces;
};

// A lane's 16 bytes of a row as fp32: 8 bf16 or 4 fp32, from element h on; those
// past H are not written.
template <bool BF16>
struct Slice {
    static constexpr int N = BF16 ? 8 : 4;
    float v[N];
    __device__ __forceinline__ void store(void* row, int64_t h, int64_t H) const
    {
        if (h + N <= H) {
            u32x4_t w;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (BF16)
                    w[i] = f32_to_bf16_rne(v[2 * i]) | (unsigned)f32_to_bf16_rne(v[2 * i + 1]) << 16;
                else
                    w[i] = __float_as_uint(v[i]);
            }
            if constexpr (BF16)
                *reinterpret_cast<u32x4_any*>(static_cast<unsigned short*>(row) + h) = w;
            else
                *reinterpret_cast<u32x4_any*>(static_cast<float*>(row) + h) = w;
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (h + i < H) {
                    if constexpr (BF16)
                        static_cast<unsigned short*>(row)[h + i] = f32_to_bf16_rne(v[i]);
                    else
                        static_cast<float*>(row)[h + i] = v[i];
                }
        }
    }
};

// The same and their weights as scalars.
template <int KM>
struct Rows {
    int r[KM];
    float w[KM];
    __device__ __forceinline__ Rows(const CombineParams& p, int64_t t, int lane)
    {
        const int at = position_of(p.position, t, p.k, p.rows, lane);
        const float wl = p.weights && lane < p.k ? p.weights[t * p.k + lane] : 1.0f;
#pragma unroll
        for (int j = 0; j < KM; ++j) {
            r[j] = __builtin_amdgcn_readlane(at, j);   // -1 from lanes k, k + 1, ..
            w[j] = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(wl), j));
        }
    }
};

template <bool BF16>
__device__ __forceinline__ char* row_at(const void* base, int64_t r, int64_t H)
{
    return const_cast<char*>(static_cast<const char*>(base)) + r * H * (BF16 ? 2 : 4);
}

// The parts of a token's rows from element h on, zeros for those that aren't there,
// and of its gradient: all of them are on their way before the first is waited for.
template <bool BF16, int KM>
struct Parts {
    Piece<BF16, Slice<BF16>::N> x[KM], dy;
    __device__ __forceinline__ Parts(const CombineParams& p, const int (&r)[KM], int64_t h, const char* grad = nullptr)
    {
        dy.clear();
#pragma unroll
        for (int j = 0; j < KM; ++j)
            x[j].clear();
        if (p.H >= Slice<BF16>::N) {
            if (grad)
                dy.load(grad, h, p.H);
#pragma unroll
            for (int j = 0; j < KM; ++j)
                if (r[j] >= 0)
                    x[j].load(row_at<BF16>(p.x, r[j], p.H), h, p.H);
        } else {
            if (grad)
                dy.load_short(grad, h, p.H);
#pragma unroll
            for (int j = 0; j < KM; ++j)
                if (r[j] >= 0)
                    x[j].load_short(row_at<BF16>(p.x, r[j], p.H), h, p.H);
        }
    }
    __device__ __forceinline__ void arrived(int64_t h, int64_t H)
    {
        dy.arrived();
        dy.end(h, H);
#pragma unroll
        for (int j = 0; j < KM; ++j) {
            x[j].arrived();
            x[j].end(h, H);
        }
    }
};

// A wave takes 1 KiB of a token's row: up to KM rows' parts are on their way at once.
template <bool BF16, int KM>
__global__ void __launch_bounds__(256) moe_combine_kernel(CombineParams p)
{
    using S = Slice<BF16>;
    const int lane = threadIdx.x & 63;
    const unsigned units = (unsigned)(p.T * p.pieces);
    for (unsigned u = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); u < units; u += gridDim.x * 4) {
        const int64_t t = u / (unsigned)p.pieces, h = (u - t * p.pieces) * 64 * S::N + lane * S::N;
        const Rows<KM> rows(p, t, lane);
        Parts<BF16, KM> in(p, rows.r, h);
        in.arrived(h, p.H);
        S y;
#pragma unroll
        for (int i = 0; i < S::N; ++i)
            y.v[i] = 0.0f;
#pragma unroll
        for (int j = 0; j < KM; ++j)
            if (rows.r[j] >= 0)
#pragma unroll
                for (int i = 0; i < S::N; ++i)
                    y.v[i] = fmaf(rows.w[j], in.x[j][i], y.v[i]);
        y.store(row_at<BF16>(p.y, t, p.H), h, p.H);
    }
}

// A workgroup takes a token: dy is read once, each of its rows once, and the k
// dot products meet at the end.
template <bool BF16, int KM>
__global__ void __launch_bounds__(256) moe_combine_grad_kernel(CombineParams p)
{
    using S = Slice<BF16>;
    __shared__ float part[4][16];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
        const Rows<KM> rows(p, t, lane);
        float dot[KM] = {};
        // the whole workgroup runs every step; threads past H load zeros and store nothing
        for (int64_t h0 = 0; h0 < p.H; h0 += 256 * S::N) {
            const int64_t h = h0 + threadIdx.x * S::N;
            Parts<BF16, KM> in(p, rows.r, h, row_at<BF16>(p.dy, t, p.H));
            in.arrived(h, p.H);
#pragma unroll
            for (int j = 0; j < KM; ++j)
                if (rows.r[j] >= 0) {
                    S d;
#pragma unroll
                    for (int i = 0; i < S::N; ++i) {
                        dot[j] = fmaf(in.dy[i], in.x[j][i], dot[j]);
                        d.v[i] = rows.w[j] * in.dy[i];
                    }
                    d.store(row_at<BF16>(p.dx, rows.r[j], p.H), h, p.H);
                }
        }
#pragma unroll
        for (int j = 0; j < KM; ++j) {
#pragma unroll
            for (int off = 1; off < 64; off <<= 1)
                dot[j] += __shfl_xor(dot[j], off);
            if (lane == 0)
                part[wave][j] = dot[j];
        }
        __syncthreads();
        if (threadIdx.x < (unsigned)p.k)
            p.dweights[t * p.k + threadIdx.x] =
                part[0][threadIdx.x] + part[1][threadIdx.x] + part[2][threadIdx.x] + part[3][threadIdx.x];
        __syncthreads();
    }
}

// Shorter rows: TEAM lanes take a token, lane j of them has its j-th row, and a
// wave's tokens go their own ways.  Sixteen lanes for rows of up to 1 KiB
// (16384 x 8 rows of 128 bf16: 6 us, with a wave for each KiB 12; gradients 15, with
// a wave a token 37, a workgroup 74; 300 x 8 rows of 768 would take 13, with a
// wave 9), a wave for gradients of up to 2 KiB (16384 x 2 rows of 1024 bf16: 28 us, 40
// with a workgroup; 16384 x 8: 114 and 111).
constexpr int64_t kTeamBytes = 1024, kWaveBytes = 2048;

template <int KM, int TEAM>
struct TeamRows {
    int r[KM];
    float w[KM];
    __device__ __forceinline__ TeamRows(const CombineParams& p, int64_t t, int lane)
    {
        const int l = lane & (TEAM - 1), first = lane & (64 - TEAM);
        const bool has = t < p.T && l < p.k;
        const int at = has ? p.position[t * p.k + l] : -1;
        const float wl = has && p.weights ? p.weights[t * p.k + l] : 1.0f;
#pragma unroll
        for (int j = 0; j < KM; ++j) {                 // every lane runs here
            const int v = __shfl(at, first | j);
            r[j] = v < p.rows ? v : -1;
            w[j] = __shfl(wl, first | j);
        }
    }
};

template <bool BF16, int KM, int TEAM>
__global__ void __launch_bounds__(256) moe_combine_narrow_kernel(CombineParams p)
{
    using S = Slice<BF16>;
    const int lane = threadIdx.x & 63;
    for (int64_t t0 = (int64_t)blockIdx.x * (256 / TEAM); t0 < p.T; t0 += (int64_t)gridDim.x * (256 / TEAM)) {
        const int64_t t = t0 + (threadIdx.x / TEAM);
        const TeamRows<KM, TEAM> rows(p, t, lane);
        for (int64_t h0 = 0; h0 < p.H; h0 += TEAM * S::N) {
            const int64_t h = h0 + (lane & (TEAM - 1)) * S::N;
            Parts<BF16, KM> in(p, rows.r, h);
            in.arrived(h, p.H);
            S y;
#pragma unroll
            for (int i = 0; i < S::N; ++i)
                y.v[i] = 0.0f;
#pragma unroll
            for (int j = 0; j < KM; ++j)
                if (rows.r[j] >= 0)
#pragma unroll
                    for (int i = 0; i < S::N; ++i)
                        y.v[i] = fmaf(rows.w[j], in.x[j][i], y.v[i]);
            if (t < p.T)
                y.store(row_at<BF16>(p.y, t, p.H), h, p.H);
        }
    }
}

template <bool BF16, int KM, int TEAM>
__global__ void __launch_bounds__(256) moe_combine_grad_narrow_kernel(CombineParams p)
{
    using S = Slice<BF16>;
    const int lane = threadIdx.x & 63;
    for (int64_t t0 = (int64_t)blockIdx.x * (256 / TEAM); t0 < p.T; t0 += (int64_t)gridDim.x * (256 / TEAM)) {
        const int64_t t = t0 + (threadIdx.x / TEAM);
        const TeamRows<KM, TEAM> rows(p, t, lane);
        float dot[KM] = {};
        for (int64_t h0 = 0; h0 < p.H; h0 += TEAM * S::N) {
            const int64_t h = t < p.T ? h0 + (lane & (TEAM - 1)) * S::N : p.H;
            Parts<BF16, KM> in(p, rows.r, h, row_at<BF16>(p.dy, t < p.T ? t : 0, p.H));
            in.arrived(h, p.H);
#pragma unroll
            for (int j = 0; j < KM; ++j)
                if (rows.r[j] >= 0) {
                    S d;
#pragma unroll
                    for (int i = 0; i < S::N; ++i) {
                        dot[j] = fmaf(in.dy[i], in.x[j][i], dot[j]);
                        d.v[i] = rows.w[j] * in.dy[i];
                    }
                    d.store(row_at<BF16>(p.dx, rows.r[j], p.H), h, p.H);
                }
        }
#pragma unroll
        for (int j = 0; j < KM; ++j) {                 // every lane runs here
#pragma unroll
            for (int off = 1; off < TEAM; off <<= 1)
                dot[j] += __shfl_xor(dot[j], off);
            if (t < p.T && (lane & (TEAM - 1)) == j && j < p.k)
                p.dweights[t * p.k + j] = dot[j];
        }
    }
}

template <bool BF16, int KM>
static void launch_combine(const CombineParams& p, hipStream_t s)
{
    if (p.H * (BF16 ? 2 : 4) <= kTeamBytes)
        hipLaunchKernelGGL((moe_combine_narrow_kernel<BF16, KM, 16>), dim3(grid_of(ceil_div(p.T, 16))), dim3(256), 0, s,
                           p);
    else
        hipLaunchKernelGGL((moe_combine_kernel<BF16, KM>), dim3(grid_of(ceil_div(p.T * p.pieces, 4))), dim3(256), 0, s,
                           p);
}

template <bool BF16, int KM>
static void launch_combine_grad(const CombineParams& p, hipStream_t s)
{
    const int64_t bytes = p.H * (BF16 ? 2 : 4);
    if (bytes <= kTeamBytes)
        hipLaunchKernelGGL((moe_combine_grad_narrow_kernel<BF16, KM, 16>), dim3(grid_of(ceil_div(p.T, 16))), dim3(256),
                           0, s, p);
    else if (bytes <= kWaveBytes)
        hipLaunchKernelGGL((moe_combine_grad_narrow_kernel<BF16, KM, 64>), dim3(grid_of(ceil_div(p.T, 4))), dim3(256),
                           0, s, p);
    else
        hipLaunchKernelGGL((moe_combine_grad_kernel<BF16, KM>), dim3(grid_of(p.T)), dim3(256), 0, s, p);
}

// Up to 4, 8 or 16 rows of a token in registers.
template <bool BF16>
static void by_choices(const CombineParams& p, bool grad, hipStream_t s)
{
    if (p.k <= 4)
        grad ? launch_combine_grad<BF16, 4>(p, s) : launch_combine<BF16, 4>(p, s);
    else if (p.k <= 8)
        grad ? launch_combine_grad<BF16, 8>(p, s) : launch_combine<BF16, 8>(p, s);
    else
        grad ? launch_combine_grad<BF16, 16>(p, s) : launch_combine<BF16, 16>(p, s);
}

// ---------------------------------------------------------------- checks
static int check_order(int64_t T, int k)
{
    if (T < 0 || k < 1)
        return set_error(TG_E_INVAL, "T must be >= 0, k >= 1");
    if (k > kOrderChoices || T > kOrderTokens)
        return set_error(TG_E_UNSUPPORTED, "at most 16 choices and 2^24 tokens");
    return TG_OK;
}

static int check_sort(int64_t T, int64_t E, int k)
{
    const int st = check_order(T, k);
    if (st != TG_OK)
        return st;
    if (E < 1)
        return set_error(TG_E_INVAL, "E must be >= 1");
    if (E > kOrderExperts)
        return set_error(TG_E_UNSUPPORTED, "at most 1024 experts");
    return TG_OK;
}

static int check_rows(int64_t T, int k, int64_t rows, const int32_t* position)
{
    const int st = check_order(T, k);
    if (st != TG_OK)
        return st;
    if (rows < 0)
        return set_error(TG_E_INVAL, "rows must be >= 0");
    if (rows > 0x7FFFFFFF)
        return set_error(TG_E_UNSUPPORTED, "rows must be below 2^31");
    if (T > 0 && (!position || ((uintptr_t)position & 3u)))
        return set_error(TG_E_INVAL, "position must be given, 4-byte aligned");
    return TG_OK;
}

static int check_combine(int64_t T, int k, int64_t rows, int64_t H, int dtype, const int32_t* position)
{
    const int st = check_rows(T, k, rows, position);
    if (st != TG_OK)
        return st;
    if (H < 1)
        return set_error(TG_E_INVAL, "H must be >= 1");
    if (H > kOrderWidth)
        return set_error(TG_E_UNSUPPORTED, "H is at most 2^24");
    if (dtype != TG_F32 && dtype != TG_BF16)
        return set_error(TG_E_INVAL, "rows are fp32 or bf16");
    return TG_OK;
}

}  // namespace tg

using namespace tg;

extern "C" {

int tg_moe_sort_workspace_bytes(int64_t T, int64_t E, int k, size_t* bytes)
{
    const int st = check_sort(T, E, k);
    if (st != TG_OK)
        return st;
    if (!bytes)
        return set_error(TG_E_INVAL, "bytes is NULL");
    int per, blocks;
    sort_blocks(T * k, per, blocks);
    *bytes = T * k <= kSortFew ? 0 : (size_t)blocks * (size_t)E * 4;
    return TG_OK;
}

int tg_moe_sort(int64_t T, int64_t E, int k, const int32_t* ids, int32_t* position, int32_t* source,
                int32_t* offsets, void* workspace, size_t workspace_bytes)
{
    const int st = check_sort(T, E, k);
    if (st != TG_OK)
        return st;
    const int64_t n = T * k;
    SortParams p{ids, position, source, offsets, static_cast<int32_t*>(workspace), (int)n, (int)E, 0, 0};
    sort_blocks(n, p.per, p.blocks);
    if (n > kSortFew &&
        (!workspace || ((uintptr_t)workspace & 15u) || workspace_bytes < (size_t)p.blocks * (size_t)E * 4))
        return set_error(TG_E_INVAL,
                         "the workspace must be 16-byte aligned and hold tg_moe_sort_workspace_bytes() bytes");
    if (!offsets || (T > 0 && (!ids || !position || !source)) ||
        (((uintptr_t)ids | (uintptr_t)position | (uintptr_t)source | (uintptr_t)offsets) & 3u))
        return set_error(TG_E_INVAL, "ids, position, source and offsets must be given, 4-byte aligned");
    if (!have_device())
        return set_error(TG_E_UNSUPPORTED, "no HIP device");
    if (n <= kSortFew) {
        hipLaunchKernelGGL(moe_sort_few_kernel, dim3((unsigned)E + 1), dim3(256), 0, current_stream(), ids, (int)n,
                           (int)E, position, source, offsets);
    } else {
        const dim3 grid((unsigned)p.blocks), block(kSortThreads);
        hipLaunchKernelGGL(moe_count_kernel, grid, block, 0, current_stream(), p);
        hipLaunchKernelGGL(moe_place_kernel, grid, block, kSortWaves * (size_t)E * 4, current_stream(), p);
    }
    return launched("moe_sort launch");
}

int tg_moe_gather(int64_t T, int k, int64_t rows, const int32_t* position, int64_t row_bytes, const void* x,
                  void* out, int64_t row2_bytes, const void* x2, void* out2)
{
    const int st = check_rows(T, k, rows, position);
    if (st != TG_OK)
        return st;
    if (row_bytes < 1 || row2_bytes < 0)
        return set_error(TG_E_INVAL, "row_bytes must be >= 1, row2_bytes >= 0");
    if (row_bytes > kOrderWidth || row2_bytes > kOrderWidth)
        return set_error(TG_E_UNSUPPORTED, "rows are at most 2^24 bytes");
    if (T == 0 || rows == 0)
        return TG_OK;
    if (!x || !out || (row2_bytes > 0 && (!x2 || !out2)))
        return set_error(TG_E_INVAL, "x and out must be given");
    if (!have_device())
        return set_error(TG_E_UNSUPPORTED, "no HIP device");
    const int pieces = (int)std::max<int64_t>(1, ceil_div(row_bytes / 16, 64 * kPiece));
    if (T * pieces > kUnits)
        return set_error(TG_E_UNSUPPORTED, "moe_gather: more than 2^31 pieces of 4 KiB");
    const GatherParams p{position, T, rows, k, pieces, {static_cast<const char*>(x), static_cast<const char*>(x2)},
                         {static_cast<char*>(out), static_cast<char*>(out2)}, {row_bytes, row2_bytes}};
    hipLaunchKernelGGL(moe_gather_kernel, dim3(grid_of(ceil_div(T * pieces, 4))), dim3(256), 0, current_stream(), p);
    return launched("moe_gather launch");
}

int tg_moe_combine(int64_t T, int k, int64_t rows, int64_t H, const void* x, int dtype, const int32_t* position,
                   const float* weights, void* y)
{
    const int st = check_combine(T, k, rows, H, dtype, position);
    if (st != TG_OK || T == 0)
        return st;
    const uintptr_t mask = dtype == TG_F32 ? 3u : 1u;
    if ((rows > 0 && !x) || !y || (((uintptr_t)x | (uintptr_t)y) & mask) || ((uintptr_t)weights & 3u))
        return set_error(TG_E_INVAL, "x and y must be given; x, y and weights aligned to their elements");
    if (!have_device())
        return set_error(TG_E_UNSUPPORTED, "no HIP device");
    const CombineParams p{x, nullptr, position, weights, y, nullptr, nullptr, T, rows, H, k,
                          (int)ceil_div(H, dtype == TG_BF16 ? 512 : 256)};
    if (T * p.pieces > kUnits)
        return set_error(TG_E_UNSUPPORTED, "moe_combine: more than 2^31 pieces of 1 KiB");
    dtype == TG_BF16 ? by_choices<true>(p, false, current_stream()) : by_choices<false>(p, false, current_stream());
    return launched("moe_combine launch");
}

int tg_moe_combine_grad(int64_t T, int k, int64_t rows, int64_t H, const void* dy, const void* x, int dtype,
                        const int32_t* position, const float* weights, void* dx, float* dweights)
{
    const int st = check_combine(T, k, rows, H, dtype, position);
    if (st != TG_OK || T == 0)
        return st;
    const uintptr_t mask = dtype == TG_F32 ? 3u : 1u;
    if (!dy || (rows > 0 && (!x || !dx)) || !weights || !dweights ||
        (((uintptr_t)dy | (uintptr_t)x | (uintptr_t)dx) & mask) || (((uintptr_t)weights | (uintptr_t)dweights) & 3u))
        return set_error(TG_E_INVAL, "dy, x, weights, dx and dweights must be given, aligned to their elements");
    if (!have_device())
        return set_error(TG_E_UNSUPPORTED, "no HIP device");
    const CombineParams p{x, dy, position, weights, nullptr, dx, dweights, T, rows, H, k, 0};
    dtype == TG_BF16 ? by_choices<true>(p, true, current_stream()) : by_choices<false>(p, true, current_stream());
    return launched("moe_combine_grad launch");
}

}  // extern "C"
