// Products of 8-bit matrices, C = act(A . B^T + bias), and the same for each
// expert on its own rows.
//
//   C[m][n] = act(sum_c sA[m][c] sB[n][c] (sum_{k in chunk c} a[m][k] b[n][k]) + bias[n])
//
// A chunk of 128 k of 16 x 16 results is summed from zero; a lane's four sums are
// multiplied by their scales as they are added up, in fp32.  B is the first
// operand: a lane then has one row m and four neighbouring columns n.  Products
// take the exact form; those of many rows the fast one where the caller asks for
// it (fp8.hpp).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <string>

#include "fp8.hpp"
#include "fp8_host.hpp"

namespace tg {

constexpr int64_t kMaxBlocks = (int64_t)1 << 22;       // of at most 512 threads: a grid has 2^32 threads
constexpr int64_t kMaxDepth = (int64_t)1 << 22;        // 256 rows of A or B stay within 32-bit offsets

struct F8Params {
    const unsigned char *A, *B;
    const float *sA, *sB;
    const float* bias;
    const int32_t* offsets;                            // experts: E + 1, else null
    void* C;
    int64_t M, N;
    int chunks, E;
    int b_rows;                                        // rows of B that share a scale, 1 or 128
    int out_bf16, act;
    int vec_out;                                       // four results of a row are one aligned access
    int line_out;                                      // and eight bf16
    int group_m;                                       // row tiles that go through the column tiles together
    int split, each;                                   // parts of the reduction, chunks of one
    float* slabs;                                      // their sums, `slab` floats apart
    int64_t slab;
};

// How many tiles of BM rows the experts up to `e` of its group of 64 have (lane
// by lane), and the rows [lo, hi) of expert e.
template <int BM>
__device__ __forceinline__ int expert_tiles(const F8Params& p, int e, int lane, int64_t& lo, int64_t& hi)
{
    lo = hi = 0;
    if (e < p.E) {
        lo = max((int64_t)0, (int64_t)p.offsets[e]);
        hi = min(p.M, (int64_t)p.offsets[e + 1]);
    }
    int n = hi > lo ? (int)((hi - lo + BM - 1) / BM) : 0;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const int o = __shfl_up(n, off);
        n += lane >= off ? o : 0;
    }
    return n;
}

// The workgroup's tile of the experts' products: rows [m0, m1) of expert
// `expert` (BM of them at most matter), column tile tn.  Tiles are numbered expert
// by expert, column tiles of a row tile in order, and each XCD has a contiguous
// range.  False past the last tile: the grid is for as many as there can be.  Every
// wave works it out by itself; all of its lanes run.
template <int BM>
__device__ __forceinline__ bool expert_tile(const F8Params& p, int tiles_n, int64_t& m0, int64_t& m1, int& tn,
                                            int& expert)
{
    const int lane = threadIdx.x & 63;
    int total = 0;
    for (int e0 = 0; e0 < p.E; e0 += 64) {
        int64_t lo, hi;
        total += __builtin_amdgcn_readlane(expert_tiles<BM>(p, e0 + lane, lane, lo, hi), 63);
    }
    const int64_t n = (int64_t)total * tiles_n, q = n >> 3, r = n & 7;
    const int64_t x = blockIdx.x & 7, i = blockIdx.x >> 3;
    if (i >= q + (x < r ? 1 : 0))
        return false;
    const int64_t id = x * q + min(x, r) + i;
    int tile = (int)(id / tiles_n);
    tn = (int)(id - (int64_t)tile * tiles_n);
    for (int e0 = 0;; e0 += 64) {
        int64_t lo, hi;
        const int upto = expert_tiles<BM>(p, e0 + lane, lane, lo, hi);
        const int here = __builtin_amdgcn_readlane(upto, 63);
        if (tile >= here) {
            tile -= here;
            continue;
        }
        const int at = __ffsll((long long)__ballot(upto > tile)) - 1;
        const int before = at ? __builtin_amdgcn_readlane(upto, at - 1) : 0;
        expert = e0 + at;
        m0 = (int64_t)__builtin_amdgcn_readlane((int)lo, at) + (int64_t)(tile - before) * BM;
        m1 = __builtin_amdgcn_readlane((int)hi, at);
        return true;
    }
}

}  // namespace tg

#include "gemm_fp8_stream.hpp"
#include "gemm_fp8_tiles.hpp"

namespace tg {

// C = act(sums of the S parts of the reduction, in order, + bias): four
// neighbouring results a thread, all of its loads on their way at once.  Bound by
// memory, 4 S bytes read a result, once; small results by a launch and one round
// trip (100 x 4096 in 4 parts and 100 x 1000 in 16: 4 us each).  (splitk_reduce does
// the same for other products, whose ReLU makes a NaN 0.)
template <int S>
__global__ void __launch_bounds__(256) gemm_fp8_parts_kernel(F8Params p)
{
    const int64_t n = p.M * p.N, stride = (int64_t)gridDim.x * 1024;
    for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4; i < n; i += stride) {
        // slabs are whole fours: what is past the last result is read and not used
        f32x4_t part[S];
#pragma unroll
        for (int s = 0; s < S; ++s)
            part[s] = __builtin_nontemporal_load(reinterpret_cast<const f32x4_t*>(p.slabs + s * p.slab + i));
        f32x4_t v = part[0];
#pragma unroll
        for (int s = 1; s < S; ++s)
            v += part[s];
        int64_t col = p.bias ? i % p.N : 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[e] = activate(v[e] + (p.bias ? p.bias[col] : 0.0f), p.act);
            col = col + 1 == p.N ? 0 : col + 1;
        }
        // as one row of n results
        store_four(p, i, n - i, v);
    }
}

static int launch_parts(const F8Params& p, hipStream_t s)
{
    const dim3 grid((unsigned)std::min<int64_t>(ceil_div(p.M * p.N, 1024), 65536)), block(256);
    switch (p.split) {
    case 2: hipLaunchKernelGGL(gemm_fp8_parts_kernel<2>, grid, block, 0, s, p); break;
    case 4: hipLaunchKernelGGL(gemm_fp8_parts_kernel<4>, grid, block, 0, s, p); break;
    case 8: hipLaunchKernelGGL(gemm_fp8_parts_kernel<8>, grid, block, 0, s, p); break;
    default: hipLaunchKernelGGL(gemm_fp8_parts_kernel<16>, grid, block, 0, s, p); break;
    }
    return launched("gemm_fp8 sums launch");
}

template <int BM, int BN, int WGM, int WGN, int ST, bool BROWS, bool EXACT>
static int launch_tiles(const F8Params& p, hipStream_t s)
{
    using Cf = F8Tile<BM, BN, WGM, WGN, ST, BROWS>;
    const int64_t tiles_m = ceil_div(p.M, BM) + (p.offsets ? std::min<int64_t>(p.E, p.M) : 0);
    const int64_t blocks = tiles_m * ceil_div(p.N, BN) * std::max(p.split, 1);
    if (blocks > kMaxBlocks)
        return set_error(TG_E_UNSUPPORTED, "too many tiles for one launch");
    hipLaunchKernelGGL((gemm_fp8_tiles_kernel<BM, BN, WGM, WGN, ST, BROWS, EXACT>), dim3((unsigned)blocks), dim3(Cf::T),
                       Cf::LDS, s, p);
    return launched("gemm_fp8 launch");
}

template <int MT, int P, int R, int W, bool BROWS>
static int launch_stream(const F8Params& p, hipStream_t s)
{
    const int64_t tiles_m = p.offsets ? ceil_div(p.M, 16 * MT) + std::min<int64_t>(p.E, p.M) : 1;
    const int64_t blocks = tiles_m * ceil_div(p.N, 16 * P);
    if (blocks > kMaxBlocks)
        return set_error(TG_E_UNSUPPORTED, "too many tiles for one launch");
    hipLaunchKernelGGL((gemm_fp8_stream_kernel<MT, P, R, W, BROWS>), dim3((unsigned)blocks), dim3(64 * W),
                       (F8Stream<MT, P, R, W, BROWS>::LDS), s, p);
    return launched("gemm_fp8 launch");
}

// Panels a workgroup, depth of the ring and waves: where there are many panels
// several of them share the rows' traffic, where there are few each gets a
// workgroup, and many waves, to itself.  With K = 4096, kernels alone, us:
//   panels            256    384    512    640    768   1024   1280   1536   1792   2560
//   16 rows   one     6.8    9.8   10.3   13.7   15.6   19.1   24.8   27.8   32.4   43.7
//            four    10.9   11.4   11.9   12.6   13.3   15.6   24.4   26.6   28.0   41.2
//           eight    18.1   18.5   19.0   19.4   19.6   20.2   21.9   24.3   26.5   45.5
//   32 rows   one     7.9   12.2   12.6   17.1   18.2   23.1   29.2   33.6   39.1   52.9
//            four    12.9   13.5   14.1   14.8   15.5   17.3   27.7   29.5   31.0   45.2
//   64 rows   one    10.6   18.6   19.4   27.3   28.1   36.6   45.6   54.1   62.8   88.7
//            four    19.8   20.3   21.0   21.7   22.5   24.2   33.4   34.5   35.2   51.1
// so one panel below some 550, and eight for 16 rows from 1200 on: the bounds are
// two workgroups, and six panels, a compute unit.  (8192 deep, 28672 columns: eight
// 44 us, one 64.)  Experts have about `rows` rows each, often fewer: one or two tiles
// of 16, and two waves, so that a compute unit holds several workgroups (64 tokens
// over 64 experts of 2816 x 2048 63 us, with four waves 72; 256 tokens: two tiles
// 83, one 94).  One panel and eight waves for few panels of all experts (2048 deep,
// 8 experts of 16 tokens: 256 panels 5.9 against 11.1 us, 512 8.0 against 11.3, 1024
// 14.5 against 12.1).
constexpr int64_t kStreamRows = 64, kStreamExpertRows = 32;
template <bool BROWS>
static int stream_by_rows(const F8Params& p, int64_t rows, hipStream_t s)
{
    const int64_t panels = ceil_div(p.N, 16);
    if (p.offsets) {
        const int64_t works = panels * std::min<int64_t>(p.E, p.M);
        if (works < 512)
            return launch_stream<1, 1, 2, 8, BROWS>(p, s);
        return rows <= 8 ? launch_stream<1, 4, 2, 2, BROWS>(p, s) : launch_stream<2, 4, 2, 2, BROWS>(p, s);
    }
    if (rows <= 16)
        return panels < 512 ? launch_stream<1, 1, 2, 8, BROWS>(p, s)
                            : panels < 1536 ? launch_stream<1, 4, 2, 4, BROWS>(p, s)
                                            : launch_stream<1, 8, 2, 4, BROWS>(p, s);
    if (rows <= 32)
        return panels < 512 ? launch_stream<2, 1, 3, 4, BROWS>(p, s) : launch_stream<2, 4, 2, 4, BROWS>(p, s);
    return panels < 512 ? launch_stream<4, 1, 2, 4, BROWS>(p, s) : launch_stream<4, 4, 1, 4, BROWS>(p, s);
}

// Tiles for more rows.
enum Tile { kTile256, kTile128x256, kTile128, kTile128Deep, kTile64, kTile32, kTiles };
struct TileForm {
    int bm, bn;
    int resident;                                      // workgroups on a compute unit
    float round_us;                                    // beginning and end of a round of them
    float chunk_us[4];                                 // a chunk of a round: [2 exact + rows of B]
};

// Measured (MI355X, 8192 x 8192 by 8192 and by 1024; the deep and the small tiles
// with 512 and 100 rows).  8192 deep, fast sums: 256 x 256 has 454 us, 128 x 256
// 554, 128 x 128 622, 64 x 64 994; with a scale for each row of B 708 (its registers
// do not suffice), 660, 705, 1,106.  Exact, fp32 results: 1,531 (registers again),
// 937, 1,002, 1,425.  Exact, 4096 x 4096, 128 x 256 to 32 x 64 without parts, bf16:
// 100 rows 55, 43, 36, 22, 18 us (as planned, in parts, 17), 512 rows 57, 44, 37, 29,
// 37 (28), 2048 rows 63, 65, 77, 97, 118 (63), 8192 rows 240, 237, 297, 366, 449 (238).
constexpr float kNever = 1e9f;
static const TileForm kForms[kTiles] = {{256, 256, 1, 8.7f, {1.64f, kNever, kNever, kNever}},
                                        {128, 256, 1, 5.3f, {1.00f, 1.21f, 1.68f, 1.85f}},
                                        {128, 128, 2, 4.3f, {1.15f, 1.30f, 1.85f, 2.00f}},
                                        {128, 128, 1, 4.0f, {0.75f, 0.80f, 1.10f, 1.20f}},
                                        {64, 64, 2, 2.5f, {0.45f, 0.50f, 0.64f, 0.72f}},
                                        {32, 64, 3, 2.0f, {0.42f, 0.46f, 0.52f, 0.58f}}};

struct TilePlan {
    Tile tile;
    int split, each;
};

// The tile, and into how many parts the reduction is split, with the smallest
// estimate: rounds of workgroups on the compute units times what they take, and
// for parts a second launch that adds up their slabs.  Without parts 100 x 1000 x
// 16384 takes 45 us, 32 workgroups of 128 chunks.
static TilePlan plan_tiles(int64_t M, int64_t N, int chunks, int64_t experts, int form)
{
    TilePlan best{kTile128, 1, chunks};
    double least = 1e30;
    const double cus = (double)compute_units();
    for (int t = 0; t < kTiles; ++t) {
        const TileForm& f = kForms[t];
        // an expert's last tile is half full
        const double tiles_m = experts ? (double)M / f.bm + 0.5 * (double)experts : (double)ceil_div(M, f.bm);
        const double tiles = std::ceil(tiles_m) * (double)ceil_div(N, f.bn);
        for (int split = 1; split <= (experts ? 1 : 16); split *= 2) {
            const int each = (int)ceil_div(chunks, split);
            if (split > 1 && (each < 4 || ceil_div(chunks, each) != split))
                break;
            const double rounds = std::ceil(tiles * split / (cus * f.resident));
            double us = rounds * (each * (double)f.chunk_us[form] + (double)f.round_us);
            if (split > 1)
                us += 3.0 + (double)M * (double)N * (8.0 * split + 4.0) / 4e6;
            if (us < least) {
                least = us;
                best = {(Tile)t, split, each};
            }
        }
    }
    return best;
}

static size_t slabs_bytes(const TilePlan& t, int64_t M, int64_t N)
{
    return t.split > 1 ? (size_t)t.split * (size_t)splitk_slab(M, N) * 4 : 0;
}

template <bool BROWS, bool EXACT>
static int launch_tile(const F8Params& p, Tile tile, hipStream_t s)
{
    // eight waves where the sums and fragments of a chunk fit their registers
    constexpr int WGN = BROWS || EXACT ? 2 : 4;
    switch (tile) {
    case kTile256:
        if constexpr (!BROWS && !EXACT)
            return launch_tiles<256, 256, 2, 4, 2, BROWS, EXACT>(p, s);
        [[fallthrough]];
    case kTile128x256:
        return launch_tiles<128, 256, 2, 4, 3, BROWS, EXACT>(p, s);
    case kTile128:
        return launch_tiles<128, 128, 2, WGN, 2, BROWS, EXACT>(p, s);
    case kTile128Deep:
        return launch_tiles<128, 128, 2, 4, 4, BROWS, EXACT>(p, s);
    case kTile64:
        return launch_tiles<64, 64, 2, 2, 4, BROWS, EXACT>(p, s);
    default:
        return launch_tiles<32, 64, 1, 4, 4, BROWS, EXACT>(p, s);
    }
}

// Rows that a workgroup of the streaming kernel would have.
static int64_t stream_rows(int64_t M, int64_t experts)
{
    return experts ? ceil_div(M, std::min(experts, M)) : M;
}

static int launch_gemm(F8Params p, bool exact, void* workspace, size_t workspace_bytes, hipStream_t s)
{
    // 8192 x 8192 x 8192, 1 to 32 row tiles: 977, 923, 906, 902, 909, 942 us (fast sums
    // 467, 448, 441, 442, 451, 478); 8192 x 28672 x 4096 1787, 1722, 1708, 1691, 1701, 1761
    p.group_m = 8;
    p.vec_out = p.N % 4 == 0 && (uintptr_t)p.C % (p.out_bf16 ? 8 : 16) == 0;
    p.line_out = p.N % 8 == 0 && (uintptr_t)p.C % 16 == 0;
    const bool by_rows = p.b_rows == 1;
    const int64_t experts = p.offsets ? std::min<int64_t>(p.E, p.M) : 0, rows = stream_rows(p.M, experts);
    if (rows <= (experts ? kStreamExpertRows : kStreamRows))
        return by_rows ? stream_by_rows<true>(p, rows, s) : stream_by_rows<false>(p, rows, s);
    const TilePlan t = plan_tiles(p.M, p.N, p.chunks, experts, 2 * exact + by_rows);
    F8Params whole = p;
    p.split = t.split;
    p.each = t.each;
    if (t.split > 1) {
        if (!workspace || ((uintptr_t)workspace & 15u) || workspace_bytes < slabs_bytes(t, p.M, p.N))
            return set_error(TG_E_INVAL,
                             "the workspace must be 16-byte aligned and hold tg_gemm_fp8_workspace_bytes() bytes");
        p.slabs = static_cast<float*>(workspace);
        p.slab = splitk_slab(p.M, p.N);
        p.bias = nullptr;
        p.act = 0;
        p.out_bf16 = 0;
        p.vec_out = p.N % 4 == 0;
    }
    const int st = exact ? by_rows ? launch_tile<true, true>(p, t.tile, s) : launch_tile<false, true>(p, t.tile, s)
                         : by_rows ? launch_tile<true, false>(p, t.tile, s) : launch_tile<false, false>(p, t.tile, s);
    if (st != TG_OK || t.split == 1)
        return st;
    whole.split = t.split;
    whole.slabs = p.slabs;
    whole.slab = p.slab;
    whole.vec_out = (uintptr_t)whole.C % (whole.out_bf16 ? 8 : 16) == 0;
    return launch_parts(whole, s);
}

// The type of C in a dtype that may have TG_FAST_SUMS.
static int c_type(int dtype) { return dtype & ~TG_FAST_SUMS; }

static int check_product(int64_t M, int64_t N, int64_t K, int dtype)
{
    if (M < 0 || N < 0 || K < 1)
        return set_error(TG_E_INVAL, "rows and N must be >= 0, K >= 1");
    if (c_type(dtype) != TG_BF16 && c_type(dtype) != TG_BF16_F32OUT)
        return set_error(TG_E_INVAL, "C is bf16 (TG_BF16) or fp32 (TG_BF16_F32OUT)");
    if (M > kMaxSide || N > kMaxSide || K > kMaxDepth)
        return set_error(TG_E_UNSUPPORTED, "rows and N are at most 2^24, K 2^22");
    return TG_OK;
}

static int check_output(const void* C, int dtype)
{
    if (!C || ((uintptr_t)C & (c_type(dtype) == TG_BF16 ? 1u : 3u)))
        return set_error(TG_E_INVAL, "C must be given, aligned to its elements");
    return TG_OK;
}

static F8Params params_of(int64_t M, int64_t N, int64_t K, const tg_f8& A, const tg_f8& B, void* C, int dtype)
{
    F8Params p{};
    p.A = static_cast<const unsigned char*>(A.codes);
    p.B = static_cast<const unsigned char*>(B.codes);
    p.sA = A.scales;
    p.sB = B.scales;
    p.C = C;
    p.M = M;
    p.N = N;
    p.chunks = (int)ceil_div(K, 128);
    p.b_rows = B.block;
    p.out_bf16 = c_type(dtype) == TG_BF16;
    return p;
}

}  // namespace tg

using namespace tg;

extern "C" {

int tg_gemm_fp8_workspace_bytes(int64_t M, int64_t N, int64_t K, size_t* bytes)
{
    if (!bytes || M < 0 || N < 0 || K < 1 || M > kMaxSide || N > kMaxSide || K > kMaxDepth)
        return set_error(TG_E_INVAL, "bad size, or bytes is NULL");
    *bytes = 0;
    if (M > kStreamRows && N > 0)
        for (int form = 0; form < 4; ++form)
            *bytes = std::max(*bytes, slabs_bytes(plan_tiles(M, N, (int)ceil_div(K, 128), 0, form), M, N));
    return TG_OK;
}

int tg_gemm_fp8(int64_t M, int64_t N, int64_t K, const tg_f8* A, const tg_f8* B, const float* bias, void* C,
                int dtype, int act, void* workspace, size_t workspace_bytes)
{
    int st = check_product(M, N, K, dtype);
    if (st != TG_OK)
        return st;
    if (act != TG_ACT_NONE && act != TG_ACT_RELU && act != TG_ACT_GELU)
        return set_error(TG_E_INVAL, "unknown activation");
    if (M == 0 || N == 0)
        return TG_OK;
    if ((st = check_f8(A, "A", true)) != TG_OK || (st = check_f8(B, "B", false)) != TG_OK ||
        (st = check_output(C, dtype)) != TG_OK)
        return st;
    if ((uintptr_t)bias & 3u)
        return set_error(TG_E_INVAL, "bias must be 4-byte aligned");
    if (!have_device())
        return set_error(TG_E_UNSUPPORTED, "no HIP device");
    F8Params p = params_of(M, N, K, *A, *B, C, dtype);
    p.bias = bias;
    p.act = act;
    return launch_gemm(p, !(dtype & TG_FAST_SUMS), workspace, workspace_bytes, current_stream());
}

int tg_moe_gemm_fp8(int64_t rows, int64_t E, int64_t N, int64_t K, const tg_f8* A, const tg_f8* B,
                    const int32_t* offsets, void* C, int dtype)
{
    int st = check_product(rows, N, K, dtype);
    if (st != TG_OK)
        return st;
    if (E < 1)
        return set_error(TG_E_INVAL, "E must be >= 1");
    if (E > 1024)
        return set_error(TG_E_UNSUPPORTED, "at most 1024 experts");
    if (rows == 0 || N == 0)
        return TG_OK;
    if ((st = check_f8(A, "A", true)) != TG_OK || (st = check_f8(B, "B", false)) != TG_OK ||
        (st = check_output(C, dtype)) != TG_OK)
        return st;
    if (!offsets || ((uintptr_t)offsets & 3u))
        return set_error(TG_E_INVAL, "offsets must be given, 4-byte aligned");
    if (!have_device())
        return set_error(TG_E_UNSUPPORTED, "no HIP device");
    F8Params p = params_of(rows, N, K, *A, *B, C, dtype);
    p.offsets = offsets;
    p.E = (int)E;
    return launch_gemm(p, !(dtype & TG_FAST_SUMS), nullptr, 0, current_stream());
}

}  // extern "C"
