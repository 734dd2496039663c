// Products of 8-bit matrices, C = act(A . B^T + bias), and the same for each
// expert on its own rows.
//
//   C[m][n] = act(sum_c sA[m][c] sB[n][c] (sum_{k in chunk c} a[m][k] b[n][k]) + bias[n])
//
// A chunk of 128 k of 16 x 16 results is summed from zero; a lane's four sums are
// multiplied by their scales as they are added up, in fp32.  B is the first
// operand: a lane then has one row m and four neighbouring columns n.  fp32
// results take the exact form of the products, bf16 results of many rows the
// fast one (fp8.hpp).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <string>

#include "fp8.hpp"
#include "fp8_host.hpp"

namespace tg {

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
    int group_m;                                       // row tiles that go through the column tiles together
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

}  // namespace tg

#include "gemm_fp8_tiles.hpp"

namespace tg {

// The rows [begin, end) and the matrix of B that row tile `tile` of BM rows
// belongs to; false past the last tile.
template <int BM>
__device__ __forceinline__ bool rows_of_tile(const F8Params& p, int64_t tile, int64_t& begin, int64_t& end, int& expert)
{
    if (!p.offsets) {
        begin = tile * BM;
        end = p.M;
        expert = 0;
        return begin < p.M;
    }
    for (int e = 0; e < p.E; ++e) {
        const int64_t lo = max((int64_t)0, (int64_t)p.offsets[e]), hi = min(p.M, (int64_t)p.offsets[e + 1]);
        const int64_t tiles = hi > lo ? (hi - lo + BM - 1) / BM : 0;
        if (tile < tiles) {
            begin = lo + tile * BM;
            end = hi;
            expert = e;
            return true;
        }
        tile -= tiles;
    }
    return false;
}

// A wave takes 16 rows and 64 columns.
__global__ void __launch_bounds__(256) gemm_fp8_kernel(F8Params p)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int l16 = lane & 15, g = lane >> 4;
    int64_t m0, m1;
    int expert;
    if (!rows_of_tile<16>(p, blockIdx.x, m0, m1, expert))
        return;
    const int64_t Kp = (int64_t)p.chunks * 128;
    const int64_t groups = (p.N + p.b_rows - 1) / p.b_rows;
    const unsigned char* B = p.B + (int64_t)expert * p.N * Kp;
    const float* sB = p.sB + (int64_t)expert * groups * p.chunks;
    for (int64_t n0 = ((int64_t)blockIdx.y * 4 + wave) * 64; n0 < p.N; n0 += (int64_t)gridDim.y * 256) {
        const int64_t m = min(m0 + l16, m1 - 1);
        f32x4_t acc[4] = {};
        for (int c = 0; c < p.chunks; ++c) {
            const u32x4_t* a = reinterpret_cast<const u32x4_t*>(p.A + m * Kp + c * 128);
            const Expanded af = expand(a[g], a[g + 4]);
            const float sa = p.sA[m * p.chunks + c];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int64_t n = min(n0 + 16 * j + l16, p.N - 1);
                const u32x4_t* b = reinterpret_cast<const u32x4_t*>(B + n * Kp + c * 128);
                const f32x4_t d = mfma_exact(expand(b[g], b[g + 4]), af);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int64_t nn = min(n0 + 16 * j + 4 * g + i, p.N - 1);
                    acc[j][i] = fmaf(d[i], sa * sB[nn / p.b_rows * p.chunks + c], acc[j][i]);
                }
            }
        }
        if (m0 + l16 < m1)
            for (int j = 0; j < 4; ++j)
                for (int i = 0; i < 4; ++i) {
                    const int64_t n = n0 + 16 * j + 4 * g + i;
                    if (n < p.N) {
                        const float v = apply_act(acc[j][i] + (p.bias ? p.bias[n] : 0.0f), p.act);
                        if (p.out_bf16)
                            static_cast<unsigned short*>(p.C)[(m0 + l16) * p.N + n] = f32_to_bf16_rne(v);
                        else
                            static_cast<float*>(p.C)[(m0 + l16) * p.N + n] = v;
                    }
                }
    }
}

template <int BM, int BN, int WGM, int WGN, bool BROWS, bool EXACT>
static int launch_tiles(const F8Params& p, hipStream_t s)
{
    using Cf = F8Tile<BM, BN, WGM, WGN, BROWS>;
    const int64_t tiles_m = ceil_div(p.M, BM) + (p.offsets ? std::min<int64_t>(p.E, p.M) : 0);
    hipLaunchKernelGGL((gemm_fp8_tiles_kernel<BM, BN, WGM, WGN, BROWS, EXACT>),
                       dim3((unsigned)(tiles_m * ceil_div(p.N, BN))), dim3(Cf::T), Cf::LDS, s, p);
    return launched("gemm_fp8 launch");
}

static int launch_gemm(F8Params p, hipStream_t s)
{
    p.group_m = 8;
    p.vec_out = p.N % 4 == 0 && (uintptr_t)p.C % (p.out_bf16 ? 8 : 16) == 0;
    if (p.M > 64) {
        if (p.out_bf16)
            return p.b_rows == 1 ? launch_tiles<256, 256, 2, 4, true, false>(p, s)
                                 : launch_tiles<256, 256, 2, 4, false, false>(p, s);
        return p.b_rows == 1 ? launch_tiles<128, 128, 2, 2, true, true>(p, s)
                             : launch_tiles<128, 128, 2, 2, false, true>(p, s);
    }
    const int64_t tiles = ceil_div(p.M, 16) + (p.offsets ? p.E : 0);
    hipLaunchKernelGGL(gemm_fp8_kernel, dim3((unsigned)tiles, (unsigned)std::min<int64_t>(ceil_div(p.N, 256), 65535)),
                       dim3(256), 0, s, p);
    return launched("gemm_fp8 launch");
}

static int check_product(int64_t M, int64_t N, int64_t K, int dtype)
{
    if (M < 0 || N < 0 || K < 1)
        return set_error(TG_E_INVAL, "rows and N must be >= 0, K >= 1");
    if (dtype != TG_BF16 && dtype != TG_BF16_F32OUT)
        return set_error(TG_E_INVAL, "C is bf16 (TG_BF16) or fp32 (TG_BF16_F32OUT)");
    if (M > kMaxSide || N > kMaxSide || K > kMaxDepth)
        return set_error(TG_E_UNSUPPORTED, "rows and N are at most 2^24, K 2^22");
    return TG_OK;
}

static int check_output(const void* C, int dtype)
{
    if (!C || ((uintptr_t)C & (dtype == TG_BF16 ? 1u : 3u)))
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
    p.out_bf16 = dtype == TG_BF16;
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
    return TG_OK;
}

int tg_gemm_fp8(int64_t M, int64_t N, int64_t K, const tg_f8* A, const tg_f8* B, const float* bias, void* C,
                int dtype, int act, void* workspace, size_t workspace_bytes)
{
    (void)workspace, (void)workspace_bytes;
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
    return launch_gemm(p, current_stream());
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
    return launch_gemm(p, current_stream());
}

}  // extern "C"
