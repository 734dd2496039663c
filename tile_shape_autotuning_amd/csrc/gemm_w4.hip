// C = act(A . W + bias), W in 4 bits with group scales (storage and
// arithmetic: w4.hpp).
//
// Few rows: the panels of W stream past rows kept in registers (panel_stream.hpp).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <string>

#include "panel_stream.hpp"
#include "w4.hpp"
#include "w4_host.hpp"

namespace tg {

struct GemmW4Params {
    const unsigned short* A;
    W4View w;
    const float* bias;
    void* C;
    int64_t M, N, K;
    int panels, out_bf16, act;
    int per, blocks;                                   // panels a workgroup, blocks of K
};

// Bias, activation and conversion of a 16 x 16 tile whose lane holds rows
// 4 (lane / 16) + 0..3 of column lane % 16.
__device__ __forceinline__ void store_tile(const GemmW4Params& p, int64_t row, int64_t col, f32x4_t v, int lane)
{
    col += lane & 15;
    row += (lane >> 4) * 4;
    if (col >= p.N)
        return;
    const float bias = p.bias ? p.bias[col] : 0.0f;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        if (row + r >= p.M)
            return;
        const float x = apply_act(v[r] + bias, p.act);
        if (p.out_bf16)
            static_cast<unsigned short*>(p.C)[(row + r) * p.N + col] = f32_to_bf16_rne(x);
        else
            static_cast<float*>(p.C)[(row + r) * p.N + col] = x;
    }
}

// One workgroup a compute unit: most of its LDS may hold sums.
template <int MT>
constexpr int kHalf = MT == 4 ? 32 : 64;

// A workgroup multiplies MT x 16 rows with p.per panels (panel_stream.hpp).  K
// beyond the waves' W x CW chunks comes in further blocks, whose sums wait in
// LDS.
template <bool ZERO, int MT, int W, int CW, int GS>
__global__ void __launch_bounds__(64 * W) gemm_w4_panels_kernel(GemmW4Params p)
{
    using S = PanelStream<true, ZERO, MT, 1, 1, W, CW, GS, kHalf<MT>>;
    __shared__ f32x4_t red[S::RED], mid[S::MID];
    extern __shared__ f32x4_t part[];                  // [p.per][MT][64] if there is more than one block
    S s(red, mid, p.w.scale_f32);
    const int lane = s.lane, l16 = lane & 15, kq = lane >> 4;
    const int panel0 = blockIdx.x * p.per;
    const int n = min(p.per, p.panels - panel0);
    const int64_t row0 = (int64_t)blockIdx.y * (16 * MT);
    const int K = (int)p.K;

    auto rows = [&](int block) {
        const int c0 = (block * W + s.wave) * CW;
#pragma unroll
        for (int i = 0; i < CW; ++i)
#pragma unroll
            for (int m = 0; m < MT; ++m) {
#pragma unroll
                for (int t = 0; t < 4; ++t)
                    s.a[i][m][0][t] = splat4(0);
                const int64_t row = row0 + 16 * m + l16;
                if (c0 + i < p.w.chunks && row < p.M)
                    load_chunk(s.a[i][m][0], p.A + row * p.K, c0 + i, kq, K);
            }
    };
    auto load = [&](int block, int index, typename S::Words& b, bool some) {
        s.load_w4(b, 0, p.w, panel0 + index, (block * W + s.wave) * CW, some);
    };
    auto done = [&](int block, int index, int m, f32x4_t (&sum)[1]) {
        f32x4_t* held = part + (index * MT + m) * 64 + lane;
        if (block > 0)
            sum[0] += *held;
        if (block + 1 < p.blocks)
            *held = sum[0];
        else
            store_tile(p, row0 + 16 * m, (int64_t)(panel0 + index) * 16, sum[0], fresh(lane));
    };
    s.run(p.blocks, n, rows, load, done);
}

template <int MT, int W, int CW>
static int launch_panels(GemmW4Params p, int per, hipStream_t s)
{
    p.blocks = (int)ceil_div(p.w.chunks, W * CW);
    // the sums of K's earlier blocks wait in what LDS is left
    using S = PanelStream<true, true, MT, 1, 1, W, CW, 1, kHalf<MT>>;
    constexpr size_t used = (S::RED + S::MID) * sizeof(f32x4_t);
    static_assert(used + MT * 1024 <= kLdsBytes, "LDS");
    if (p.blocks > 1)
        per = (int)std::min<size_t>(per, (kLdsBytes - used) / (MT * 1024));
    p.per = per;
    const size_t lds = p.blocks > 1 ? (size_t)per * MT * 1024 : 0;
    const dim3 grid((unsigned)ceil_div(p.panels, per), (unsigned)ceil_div(p.M, 16 * MT)), block(64 * W);
    if (p.w.zeros) {
        if (p.w.group >= 128)
            hipLaunchKernelGGL((gemm_w4_panels_kernel<true, MT, W, CW, 4>), grid, block, lds, s, p);
        else
            hipLaunchKernelGGL((gemm_w4_panels_kernel<true, MT, W, CW, 1>), grid, block, lds, s, p);
    } else {
        if (p.w.group >= 128)
            hipLaunchKernelGGL((gemm_w4_panels_kernel<false, MT, W, CW, 4>), grid, block, lds, s, p);
        else
            hipLaunchKernelGGL((gemm_w4_panels_kernel<false, MT, W, CW, 1>), grid, block, lds, s, p);
    }
    return launched("gemm_w4 launch");
}

}  // namespace tg

using namespace tg;

extern "C" int tg_gemm_w4(int64_t M, int64_t N, int64_t K, const void* A, const tg_weight* B, const float* bias,
                          void* C, int dtype, int act)
{
    if (M < 0 || N < 0 || K < 1)
        return set_error(TG_E_INVAL, "M and N must be >= 0, K >= 1");
    if (dtype != TG_BF16 && dtype != TG_BF16_F32OUT)
        return set_error(TG_E_INVAL, "A is bf16: dtype must be TG_BF16 or TG_BF16_F32OUT");
    if (act < TG_ACT_NONE || act > TG_ACT_GELU)
        return set_error(TG_E_INVAL, "unknown activation " + std::to_string(act));
    if (K > (1 << 21) || N > (1 << 21) || M > (1 << 20))
        return set_error(TG_E_UNSUPPORTED, "K and N are at most 2^21, M at most 2^20");
    if (M == 0 || N == 0)
        return TG_OK;
    const int st = check_weight(B, K, N, "gemm_w4");
    if (st != TG_OK)
        return st;
    if (B->format != TG_W_W4)
        return set_error(TG_E_INVAL, "gemm_w4 takes 4-bit weights (gemm_bias_act takes bf16)");
    if (!A || !C || ((uintptr_t)A & 1u) || ((uintptr_t)bias & 3u) || ((uintptr_t)C & (dtype == TG_BF16 ? 1u : 3u)))
        return set_error(TG_E_INVAL, "A, C and bias must be aligned to their elements, A and C not NULL");
    if (!have_device())
        return set_error(TG_E_UNSUPPORTED, "no HIP device");
    GemmW4Params p{};
    p.A = static_cast<const unsigned short*>(A);
    p.w = view_w4(*B, K, N, 0);
    p.bias = bias;
    p.C = C;
    p.M = M;
    p.N = N;
    p.K = K;
    p.panels = (int)ceil_div(N, 16);
    p.out_bf16 = dtype == TG_BF16;
    p.act = act;
    hipStream_t s = current_stream();
    // A workgroup a compute unit, with equal shares of the panels.  Measured on
    // 16 x 28672 x 8192: 7 panels for each of 256 workgroups 26.7 us, 8 for 224
    // 28.5, 4 for 448 40 (two thirds of which start when others end); 16 waves
    // of 2 chunks 26.7, 8 of 4 28.6, 8 of 2 31.6.  With more rows A's fragments
    // leave room for fewer waves.
    const int per = (int)ceil_div(p.panels, kCus);
    if (M <= 16)
        return p.w.chunks <= 16 ? launch_panels<1, 16, 1>(p, per, s) : launch_panels<1, 16, 2>(p, per, s);
    if (M <= 32)
        return launch_panels<2, 16, 1>(p, per, s);
    return launch_panels<4, 8, 2>(p, per, s);
}
