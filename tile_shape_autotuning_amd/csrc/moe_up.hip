// Gate and up projections of the chosen experts (moe.hip).
#include <hip/hip_runtime.h>

#include <cmath>

#include "moe.hpp"

namespace tg {

// expf: the fast exponential rounds g log2(e) to fp32, and what that is off by
// grows with |g| (2e-6 of the value at g = -80).
__device__ __forceinline__ float gated(float g, float u, int gelu)
{
    return (gelu ? gelu_erf(g) : g / (1.0f + expf(-g))) * u;
}

template <bool W4F, bool ZERO, int MT, int W, int CW, int GS, bool VEC, bool ONE>
__global__ void __launch_bounds__(64 * W) moe_up_kernel(MoeParams p)
{
    using S = PanelStream<W4F, ZERO, MT, 2, 1, W, CW, GS, ONE ? 1 : 32>;
    __shared__ f32x4_t red[S::RED], mid[S::MID];
    __shared__ int ids[kTokens * kMaxChoices];
    __shared__ unsigned bits[kExpertWords];
    extern __shared__ f32x4_t part[];                  // [p.up_per][MT][2][64] if it is used
    S s(red, mid, p.up.w4.scale_f32);
    const int lane = s.lane, l16 = lane & 15;
    Share e;
    if (!share_of(p, blockIdx.y, ids, bits, p.weights, lane, e))
        return;
    const int panel0 = blockIdx.x * p.up_per;
    const int n = min(p.up_per, p.up.panels - panel0);
    const W4Source v[2] = {W4Source(matrix(p.up, 2 * (int64_t)e.expert), panel0, p.up.panels),
                           W4Source(matrix(p.up, 2 * (int64_t)e.expert + 1), panel0, p.up.panels)};
    const unsigned short* wb = p.up.bf16 + (W4F ? 0 : 2 * (int64_t)e.expert * p.I * p.H);

    for (int r0 = 0; r0 < e.rows; r0 += 16 * MT) {
        auto rows = [&](int block, typename S::Rows& x, bool some) {
            const int c0 = (block * W + s.wave) * CW;
            const __amdgpu_buffer_rsrc_t rx = wave_rsrc(p.x, some ? (int64_t)p.T * p.H * 2 : 0);
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const int r = r0 + 16 * m + l16, t = __shfl(e.pair, r & 63) / p.k;
                if constexpr (VEC)
                    s.load_rows(x, m, rx, r < e.rows ? t * p.H * 2 : kOOB, p.H, c0);
                else
                    s.load_rows(x, m, some && r < e.rows ? p.x + (int64_t)t * p.H : nullptr, p.H, c0);
            }
        };
        auto load = [&](int block, int index, typename S::Words& b, bool some) {
            const int c0 = (block * W + s.wave) * CW;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                if constexpr (W4F)
                    s.load_w4(b, j, v[j], index, c0, some);
                else
                    s.template load_bf16<VEC>(b, j, wb + (int64_t)j * p.I * p.H, p.I, p.H, panel0 + index, c0, some);
            }
        };
        auto done = [&](int block, int index, int m, f32x4_t (&sum)[2]) {
            if constexpr (!ONE) {
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
                p.h[(int64_t)to * p.stride + col] = col < p.I ? w * gated(sum[0][r], sum[1][r], p.gelu) : 0.0f;
            }
        };
        if constexpr (ONE)
            s.run_one(p.up_blocks, rows, load, done);
        else
            s.template run<kDepth<W4F>>(p.up_blocks, n, rows, load, done);
    }
}

struct Up {
    static constexpr int kMany = 2;
    template <bool W4F, bool ZERO, int MT, int CW, int GS, bool VEC>
    static void go(MoeParams p, hipStream_t s)
    {
        constexpr int W = 8;
        using S = PanelStream<W4F, ZERO, MT, 2, 1, W, CW, GS, 32>;
        constexpr size_t used = (S::RED + S::MID) * 16 + (kTokens * kMaxChoices + kExpertWords) * 4;
        static_assert(used + MT * 2048 <= kLdsBytes, "LDS");
        const int slots = std::min(p.E, p.T * p.k);
        static const int resident = resident_on_cu(moe_up_kernel<W4F, ZERO, MT, W, CW, GS, VEC, false>, 64 * W);
        p.up_blocks = (int)ceil_div(ceil_div(p.H, 128), W * CW);
        p.up_per = panels_per(p.up.panels, p, resident, p.up_blocks, used, MT * 2048);
        const bool one = MT == 1 && VEC && p.up_per == 1 && p.up_blocks > 1;
        const size_t lds = p.up_blocks > 1 && !one ? (size_t)p.up_per * MT * 2048 : 0;
        const dim3 grid((unsigned)ceil_div(p.up.panels, p.up_per), (unsigned)slots);
        if constexpr (MT == 1 && VEC) {
            if (one) {
                hipLaunchKernelGGL((moe_up_kernel<W4F, ZERO, MT, W, CW, GS, VEC, true>), grid, dim3(64 * W), 0, s, p);
                return;
            }
        }
        hipLaunchKernelGGL((moe_up_kernel<W4F, ZERO, MT, W, CW, GS, VEC, false>), grid, dim3(64 * W), lds, s, p);
    }
};

int launch_up(const MoeParams& p, const tg_weight& w, hipStream_t s)
{
    by_weight<Up>(w, p.H, p.H % 8 == 0 && ((uintptr_t)p.x & 15u) == 0, p, s);
    return launched("moe gate and up launch");
}

}  // namespace tg
