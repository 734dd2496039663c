// Down projections of the chosen experts (moe.hip).
#include <hip/hip_runtime.h>

#include "moe.hpp"

namespace tg {

template <bool W4F, bool ZERO, int MT, int W, int CW, int GS, bool VEC, bool ONE>
__global__ void __launch_bounds__(64 * W) moe_down_kernel(MoeParams p)
{
    using S = PanelStream<W4F, ZERO, MT, 1, 3, W, CW, GS, ONE ? 1 : 32>;
    __shared__ f32x4_t red[S::RED], mid[S::MID];
    __shared__ int ids[kTokens * kMaxChoices];
    __shared__ unsigned bits[kExpertWords];
    extern __shared__ f32x4_t part[];                  // [p.down_per][MT][64] if it is used
    S s(red, mid, p.down.w4.scale_f32);
    const int lane = s.lane, l16 = lane & 15;
    Share e;
    if (!share_of(p, blockIdx.y, ids, bits, nullptr, lane, e))
        return;
    const int panel0 = blockIdx.x * p.down_per;
    const int n = min(p.down_per, p.down.panels - panel0);
    const W4Source v(matrix(p.down, e.expert), panel0, p.down.panels);
    const unsigned short* wb = p.down.bf16 + (W4F ? 0 : (int64_t)e.expert * p.H * p.I);

    for (int r0 = 0; r0 < e.rows; r0 += 16 * MT) {
        auto rows = [&](int block, typename S::Rows& x, bool some) {
            const int c0 = (block * W + s.wave) * CW;
            const __amdgpu_buffer_rsrc_t rh = wave_rsrc(p.h, some ? (int64_t)p.T * p.k * p.stride * 4 : 0);
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const int r = r0 + 16 * m + l16, pair = __shfl(e.pair, r & 63);
                s.load_floats(x, m, rh, r < e.rows ? pair * (int)p.stride * 4 : kOOB, (int)p.stride, c0);
            }
        };
        auto load = [&](int block, int index, typename S::Words& b, bool some) {
            const int c0 = (block * W + s.wave) * CW;
            if constexpr (W4F)
                s.load_w4(b, 0, v, index, c0, some);
            else
                s.template load_bf16<VEC>(b, 0, wb, p.H, p.I, panel0 + index, c0, some);
        };
        auto done = [&](int block, int index, int m, f32x4_t (&sum)[1]) {
            if constexpr (!ONE) {
                f32x4_t* held = part + (index * MT + m) * 64 + lane;
                if (block > 0)
                    sum[0] += *held;
                if (block + 1 < p.down_blocks) {
                    *held = sum[0];
                    return;
                }
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
        if constexpr (ONE)
            s.run_one(p.down_blocks, rows, load, done);
        else
            s.template run<kDepth<W4F>>(p.down_blocks, n, rows, load, done);
    }
}

struct Down {
    // rows of two tiles and two chunks in three parts do not fit in registers (64
    // tokens over 8 4-bit experts of 2048 x 1408: 95 us, with one chunk 65)
    static constexpr int kMany = 1;
    template <bool W4F, bool ZERO, int MT, int CW, int GS, bool VEC>
    static void go(MoeParams p, hipStream_t s)
    {
        constexpr int W = 8;
        using S = PanelStream<W4F, ZERO, MT, 1, 3, W, CW, GS, 32>;
        constexpr size_t used = (S::RED + S::MID) * 16 + (kTokens * kMaxChoices + kExpertWords) * 4;
        static_assert(used + MT * 1024 <= kLdsBytes, "LDS");
        const int slots = std::min(p.E, p.T * p.k);
        static const int resident = resident_on_cu(moe_down_kernel<W4F, ZERO, MT, W, CW, GS, VEC, false>, 64 * W);
        p.down_blocks = (int)ceil_div(ceil_div(p.I, 128), W * CW);
        p.down_per = panels_per(p.down.panels, p, resident, p.down_blocks, used, MT * 1024);
        const bool one = MT == 1 && VEC && p.down_per == 1 && p.down_blocks > 1;
        const size_t lds = p.down_blocks > 1 && !one ? (size_t)p.down_per * MT * 1024 : 0;
        const dim3 grid((unsigned)ceil_div(p.down.panels, p.down_per), (unsigned)slots);
        if constexpr (MT == 1 && VEC) {
            if (one) {
                hipLaunchKernelGGL((moe_down_kernel<W4F, ZERO, MT, W, CW, GS, VEC, true>), grid, dim3(64 * W), 0, s, p);
                return;
            }
        }
        hipLaunchKernelGGL((moe_down_kernel<W4F, ZERO, MT, W, CW, GS, VEC, false>), grid, dim3(64 * W), lds, s, p);
    }
};

int launch_down(const MoeParams& p, const tg_weight& w, hipStream_t s)
{
    by_weight<Down>(w, p.I, w.format == TG_W_W4 || p.I % 8 == 0, p, s);
    return launched("moe down launch");
}

}  // namespace tg
