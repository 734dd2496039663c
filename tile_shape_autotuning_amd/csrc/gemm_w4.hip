// C = act(A . W + bias), W in 4 bits with group scales (storage and
// arithmetic: w4.hpp).
//
// The streaming kernel.  With few rows every weight is used once and the
// kernel is bound by the stream of words from HBM.  A workgroup owns NT panels
// of 16 columns and MT tiles of 16 rows; its W waves take interleaved chunks of
// 128 rows of W (adjacent waves read adjacent KiB), one 16-byte load a lane and
// panel.  A's fragments come straight from L2: no two waves of a workgroup
// need the same ones.  The next chunk's loads are issued before the current
// chunk's MFMAs.  Sums over a group stay in their own accumulators until the
// group's scale multiplies them into the fp32 totals; the waves' totals meet
// in LDS in wave order, so results do not depend on timing.
#include <hip/hip_runtime.h>

#include <string>

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
};

// GS: MFMA steps (of 32 rows) between two scales: 1, 2 or 4 (a whole chunk)
template <int MT, int NT, int W, int GS, bool VEC>
__global__ void __launch_bounds__(64 * W) gemm_w4_stream_kernel(GemmW4Params p)
{
    __shared__ f32x4_t red[W * MT * NT * 64];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int l16 = lane & 15, kq = lane >> 4;
    const int panel0 = blockIdx.x * NT;
    const int64_t row0 = (int64_t)blockIdx.y * (16 * MT);
    const bool zero = p.w.zeros != nullptr;

    struct Buf {
        PanelChunk<true, NT, GS> w;
        u32x4_t a[MT][1][4];
    };
    auto load = [&](int c, Buf& b) {
#pragma unroll
        for (int j = 0; j < NT; ++j)
            b.w.load_w4(p.w, j, min(panel0 + j, p.panels - 1), c, lane);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const int64_t row = row0 + 16 * m + l16;
#pragma unroll
            for (int t = 0; t < 4; ++t)
                b.a[m][0][t] = row < p.M ? load8<VEC>(p.A + row * p.K, (int64_t)c * 128 + 32 * t + 8 * kq, p.K)
                                         : splat4(0);
        }
    };

    const f32x4_t none = {0.f, 0.f, 0.f, 0.f};
    f32x4_t total[MT][NT];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int j = 0; j < NT; ++j)
            total[m][j] = none;

    auto use = [&](const Buf& b) { mac_chunk<true, MT, NT, 1, GS>(total, b.a, b.w, zero, ~0u); };

    Buf buf[2];
    int c = wave;
    if (c < p.w.chunks)
        load(c, buf[0]);
    for (; c < p.w.chunks; c += 2 * W) {
        if (c + W < p.w.chunks)
            load(c + W, buf[1]);
        use(buf[0]);
        if (c + W < p.w.chunks) {
            if (c + 2 * W < p.w.chunks)
                load(c + 2 * W, buf[0]);
            use(buf[1]);
        }
    }

#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int j = 0; j < NT; ++j)
            red[((m * NT + j) * W + wave) * 64 + lane] = total[m][j];
    __syncthreads();
    // tile i of the workgroup's MT x NT is finished by wave i % W
    for (int i = wave; i < MT * NT; i += W) {
        f32x4_t v = none;
#pragma unroll
        for (int q = 0; q < W; ++q)
            v += red[(i * W + q) * 64 + lane];
        const int64_t col = (int64_t)(panel0 + i % NT) * 16 + l16;
        if (col >= p.N)
            continue;
        const float bias = p.bias ? p.bias[col] : 0.0f;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int64_t row = row0 + (i / NT) * 16 + kq * 4 + r;
            if (row >= p.M)
                continue;
            const float x = apply_act(v[r] + bias, p.act);
            if (p.out_bf16)
                static_cast<unsigned short*>(p.C)[row * p.N + col] = f32_to_bf16_rne(x);
            else
                static_cast<float*>(p.C)[row * p.N + col] = x;
        }
    }
}

template <int MT, int NT, int W>
static int launch_stream(const GemmW4Params& p, bool vec, hipStream_t s)
{
    const dim3 grid((unsigned)ceil_div(p.panels, NT), (unsigned)ceil_div(p.M, 16 * MT)), block(64 * W);
    const int gs = p.w.group >= 128 ? 4 : p.w.group / 32;
#define TG_LAUNCH(GS, VEC) hipLaunchKernelGGL((gemm_w4_stream_kernel<MT, NT, W, GS, VEC>), grid, block, 0, s, p)
    if (vec) {
        if (gs == 4) TG_LAUNCH(4, true); else if (gs == 2) TG_LAUNCH(2, true); else TG_LAUNCH(1, true);
    } else {
        if (gs == 4) TG_LAUNCH(4, false); else if (gs == 2) TG_LAUNCH(2, false); else TG_LAUNCH(1, false);
    }
#undef TG_LAUNCH
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
    const bool vec = K % 8 == 0 && ((uintptr_t)A & 15u) == 0;
    hipStream_t s = current_stream();
    if (M <= 16)
        return launch_stream<1, 1, 8>(p, vec, s);
    if (M <= 32)
        return launch_stream<2, 2, 8>(p, vec, s);
    return launch_stream<4, 2, 8>(p, vec, s);
}
