// C = act(A . W + bias), W in 4 bits with group scales (storage and
// arithmetic: w4.hpp).
//
// Few rows: the panels of W stream past rows kept in registers (panel_stream.hpp).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <string>
#include <type_traits>

#include "kernels/gemm_tiled_dma.hpp"
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
// beyond the waves' W x CW chunks comes in further blocks; with more than one
// panel (!ONE) the sums of the earlier blocks wait in LDS.
template <bool ZERO, int MT, int W, int CW, int GS, bool VEC, bool ONE>
__global__ void __launch_bounds__(64 * W) gemm_w4_panels_kernel(GemmW4Params p)
{
    using S = PanelStream<true, ZERO, MT, 1, 1, W, CW, GS, ONE ? 1 : kHalf<MT>>;
    __shared__ f32x4_t red[S::RED], mid[S::MID];
    extern __shared__ f32x4_t part[];                  // [p.per][MT][64] if it is used
    S s(red, mid, p.w.scale_f32);
    const int lane = s.lane, l16 = lane & 15;
    const int panel0 = blockIdx.x * p.per;
    const int n = min(p.per, p.panels - panel0);
    const int64_t row0 = (int64_t)blockIdx.y * (16 * MT);
    const int K = (int)p.K, here = (int)min((int64_t)(16 * MT), p.M - row0);
    const unsigned short* A = p.A + row0 * K;

    const W4Source source(p.w, panel0, p.panels);
    auto rows = [&](int block, typename S::Rows& x, bool some) {
        const int c0 = (block * W + s.wave) * CW;
        const __amdgpu_buffer_rsrc_t r = wave_rsrc(A, some ? (int64_t)here * K * 2 : 0);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const int row = 16 * m + l16;
            if constexpr (VEC)
                s.load_rows(x, m, r, row < here ? row * K * 2 : kOOB, K, c0);
            else
                s.load_rows(x, m, some && row < here ? A + (int64_t)row * K : nullptr, K, c0);
        }
    };
    auto load = [&](int block, int index, typename S::Words& b, bool some) {
        s.load_w4(b, 0, source, index, (block * W + s.wave) * CW, some);
    };
    auto done = [&](int block, int index, int m, f32x4_t (&sum)[1]) {
        if constexpr (!ONE) {
            f32x4_t* held = part + (index * MT + m) * 64 + lane;
            if (block > 0)
                sum[0] += *held;
            if (block + 1 < p.blocks) {
                *held = sum[0];
                return;
            }
        }
        store_tile(p, row0 + 16 * m, (int64_t)(panel0 + index) * 16, sum[0], fresh(lane));
    };
    if constexpr (ONE)
        s.run_one(p.blocks, rows, load, done);
    else
        s.template run<4>(p.blocks, n, rows, load, done);
}

using One = std::integral_constant<int, 1>;
using Two = std::integral_constant<int, 2>;
using Four = std::integral_constant<int, 4>;

// f(zero points?, MFMA steps between scales) as constants
template <class F>
static void by_storage(const W4View& w, const F& f)
{
    auto pick = [&](auto zero) {
        w.group >= 128 ? f(zero, Four{}) : w.group == 64 ? f(zero, Two{}) : f(zero, One{});
    };
    w.zeros ? pick(std::true_type{}) : pick(std::false_type{});
}

static bool aligned_rows(const GemmW4Params& p) { return p.K % 8 == 0 && ((uintptr_t)p.A & 15u) == 0; }

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
    per = std::min(per, panels_in_reach(p.w.chunks));
    p.per = per;
    // rows for two blocks at once do not fit in registers with MT = 4
    const bool vec = aligned_rows(p), one = MT < 4 && vec && per == 1 && p.blocks > 1;
    const size_t lds = p.blocks > 1 && !one ? (size_t)per * MT * 1024 : 0;
    const dim3 grid((unsigned)ceil_div(p.panels, per), (unsigned)ceil_div(p.M, 16 * MT)), block(64 * W);
    by_storage(p.w, [&](auto zero, auto gs) {
        constexpr bool Z = decltype(zero)::value;
        constexpr int G = decltype(gs)::value;
        if constexpr (MT < 4) {
            if (one) {
                hipLaunchKernelGGL((gemm_w4_panels_kernel<Z, MT, W, CW, G, true, true>), grid, block, 0, s, p);
                return;
            }
        }
        if (vec)
            hipLaunchKernelGGL((gemm_w4_panels_kernel<Z, MT, W, CW, G, true, false>), grid, block, lds, s, p);
        else
            hipLaunchKernelGGL((gemm_w4_panels_kernel<Z, MT, W, CW, G, false, false>), grid, block, lds, s, p);
    });
    return launched("gemm_w4 launch");
}

// Many rows: a workgroup's four waves stand side by side over 64 NT columns and
// share MT x 16 rows of A, whose chunks of 128 k arrive in LDS (16-byte
// transfers straight from memory, three stages).  W's codes are a quarter of
// A's bytes, so tiles are wide rather than tall, and no two waves expand the
// same codes: with MT = NT = 4, 144 expanding instructions a chunk beside 64
// MFMAs, 64 FMAs of the scales and as many copies of the starting sums.  The sums that do not depend on the column
// (w4.hpp) are computed one chunk ahead, each wave a quarter of the rows, and
// start the accumulators.  One barrier a chunk; it and the transfers are
// covered by the other workgroups of the compute unit (two of 256 registers
// with NT = 4, three with NT = 2).  Calls back to back: 2048 x 4096 x 4096 78 to
// 85 us, 0.85 PFLOP/s (zero points 98; groups of 64 91 and 143, of 32 107 and
// 142; K one less, through registers, 117); 4096 x 8192 x 8192 580 us, 0.95
// PFLOP/s.  By counters the first keeps the matrix cores busy 42 % of the time
// and the vector units 50 % with what is beside them (324 instructions and 68
// MFMAs a wave and chunk): two waves a SIMD hide little of one behind the
// other, and wait for the chunk's transfers and its barrier 23 % of theirs.
//
// Stage layout: row r of A, 256 bytes, 16-byte piece q at q ^ swz<16>(r): the
// 16 rows of a fragment read hit 16 different pieces.
template <bool ZERO, int MT, int NT, int GS>
struct TiledW4 {
    static constexpr int BM = 16 * MT, SC = 4 / GS, STAGE = BM * 256, STAGES = 3;
    static constexpr int MIDS = SC * MT * 4 * (ZERO ? 2 : 1);          // f32x4, held twice
    static constexpr int LDS = STAGES * STAGE + 2 * MIDS * 16;
};

template <bool ZERO, int MT, int NT, int GS, bool VEC>
__global__ void __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(NT == 1 ? 4 : NT == 2 ? 3 : 2)))
gemm_w4_tiled_kernel(GemmW4Params p)
{
    using T = TiledW4<ZERO, MT, NT, GS>;
    constexpr int SC = T::SC, BM = T::BM;
    extern __shared__ u32x4_t lds[];
    f32x4_t* mids = reinterpret_cast<f32x4_t*>(lds + T::STAGES * T::STAGE / 16);
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int l16 = lane & 15, kq = lane >> 4;
    const int tiles_n = (p.panels + 4 * NT - 1) / (4 * NT), tiles_m = (int)((p.M + BM - 1) / BM);
    int tile, tm, tn, split;
    map_block(blockIdx.x, gridDim.x, tiles_m, tiles_n, 8, tile, tm, tn, split);
    const int64_t row0 = (int64_t)tm * BM;
    const int panel0 = (tn * 4 + wave) * NT;
    const int K = (int)p.K, chunks = p.w.chunks;
    const int rows = (int)min((int64_t)BM, p.M - row0);
    const unsigned short* A = p.A + row0 * K;
    const CodeConsts code;
    const unsigned up = p.w.scale_f32 || (lane & 1) ? 0 : 16, keep = p.w.scale_f32 ? ~0u : 0xFFFF0000u;

    // A's chunk c into its stage: transfer j brings rows 4 j .. 4 j + 3
    const i32x4_t ra = rsrc_words(A, (int64_t)rows * K * 2);
    const unsigned lds0 = (unsigned)(uintptr_t)(__attribute__((address_space(3))) void*)lds;
    auto fetch = [&](int c) {
        const unsigned base = c % T::STAGES * T::STAGE;
#pragma unroll
        for (int q = 0; q < BM / 16; ++q) {
            const int j = q * 4 + wave, row = 4 * j + kq;
            const int k = c * 128 + (l16 ^ swz<16>(row)) * 8;
            if constexpr (VEC) {
                dma16(ra, row < rows && k < K ? (row * K + k) * 2 : kOOB, lds0 + base + j * 1024);
            } else {
                u32x4_t v = splat4(0);
                if (row < rows)
                    v = load8(A + (int64_t)row * K, k, K);
                lds[base / 16 + j * 64 + lane] = v;
            }
        }
    };
    auto fragment = [&](int c, int m, int t) {
        const int row = 16 * m + l16;
        return lds[c % T::STAGES * (T::STAGE / 16) + row * 16 + ((4 * t + kq) ^ swz<16>(row))];
    };
    // the constant sums of chunk c: this wave's quarter of the rows
    auto correct = [&](int c) {
        f32x4_t* to = mids + (c & 1) * T::MIDS;
        const f32x4_t none = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int h = 0; h < MT / 4; ++h) {
            const int m = wave * (MT / 4) + h;
#pragma unroll
            for (int q = 0; q < SC; ++q) {
                f32x4_t v = none, s = none;
#pragma unroll
                for (int t = q * GS; t < (q + 1) * GS; ++t) {
                    const u32x4_t a = fragment(c, m, t);
                    v = mfma_bf16(a, splat4(kCentre), v);
                    if constexpr (ZERO)
                        s = mfma_bf16(a, splat4(kOnes), s);
                }
                if (l16 == 0) {
                    to[(q * MT + m) * 4 + kq] = v;
                    if constexpr (ZERO)
                        to[(SC * MT + q * MT + m) * 4 + kq] = s;
                }
            }
        }
    };
    // With several groups a chunk, each quarter of the wave holds one's scale and
    // zero point.
    struct Words {
        u32x4_t w[NT];
        unsigned s[NT];
        unsigned char z[NT];
    };
    auto load = [&](int c, Words& b) {
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const int panel = panel0 + j;
            const bool some = panel < p.panels && c < chunks;
            const __amdgpu_buffer_rsrc_t rw =
                wave_rsrc(p.w.words + (int64_t)panel * chunks * 64, some ? (int64_t)chunks * 1024 : 0);
            const int64_t per = (int64_t)panel * p.w.groups * 16;
            const int n = some ? p.w.groups * 16 : 0;
            const __amdgpu_buffer_rsrc_t rs = wave_rsrc(
                static_cast<const char*>(p.w.scales) + per * (p.w.scale_f32 ? 4 : 2), n * (p.w.scale_f32 ? 4 : 2));
            const __amdgpu_buffer_rsrc_t rz = wave_rsrc(p.w.zeros + (ZERO ? per : 0), n);
            b.w[j] = load16(rw, c * 1024 + lane * 16);
            const int k = c * 128 + (SC == 1 ? 0 : 32 * GS * min(kq, SC - 1));
            const int at = (int)((unsigned)k / (unsigned)p.w.group) * 16 + l16;
            b.s[j] = load4(rs, p.w.scale_f32 ? at * 4 : at / 2 * 4);
            if constexpr (ZERO)
                b.z[j] = __builtin_amdgcn_raw_buffer_load_b8(rz, at, 0, 0);
        }
    };

    f32x4_t total[MT][NT];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int j = 0; j < NT; ++j)
            total[m][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};

    auto multiply = [&](int c, const Words& b) {
        const f32x4_t* from = mids + (c & 1) * T::MIDS;
        float scale[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j)
            scale[j] = __uint_as_float((b.s[j] << up) & keep);
        f32x4_t acc[MT][NT];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const int q = t / GS;
            u32x4_t w[NT];
#pragma unroll
            for (int j = 0; j < NT; ++j)
                w[j] = w4_expand(b.w[j][t], code);
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const u32x4_t a = fragment(c, m, t);
                if (t % GS == 0) {
                    const f32x4_t v = from[(q * MT + m) * 4 + kq];
#pragma unroll
                    for (int j = 0; j < NT; ++j)
                        acc[m][j] = v;
                }
#pragma unroll
                for (int j = 0; j < NT; ++j)
                    acc[m][j] = mfma_bf16(a, w[j], acc[m][j]);
            }
            if (t % GS == GS - 1) {
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    const float sc = SC == 1 ? scale[j]
                                             : __int_as_float(__builtin_amdgcn_ds_bpermute(
                                                   4 * (16 * q + l16), __float_as_int(scale[j])));
                    float d = 0.0f;
                    if constexpr (ZERO && SC == 1)
                        d = 8.0f - (float)b.z[j];
#pragma unroll
                    for (int m = 0; m < MT; ++m) {
                        f32x4_t s = {0.f, 0.f, 0.f, 0.f};
                        if constexpr (ZERO && SC == 1)
                            s = from[(MT + m) * 4 + kq];
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            total[m][j][r] = fmaf(
                                sc, ZERO && SC == 1 ? fmaf(d, s[r], acc[m][j][r]) : acc[m][j][r], total[m][j][r]);
                    }
                }
                // the scheduler would begin all groups at once, and spill
                if constexpr (SC > 1)
                    __builtin_amdgcn_sched_barrier(0);
            }
        }
        // (8 - z) sum A of several groups: one fp32 MFMA a tile, whose k is the group
        if constexpr (ZERO && SC > 1) {
            const float* sums = reinterpret_cast<const float*>(from + SC * MT * 4);
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const float sum = kq < SC ? sums[(kq * MT + m) * 16 + l16] : 0.0f;
#pragma unroll
                for (int j = 0; j < NT; ++j)
                    total[m][j] = mfma_f32(sum, kq < SC ? scale[j] * (8.0f - (float)b.z[j]) : 0.0f, total[m][j]);
            }
        }
    };

    Words b[2];
    load(0, b[0]);
    fetch(0);
    fetch(1);
    wait_vm_all();
    lds_barrier();
    correct(0);
    // the transfers are not the compiler's to wait for: every chunk waits for
    // all that is on its way, A's chunk c + 1 and the words of chunk c, both
    // asked for a whole chunk ago
    auto one = [&](int c, const Words& now, Words& next) {
        wait_vm_all();
        lds_barrier();
        load(c + 1, next);
        fetch(c + 2);
        correct(c + 1);
        multiply(c, now);
        return c + 1 < chunks;
    };
    for (int c = 0;; c += 2)
        if (!one(c, b[0], b[1]) || !one(c + 1, b[1], b[0]))
            break;
    // nothing may still be writing LDS when the workgroup ends
    wait_vm_all();

#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int j = 0; j < NT; ++j)
            store_tile(p, row0 + 16 * m, (int64_t)(panel0 + j) * 16, total[m][j], lane);
}

template <int MT, int NT>
static int launch_tiled(const GemmW4Params& p, hipStream_t s)
{
    const bool vec = aligned_rows(p);
    const dim3 grid((unsigned)(ceil_div(p.panels, 4 * NT) * ceil_div(p.M, 16 * MT))), block(256);
    by_storage(p.w, [&](auto zero, auto gs) {
        constexpr bool Z = decltype(zero)::value;
        // groups of 64 with zero points as pairs of 32: the kernel for two groups a chunk spills (2048 x 4096 x
        // 4096 565 us, so 141)
        constexpr int G = Z && decltype(gs)::value == 2 ? 1 : decltype(gs)::value;
        constexpr size_t lds = TiledW4<Z, MT, NT, G>::LDS;
        if (vec)
            hipLaunchKernelGGL((gemm_w4_tiled_kernel<Z, MT, NT, G, true>), grid, block, lds, s, p);
        else
            hipLaunchKernelGGL((gemm_w4_tiled_kernel<Z, MT, NT, G, false>), grid, block, lds, s, p);
    });
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
    const int st = check_weight(B, "gemm_w4");
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
    p.w = view_w4(*B, K);
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
    const int64_t cus = compute_units();
    const int per = (int)ceil_div(p.panels, cus);
    if (M <= 16)
        return p.w.chunks <= 16 ? launch_panels<1, 16, 1>(p, per, s) : launch_panels<1, 16, 2>(p, per, s);
    if (M <= 32)
        return launch_panels<2, 16, 1>(p, per, s);
    if (M <= 64)
        return p.w.chunks <= 8 ? launch_panels<4, 8, 1>(p, per, s) : launch_panels<4, 8, 2>(p, per, s);
    // 64 x 256 tiles where two workgroups a compute unit have one, 64 x 128 where
    // one has, else 64 x 64.  Symmetric groups of 128 in the three: 2048 x 4096 x
    // 4096 86, 95 and 126 us, 512 x 4096 x 4096 53, 37 and 39, 100 x 28672 x 4096
    // 54, 48 and 67, 128 x 4096 x 4096 52, 35 and 30; groups of 32 with zero
    // points 143, 179 and 261, 111, 82 and 87, 112, 98 and 166, 112, 81 and 77.
    // At eight shapes in all six storage forms the rule's tile is within 6 % of
    // the best, but where the widest just misses two workgroups (256 x 28672 x
    // 4096, 448 tiles: 79 and 89 us, groups of 32 with zero points 142 and 182).
    // (128 x 256 leaves one workgroup a compute unit: 151 us for the first.)
    if (ceil_div(M, 64) * ceil_div(p.panels, 16) >= 2 * cus)
        return launch_tiled<4, 4>(p, s);
    if (ceil_div(M, 64) * ceil_div(p.panels, 8) >= cus)
        return launch_tiled<4, 2>(p, s);
    return launch_tiled<4, 1>(p, s);
}
