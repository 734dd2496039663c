// Building blocks of the kernels that stream expert and 4-bit weights (gfx950).
//
// Storage of a 4-bit weight W [K][N] (rows are the reduction index):
//   words  [ceil(N/16)][ceil(K/128)][64][4] u32: a panel of 16 columns, cut
//     into chunks of 128 rows of 1 KiB.  Word (l, t) of a chunk holds column
//     l % 16, rows 32 t + 8 (l / 16) + 0..7: what lane l of a wave feeds to
//     the t-th v_mfma_f32_16x16x32_bf16 of the chunk, so one 16-byte load a
//     lane brings a whole chunk, contiguous in memory, with no shuffle.
//     Nibbles 0..3 hold rows 0, 2, 4, 6 of the eight and nibbles 4..7 rows
//     1, 3, 5, 7: the pair (nibble j, nibble j + 4) sits 16 bits apart and
//     lands in the two halves of a dword of the operand in row order.
//   scales [ceil(N/16)][G][16], zero points [ceil(N/16)][G][16] bytes,
//     G = ceil(K / group).  Element = scale * (code - zero), zero = 8 if absent.
//
// Arithmetic.  A code q goes into the top four mantissa bits of a bf16 of
// exponent 4: 16 + q exactly, one shift and one bit-field insert a pair.  Odd
// rows use the complement and the other sign, -(16 + 15 - q) = q - 31, so that
// the constant parts of neighbouring rows cancel while they are summed:
//   sum A (q - z) = [sum_even A (16 + q) + sum_odd A (q - 31)]
//                 + [-24 sum_even A + 23 sum_odd A] + (8 - z) sum A.
// Products of two bf16 are exact in fp32.  The second and third brackets do
// not depend on the column: they are MFMAs against constant operands, shared
// by every panel that a wave works on.  (An offset of 128, the mantissa's low
// bits, would save a shift and cost 8x the cancellation.)  A row of A that
// holds an infinity gives NaN.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kernels/common.hpp"

namespace tg {

constexpr unsigned kCodeMask = 0x00780078u;    // a code in mantissa bits 3..6 of both halves
constexpr unsigned kCodeBase = 0xC1804180u;    // -16 | 16
constexpr unsigned kCentre = 0x41B8C1C0u;      // 23 | -24
constexpr unsigned kOnes = 0x3F803F80u;

__device__ __forceinline__ u32x4_t w4_expand(unsigned w)
{
    w ^= 0xFFFF0000u;                          // complement the odd rows' codes
    return u32x4_t{((w << 3) & kCodeMask) | kCodeBase, ((w >> 1) & kCodeMask) | kCodeBase,
                   ((w >> 5) & kCodeMask) | kCodeBase, ((w >> 9) & kCodeMask) | kCodeBase};
}

__device__ __forceinline__ u32x4_t splat4(unsigned v) { return u32x4_t{v, v, v, v}; }

// One matrix of 4-bit weights on the device.
struct W4View {
    const u32x4_t* words;                      // one lane's four words
    const void* scales;
    const unsigned char* zeros;                // NULL: 8
    int group, scale_f32;
    int chunks, groups;                        // ceil(K / 128), ceil(K / group)
};

__device__ __forceinline__ float w4_scale(const W4View& v, int panel, int g, int n)
{
    const int64_t i = ((int64_t)panel * v.groups + g) * 16 + n;
    if (v.scale_f32)
        return static_cast<const float*>(v.scales)[i];
    return __uint_as_float((unsigned)static_cast<const unsigned short*>(v.scales)[i] << 16);
}

// 8 - zero point
__device__ __forceinline__ float w4_shift(const W4View& v, int panel, int g, int n)
{
    return 8.0f - (float)v.zeros[((int64_t)panel * v.groups + g) * 16 + n];
}

// Eight bf16 at p + k (k < n counted from p); elements at and past n are zero.
// VEC: n a multiple of 8 and p + k 16-byte aligned.
template <bool VEC>
__device__ __forceinline__ u32x4_t load8(const unsigned short* p, int64_t k, int64_t n)
{
    u32x4_t v = splat4(0);
    if constexpr (VEC) {
        if (k < n)
            v = *reinterpret_cast<const u32x4_t*>(p + k);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (k + e < n)
                v[e >> 1] |= (unsigned)p[k + e] << (16 * (e & 1));
    }
    return v;
}

// What a lane holds of a chunk of 128 rows of NT panels: the four words of its
// column, or four fragments of eight bf16; scales and 8 - zero point of the
// chunk's 4 / GS groups (GS: MFMA steps of 32 rows from one scale to the next).
template <bool W4F, int NT, int GS>
struct PanelChunk {
    static constexpr int SC = 4 / GS;
    u32x4_t w[NT][W4F ? 1 : 4];
    float s[NT][SC], d[NT][SC];

    __device__ __forceinline__ void load_w4(const W4View& v, int j, int panel, int c, int lane)
    {
        w[j][0] = __builtin_nontemporal_load(v.words + ((int64_t)panel * v.chunks + c) * 64 + lane);
#pragma unroll
        for (int i = 0; i < SC; ++i) {
            // past the last group A is zero: any finite scale of the column will do
            const int g = min(SC == 1 ? (int)((int64_t)c * 128 / v.group) : c * SC + i, v.groups - 1);
            s[j][i] = w4_scale(v, panel, g, lane & 15);
            d[j][i] = v.zeros ? w4_shift(v, panel, g, lane & 15) : 0.0f;
        }
    }

    // column `col` of a matrix stored [N][K], its K elements at p + col * K
    template <bool VEC>
    __device__ __forceinline__ void load_bf16(const unsigned short* p, int j, int64_t col, int c, int64_t K, int lane)
    {
#pragma unroll
        for (int t = 0; t < 4; ++t)
            w[j][t] = load8<VEC>(p + col * K, (int64_t)c * 128 + 32 * t + 8 * (lane >> 4), K);
    }
};

// total += A . W over one chunk, for the row tiles whose bit is set in `tiles`
// (the same for the whole wave).  NA: A is the sum of NA bf16 fragments.
template <bool W4F, int MT, int NT, int NA, int GS>
__device__ __forceinline__ void mac_chunk(f32x4_t (&total)[MT][NT], const u32x4_t (&a)[MT][NA][4],
                                          const PanelChunk<W4F, NT, GS>& b, bool zero, unsigned tiles)
{
    const f32x4_t none = {0.f, 0.f, 0.f, 0.f};
    if constexpr (W4F) {
        f32x4_t acc[MT][NT], mid[MT], sum[MT];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            if (t % GS == 0) {
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    mid[m] = sum[m] = none;
#pragma unroll
                    for (int j = 0; j < NT; ++j)
                        acc[m][j] = none;
                }
            }
            u32x4_t q[NT];
#pragma unroll
            for (int j = 0; j < NT; ++j)
                q[j] = w4_expand(b.w[j][0][t]);
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                if (!(tiles >> m & 1))
                    continue;
#pragma unroll
                for (int n = 0; n < NA; ++n) {
                    mid[m] = mfma_bf16(a[m][n][t], splat4(kCentre), mid[m]);
                    if (zero)
                        sum[m] = mfma_bf16(a[m][n][t], splat4(kOnes), sum[m]);
#pragma unroll
                    for (int j = 0; j < NT; ++j)
                        acc[m][j] = mfma_bf16(a[m][n][t], q[j], acc[m][j]);
                }
            }
            if (t % GS == GS - 1) {
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    if (!(tiles >> m & 1))
                        continue;
#pragma unroll
                    for (int j = 0; j < NT; ++j)
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            float v = acc[m][j][r] + mid[m][r];
                            if (zero)
                                v = fmaf(b.d[j][t / GS], sum[m][r], v);
                            total[m][j][r] = fmaf(b.s[j][t / GS], v, total[m][j][r]);
                        }
                }
            }
        }
    } else {
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                if (!(tiles >> m & 1))
                    continue;
#pragma unroll
                for (int n = 0; n < NA; ++n)
#pragma unroll
                    for (int j = 0; j < NT; ++j)
                        total[m][j] = mfma_bf16(a[m][n][t], b.w[j][t], total[m][j]);
            }
    }
}

}  // namespace tg
