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
// bits, would save a shift and cost 8x the cancellation.)  Partial sums of a
// chunk reach 31 S, S the sum of |A| over its k: up to S = 2^123 nothing
// overflows.  A row of A beyond, or with an infinity, gives NaN.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kernels/common.hpp"

namespace tg {

constexpr unsigned kCodeMask = 0x00780078u;    // a code in mantissa bits 3..6 of both halves
constexpr unsigned kCodeBase = 0xC1804180u;    // -16 | 16
constexpr unsigned kCentre = 0x41B8C1C0u;      // 23 | -24
constexpr unsigned kOnes = 0x3F803F80u;

// The two constants of w4_expand, where one instruction can take them both (a
// scalar register and a vector register: three-operand instructions hold no
// literals), opaque to the compiler, which would fold them back into literals.
struct CodeConsts {
    unsigned mask, base;
    __device__ __forceinline__ CodeConsts() : mask(kCodeMask), base(kCodeBase)
    {
        __asm__ __volatile__("" : "+s"(mask), "+v"(base));
    }
};

__device__ __forceinline__ u32x4_t w4_expand(unsigned w, const CodeConsts& k)
{
    w ^= 0xFFFF0000u;                          // complement the odd rows' codes
    return u32x4_t{((w << 3) & k.mask) | k.base, ((w >> 1) & k.mask) | k.base, ((w >> 5) & k.mask) | k.base,
                   ((w >> 9) & k.mask) | k.base};
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

// A pointer that is the same in the whole wave, said so: where the compiler's
// analysis loses track of that it wraps every buffer load in a loop over the
// lanes' descriptors.
__device__ __forceinline__ const void* same_in_wave(const void* p)
{
    const uint64_t a = reinterpret_cast<uint64_t>(p);
    return reinterpret_cast<const void*>(
        (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(a >> 32)) << 32 |
        (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)a));
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t wave_rsrc(const void* base, int64_t bytes)
{
    const int64_t n = bytes < 0 ? 0 : (bytes > kMaxRecords ? kMaxRecords : bytes);
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(same_in_wave(base)), (short)0,
                                             __builtin_amdgcn_readfirstlane((int)n), kRsrcWord3);
}

// Sixteen bytes from any element address: one load, the hardware takes it unaligned.
struct __attribute__((packed, aligned(2))) Unaligned16 {
    u32x4_t v;
};

// Eight bf16 at p + k; elements at and past n are zero and not read.  Where the
// eight reach past n, the last eight are read instead and the ones before k
// shifted out, so that every lane makes one load.
__device__ __forceinline__ u32x4_t load8(const unsigned short* p, int64_t k, int64_t n)
{
    u32x4_t v = splat4(0);
    if (n < 8) {
        for (int e = 0; e < 4; ++e) {
            const unsigned lo = k + 2 * e < n ? p[k + 2 * e] : 0u, hi = k + 2 * e + 1 < n ? p[k + 2 * e + 1] : 0u;
            v[e] = lo | hi << 16;
        }
        return v;
    }
    const int64_t at = min(k, n - 8);
    v = reinterpret_cast<const Unaligned16*>(p + at)->v;
    const int out = (int)min(k - at, (int64_t)8);      // elements to shift out
    if (out & 8)
        v = splat4(0);
    if (out & 4)
        v = u32x4_t{v[2], v[3], 0u, 0u};
    if (out & 2)
        v = u32x4_t{v[1], v[2], v[3], 0u};
    if (out & 1)
        v = u32x4_t{v[0] >> 16 | v[1] << 16, v[1] >> 16 | v[2] << 16, v[2] >> 16 | v[3] << 16, v[3] >> 16};
    return v;
}

// Four fragments: rows 128 c + 32 t + 8 kq + 0..7 of a vector of n at p.
__device__ __forceinline__ void load_chunk(u32x4_t (&f)[4], const unsigned short* p, int c, int kq, int n)
{
    const int k0 = c * 128;
    if (k0 + 128 <= n) {
#pragma unroll
        for (int t = 0; t < 4; ++t)
            f[t] = reinterpret_cast<const Unaligned16*>(p + k0 + 32 * t + 8 * kq)->v;
    } else {
#pragma unroll
        for (int t = 0; t < 4; ++t)
            f[t] = load8(p, k0 + 32 * t + 8 * kq, n);
    }
}

}  // namespace tg
