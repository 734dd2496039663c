// Building blocks of the kernels on 8-bit matrices (gfx950).
//
// An element is code * scale, the code e4m3 (values up to 448, steps of 2^-9
// below 2^-6), the scale fp32 and shared by 128 elements of a row or by a block
// of 128 x 128.  Rows are padded with zero codes to whole blocks, so that no
// kernel has a ragged reduction.
//
// A chunk of 128 k of 16 x 16 results takes lane l's 32 codes of row l % 16 of
// either operand.  Which 32 is free as long as both operands agree; here they are
// the 16-byte pieces l / 16 and l / 16 + 4 of the chunk's eight.  Result:
// D[4 (l / 16) + i][l % 16], i = 0..3.  Two ways to multiply them:
//   exact   codes become bf16 (which holds every e4m3), four
//           v_mfma_f32_16x16x32_bf16: products and sums are fp32;
//   fast    one v_mfma_f32_16x16x128_f8f6f4, a quarter of the instructions and
//           half the time.  It adds eight products at a time (bytes 8 j .. 8 j + 7 of
//           a lane's 32), each cut to a multiple of 2^-13 of the power of two of
//           the largest, then in fp32 (measured on the device; the older
//           v_mfma_f32_16x16x32_fp8_fp8 does the same).  Where the largest cancel,
//           what is left of the others can be lost whole: so only calls that ask
//           for it (TG_FAST_SUMS) get it.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/tilegemm.h"
#include "kernels/common.hpp"

namespace tg {

typedef int i32x8_t __attribute__((ext_vector_type(8)));

__device__ __forceinline__ i32x8_t join8(u32x4_t a, u32x4_t b)
{
    return i32x8_t{(int)a[0], (int)a[1], (int)a[2], (int)a[3], (int)b[0], (int)b[1], (int)b[2], (int)b[3]};
}

__device__ __forceinline__ f32x4_t mfma_fp8(i32x8_t a, i32x8_t b, f32x4_t c)
{
    // scale operands of zero: the form without scales
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, 0, 0, 0, 0);
}

// Sixteen codes as bf16, in order.
__device__ __forceinline__ void expand(u32x4_t c, u32x4_t& lo, u32x4_t& hi)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        u32x4_t& to = i < 2 ? lo : hi;
        to[2 * (i & 1)] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)c[i], 1.0f, false));
        to[2 * (i & 1) + 1] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)c[i], 1.0f, true));
    }
}

// A lane's 32 codes of a chunk as bf16.
struct Expanded {
    u32x4_t v[4];
};

__device__ __forceinline__ Expanded expand(u32x4_t a, u32x4_t b)
{
    Expanded e;
    expand(a, e.v[0], e.v[1]);
    expand(b, e.v[2], e.v[3]);
    return e;
}

__device__ __forceinline__ f32x4_t mfma_exact(const Expanded& a, const Expanded& b)
{
    f32x4_t d = mfma_bf16(a.v[0], b.v[0], f32x4_t{0.f, 0.f, 0.f, 0.f});
#pragma unroll
    for (int i = 1; i < 4; ++i)
        d = mfma_bf16(a.v[i], b.v[i], d);
    return d;
}

// The activation of these products; a NaN stays one (apply_act's ReLU gives 0).
__device__ __forceinline__ float activate(float v, int act)
{
    if (act == TG_ACT_RELU)
        return v <= 0.0f ? 0.0f : v;
    return act == TG_ACT_GELU ? gelu_erf(v) : v;
}

}  // namespace tg
