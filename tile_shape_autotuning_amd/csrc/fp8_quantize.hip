// Quantisation to e4m3 with a scale for each 128 elements of a row, or for
// each block of 128 x 128.
//
//   s = fp32(max |x| / 448) over the block,  code = e4m3(x / s), nearest, ties to
//   even, at most 448; 0 where s is 0.  The quotient is rounded as if exact: an
//   estimate x * (1 / s) is off by at most 2^-23 of its value, so where both ends
//   of the estimate +- 2^-22 have the same code it is the quotient's; elsewhere
//   (one element in about 2^17) the quotient is taken in fp64, which cannot fall
//   on the middle of two codes unless the exact one does (x and the middle times
//   s have 24 and 29 bits).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <string>

#include "fp8.hpp"
#include "fp8_host.hpp"

namespace tg {

struct F8QuantParams {
    const void* x;
    unsigned char* codes;
    float* scales;
    void* values;
    int64_t R, K;
    int64_t rs, ks;                                    // elements from one row, one column to the next
    int chunks;
};

constexpr unsigned kInfBits = 0x7F800000u;

template <bool BF16>
__device__ __forceinline__ float load_element(const void* p, int64_t i)
{
    if constexpr (BF16)
        return __uint_as_float((unsigned)static_cast<const unsigned short*>(p)[i] << 16);
    else
        return static_cast<const float*>(p)[i];
}

template <bool BF16>
__device__ __forceinline__ void store_element(void* p, int64_t i, float v)
{
    if constexpr (BF16)
        static_cast<unsigned short*>(p)[i] = f32_to_bf16_rne(v);
    else
        static_cast<float*>(p)[i] = v;
}

// A block's scale from the largest |x|, as bits: infinities and NaN are above
// every number.
__device__ __forceinline__ float scale_of(unsigned top)
{
    return top >= kInfBits ? __uint_as_float(0x7FC00000u) : __uint_as_float(top) / 448.0f;
}

// The value of the code nearest to x / s.
__device__ float nearest_exact(float x, float s)
{
    const double q = (double)x / (double)s, a = fabs(q);
    const int e = max(ilogb(a), -6) - 3;
    const float r = (float)fmin(ldexp(rint(ldexp(a, -e)), e), 448.0);
    return copysignf(a == 0.0 ? 0.0f : r, x);
}

// Code of x with scale s, inv = 1 / s.
__device__ __forceinline__ unsigned code_of(float x, float s, float inv)
{
    if (!(s > 0.0f))
        return s == 0.0f ? 0u : 0x7Fu;
    const float q = x * inv;
    const float lo = __builtin_amdgcn_fmed3f(q * (1.0f - 0x1p-22f), -448.0f, 448.0f);
    const float hi = __builtin_amdgcn_fmed3f(q * (1.0f + 0x1p-22f), -448.0f, 448.0f);
    unsigned c = (unsigned)__builtin_amdgcn_cvt_pk_fp8_f32(lo, hi, 0, false) & 0xFFFFu;
    // below 2^-100 the reciprocal may overflow, and the quotient is no longer accurate
    if ((c & 0xFFu) != c >> 8 || s < 0x1p-100f)
        c = (unsigned)__builtin_amdgcn_cvt_pk_fp8_f32(nearest_exact(x, s), 0.0f, 0, false);
    return c & 0xFFu;
}

__device__ __forceinline__ float value_of(unsigned code, float s)
{
    return __builtin_amdgcn_cvt_f32_fp8((int)code, 0) * s;
}

__device__ __forceinline__ unsigned wave_max_bits(unsigned v)
{
#pragma unroll
    for (int off = 1; off < 64; off <<= 1)
        v = max(v, (unsigned)__shfl_xor((int)v, off));
    return v;
}

// A workgroup of 256 takes BLOCK rows of one chunk of 128 columns: a wave each
// for BLOCK = 1, all of them together for 128.
template <bool BF16, int BLOCK>
__global__ void __launch_bounds__(256) fp8_quantize_kernel(F8QuantParams p)
{
    __shared__ unsigned tops[4];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t mat = blockIdx.z;
    const int64_t group = BLOCK == 1 ? (int64_t)blockIdx.x * 4 + wave : blockIdx.x;
    const int64_t row0 = group * BLOCK, row1 = min(p.R, row0 + BLOCK);
    const int64_t Kp = (int64_t)p.chunks * 128;
    const int64_t base = mat * p.R * p.K;
    const int first = BLOCK == 1 ? 0 : wave, step = BLOCK == 1 ? 1 : 4;
    for (int chunk = blockIdx.y; chunk < p.chunks; chunk += gridDim.y) {
    unsigned top = 0;
    for (int64_t r = row0 + first; r < row1; r += step)
        for (int i = 0; i < 2; ++i) {
            const int64_t k = chunk * 128 + 64 * i + lane;
            if (k < p.K)
                top = max(top, __float_as_uint(load_element<BF16>(p.x, base + r * p.rs + k * p.ks)) & 0x7FFFFFFFu);
        }
    top = wave_max_bits(top);
    if constexpr (BLOCK == 128) {
        if (lane == 0)
            tops[wave] = top;
        __syncthreads();
        top = max(max(tops[0], tops[1]), max(tops[2], tops[3]));
    }
    const float s = scale_of(top), inv = 1.0f / s;
    for (int64_t r = row0 + first; r < row1; r += step)
        for (int i = 0; i < 2; ++i) {
            const int64_t k = chunk * 128 + 64 * i + lane;
            unsigned c = 0;
            if (k < p.K) {
                const int64_t at = base + r * p.rs + k * p.ks;
                c = code_of(load_element<BF16>(p.x, at), s, inv);
                if (p.values)
                    store_element<BF16>(p.values, at, value_of(c, s));
            }
            p.codes[(mat * p.R + r) * Kp + k] = (unsigned char)c;
        }
    const int64_t groups = (p.R + BLOCK - 1) / BLOCK;
    if (row0 < p.R && lane == 0 && (BLOCK == 1 || wave == 0))
        p.scales[(mat * groups + group) * p.chunks + chunk] = s;
    __syncthreads();
    }
}

template <bool BF16>
static int launch_quantize(const F8QuantParams& p, int64_t count, int block, hipStream_t s)
{
    const dim3 grid((unsigned)ceil_div(p.R, block == 1 ? 4 : 128), (unsigned)std::min(p.chunks, 65535),
                    (unsigned)count);
    if (block == 1)
        hipLaunchKernelGGL((fp8_quantize_kernel<BF16, 1>), grid, dim3(256), 0, s, p);
    else
        hipLaunchKernelGGL((fp8_quantize_kernel<BF16, 128>), grid, dim3(256), 0, s, p);
    return launched("fp8_quantize launch");
}

}  // namespace tg

using namespace tg;

extern "C" {

int tg_fp8_quantize(int64_t count, int64_t R, int64_t K, int block, const void* x, int dtype, int rows_first,
                    void* codes, float* scales, void* values)
{
    if (count < 0 || R < 0 || K < 1)
        return set_error(TG_E_INVAL, "count and R must be >= 0, K >= 1");
    if (block != 1 && block != 128)
        return set_error(TG_E_INVAL, "block must be 1 or 128");
    if (dtype != TG_F32 && dtype != TG_BF16)
        return set_error(TG_E_INVAL, "x is fp32 or bf16");
    if (R > kMaxSide || K > kMaxSide || count > 65535 || R * K >= (int64_t)1 << 40)
        return set_error(TG_E_UNSUPPORTED, "R and K are at most 2^24, count 65535, a matrix below 2^40 elements");
    if (count == 0 || R == 0)
        return TG_OK;
    const uintptr_t mask = dtype == TG_F32 ? 3u : 1u;
    if (!x || !codes || !scales || (((uintptr_t)x | (uintptr_t)values) & mask) || ((uintptr_t)codes & 15u) ||
        ((uintptr_t)scales & 3u))
        return set_error(TG_E_INVAL, "x, codes and scales must be given; elements aligned, codes 16-byte aligned");
    if (!have_device())
        return set_error(TG_E_UNSUPPORTED, "no HIP device");
    F8QuantParams p{};
    p.x = x;
    p.codes = static_cast<unsigned char*>(codes);
    p.scales = scales;
    p.values = values;
    p.R = R;
    p.K = K;
    p.rs = rows_first ? K : 1;
    p.ks = rows_first ? 1 : R;
    p.chunks = (int)ceil_div(K, 128);
    return dtype == TG_BF16 ? launch_quantize<true>(p, count, block, current_stream())
                            : launch_quantize<false>(p, count, block, current_stream());
}

}  // extern "C"
