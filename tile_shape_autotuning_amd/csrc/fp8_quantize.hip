// Quantisation to e4m3 with a scale for each 128 elements of a row, or for
// each block of 128 x 128.
//
//   s = fp32(max |x| / 448) over the block,  code = e4m3(x / s), nearest, ties to
//   even, at most 448; 0 where s is 0.  The quotient is rounded as if exact: an
//   estimate x * (1 / s) is off by at most 2^-23 of its value, so where both ends
//   of the estimate +- 2^-22 have the same code it is the quotient's; elsewhere
//   (one element in about 2^17) the two codes are neighbours, and the sign of
//   |x| - t s, t the middle of their values, decides: one FMA gives it exactly (t s
//   has 29 bits at most).  Scales below 2^-100 are taken times 2^100, with x.
//
// Bound by memory: x is read once, into registers, 16 bytes a lane and load at
// any alignment.  Sixteen lanes have 128 elements of a row.  The transpose's
// codes, four neighbouring k a thread, cross LDS and leave in whole lines.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <string>

#include "fp8.hpp"
#include "fp8_host.hpp"
#include "row_piece.hpp"

namespace tg {

struct F8QuantParams {
    const void* x;
    unsigned char* codes;
    float* scales;
    void* values;
    int64_t rows;                                      // of all matrices
    int64_t R, K;
    int64_t works;                                     // workgroups' shares
    int chunks;
};

constexpr unsigned kInfBits = 0x7F800000u, kNanBits = 0x7FC00000u;
typedef unsigned u32x2_t8 __attribute__((ext_vector_type(2)));

// Eight neighbouring elements; those from `n` on are not written.
template <bool BF16>
__device__ __forceinline__ void store8(void* base, int64_t at, int n, const float (&v)[8])
{
    if (n >= 8) {
        if constexpr (BF16) {
            u32x4_t w;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w[i] = f32_to_bf16_rne(v[2 * i]) | (unsigned)f32_to_bf16_rne(v[2 * i + 1]) << 16;
            *reinterpret_cast<u32x4_any*>(static_cast<unsigned short*>(base) + at) = w;
        } else {
            u32x4_any* to = reinterpret_cast<u32x4_any*>(static_cast<float*>(base) + at);
            to[0] = u32x4_t{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
            to[1] = u32x4_t{__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7])};
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) {
                if constexpr (BF16)
                    static_cast<unsigned short*>(base)[at + i] = f32_to_bf16_rne(v[i]);
                else
                    static_cast<float*>(base)[at + i] = v[i];
            }
    }
}

// The largest |x| as bits: infinities and NaN are above every number.
__device__ __forceinline__ unsigned top_of(const float (&v)[8])
{
    unsigned top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        top = max(top, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    return top;
}

template <int CTRL>
__device__ __forceinline__ unsigned max_with(unsigned v)
{
    return max(v, (unsigned)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, false));
}

// Over each row of 16 lanes (rotations by 8, 4, 2, 1).
__device__ __forceinline__ unsigned max16(unsigned v)
{
    return max_with<0x121>(max_with<0x122>(max_with<0x124>(max_with<0x128>(v))));
}

// Lane U's of each four lanes.
template <int U>
__device__ __forceinline__ float quad(float v)
{
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), U * 0x55, 0xf, 0xf, false));
}

struct Scale {
    float s;                                           // as stored
    float t, inv, by;                                  // that x * by is divided by, its reciprocal
    __device__ __forceinline__ explicit Scale(unsigned top)
    {
        s = top >= kInfBits ? __uint_as_float(kNanBits) : __uint_as_float(top) / 448.0f;
        by = s < 0x1p-100f ? 0x1p100f : 1.0f;
        t = s * by;
        inv = t > 0.0f ? 1.0f / t : 0.0f;
    }
    __device__ __forceinline__ Scale() {}
    // one that another thread has worked out
    __device__ __forceinline__ Scale(float s_, float inv_) : s(s_), inv(inv_)
    {
        by = s < 0x1p-100f ? 0x1p100f : 1.0f;
        t = s * by;
    }
};

// Codes of four elements whose estimates' ends differ somewhere (lo, hi).
__device__ __forceinline__ unsigned resolve4(const float* x, const Scale& s, unsigned lo, unsigned hi)
{
    unsigned c = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const unsigned a = lo >> (8 * i) & 0x7Fu, b = hi >> (8 * i) & 0x7Fu;
        const float va = __builtin_amdgcn_cvt_f32_fp8((int)a, 0), vb = __builtin_amdgcn_cvt_f32_fp8((int)b, 0);
        const float d = fmaf(-0.5f * (va + vb), s.t, fabsf(x[i] * s.by));
        const unsigned code = d > 0.0f || (d == 0.0f && (b & 1) == 0) ? b : a;
        c |= (code | (lo >> (8 * i) & 0x80u)) << (8 * i);
    }
    return c;
}

__device__ __forceinline__ unsigned encode4(const float* x, const Scale& s)
{
    float lo[4], hi[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        // above 448 only where a subnormal scale was rounded down
        float q = x[i] * s.inv;
        if (s.by != 1.0f)
            q = __builtin_amdgcn_fmed3f((x[i] * s.by) * s.inv, -448.0f, 448.0f);
        lo[i] = q * (1.0f - 0x1p-22f);
        hi[i] = q * (1.0f + 0x1p-22f);
    }
    const int a = __builtin_amdgcn_cvt_pk_fp8_f32(lo[2], lo[3], __builtin_amdgcn_cvt_pk_fp8_f32(lo[0], lo[1], 0, false), true);
    const int b = __builtin_amdgcn_cvt_pk_fp8_f32(hi[2], hi[3], __builtin_amdgcn_cvt_pk_fp8_f32(hi[0], hi[1], 0, false), true);
    unsigned out = (unsigned)a;
    if (a != b)
        out = resolve4(x, s, (unsigned)a, (unsigned)b);
    if (!(s.s > 0.0f))
        out = s.s == 0.0f ? 0u : 0x7F7F7F7Fu;
    return out;
}

__device__ __forceinline__ u32x2_t8 encode8(const float (&v)[8], const Scale& s)
{
    return u32x2_t8{encode4(v, s), encode4(v + 4, s)};
}

// Codes from element n on are zero.
__device__ __forceinline__ u32x2_t8 first_of(u32x2_t8 c, int n)
{
    if (n < 8) {
        c[1] = n <= 4 ? 0u : c[1] & ((1u << (8 * (n - 4))) - 1);
        c[0] = n <= 0 ? 0u : n < 4 ? c[0] & ((1u << (8 * n)) - 1) : c[0];
    }
    return c;
}

__device__ __forceinline__ void decode4(unsigned c, const Scale& s, float* v)
{
    v[0] = __builtin_amdgcn_cvt_f32_fp8((int)c, 0) * s.s;
    v[1] = __builtin_amdgcn_cvt_f32_fp8((int)c, 1) * s.s;
    v[2] = __builtin_amdgcn_cvt_f32_fp8((int)c, 2) * s.s;
    v[3] = __builtin_amdgcn_cvt_f32_fp8((int)c, 3) * s.s;
}

// x [R][K].  Sixteen lanes take a chunk of a row.  BLOCK = 1: U of them, each on
// its own; 128: U = 8, a workgroup's 16 rows eight times over make its block.
template <bool BF16, int BLOCK, int U>
__global__ void __launch_bounds__(256) fp8_quantize_along_kernel(F8QuantParams p)
{
    __shared__ unsigned tops[4];
    const int l16 = threadIdx.x & 15, team = threadIdx.x >> 4, wave = threadIdx.x >> 6;
    const int64_t Kp = (int64_t)p.chunks * 128;
    for (int64_t work = blockIdx.x; work < p.works; work += gridDim.x) {
        int64_t row[U], from[U], block = 0;            // rows past the last read the last
        int chunk[U];
        if constexpr (BLOCK == 1) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const unsigned g = (unsigned)(work * U + u) * 16 + team;
                row[u] = g / (unsigned)p.chunks;
                chunk[u] = (int)(g - (unsigned)row[u] * (unsigned)p.chunks);
                from[u] = min(row[u], p.rows - 1);
            }
        } else {
            const int64_t blocks = (p.R + 127) / 128, rb = work / p.chunks, mat = rb / blocks;
            block = work;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t r = (rb - mat * blocks) * 128 + u * 16 + team;
                row[u] = r < p.R ? mat * p.R + r : p.rows;
                from[u] = mat * p.R + min(r, p.R - 1);
                chunk[u] = (int)(work - rb * p.chunks);
            }
        }
        Piece<BF16, 8> x[U];
        if (p.K >= 8) {
#pragma unroll
            for (int u = 0; u < U; ++u)
                x[u].load(static_cast<const char*>(p.x) + from[u] * p.K * (BF16 ? 2 : 4), chunk[u] * 128 + 8 * l16, p.K);
        } else {
#pragma unroll
            for (int u = 0; u < U; ++u)
                x[u].load_short(static_cast<const char*>(p.x) + from[u] * p.K * (BF16 ? 2 : 4), 8 * l16, p.K);
        }
        float v[U][8];
        unsigned top[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            x[u].arrived();
            x[u].end(chunk[u] * 128 + 8 * l16, p.K);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[u][i] = x[u][i];
            top[u] = top_of(v[u]);
        }
        if constexpr (BLOCK == 128) {
#pragma unroll
            for (int u = 1; u < U; ++u)
                top[0] = max(top[0], top[u]);
            unsigned t = max16(top[0]);
            t = max(t, (unsigned)__shfl_xor((int)t, 16));
            t = max(t, (unsigned)__shfl_xor((int)t, 32));
            __syncthreads();
            if ((threadIdx.x & 63) == 0)
                tops[wave] = t;
            __syncthreads();
            top[0] = max(max(tops[0], tops[1]), max(tops[2], tops[3]));
        } else {
#pragma unroll
            for (int u = 0; u < U; ++u)
                top[u] = max16(top[u]);
        }
        Scale scale[U == 4 ? 4 : 1];
        if constexpr (U == 4) {
            // all lanes have all four: each works out one (4096 x 8192 bf16 25.8 us, all four 26.7)
            const int l4 = l16 & 3;
            const Scale mine(l4 == 0 ? top[0] : l4 == 1 ? top[1] : l4 == 2 ? top[2] : top[3]);
            scale[0] = Scale(quad<0>(mine.s), quad<0>(mine.inv));
            scale[1] = Scale(quad<1>(mine.s), quad<1>(mine.inv));
            scale[2] = Scale(quad<2>(mine.s), quad<2>(mine.inv));
            scale[3] = Scale(quad<3>(mine.s), quad<3>(mine.inv));
        } else {
            scale[0] = Scale(top[0]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const Scale s = scale[U == 4 ? u : 0];
            const int64_t k = chunk[u] * 128 + 8 * l16;
            const int n = (int)min((int64_t)8, p.K - k);
            if (row[u] < p.rows) {
                const u32x2_t8 c = first_of(encode8(v[u], s), n);
                *reinterpret_cast<u32x2_t8*>(p.codes + row[u] * Kp + k) = c;
                if (p.values) {
                    decode4(c[0], s, v[u]);
                    decode4(c[1], s, v[u] + 4);
                    store8<BF16>(p.values, row[u] * p.K + k, n, v[u]);
                }
                if (BLOCK == 1 && l16 == 0)
                    p.scales[row[u] * p.chunks + chunk[u]] = s.s;
            }
            if (BLOCK == 128 && u == 0 && threadIdx.x == 0)
                p.scales[block] = s.s;
        }
    }
}

// x [K][R]: a workgroup takes 128 k of ROWS rows, a thread eight neighbouring rows
// of four neighbouring k.  64 rows where they need no common scale: more, smaller
// workgroups a compute unit load, compute and store beside each other; one thread a
// row works out its scale for the others (4096 x 8192 bf16 with values 36 us, 4.6
// TB/s; every thread for itself 41, and 128 rows that way 55).  Workgroups
// numbered along k instead of the rows took 1.4 times as long.  bf16 loads do not
// stay in the caches: 37 us for x that is in none, 42 with the usual policy, and 37
// against 36 for x that was read just before; fp32 loads do (8192 x 28672 with values
// 431 us, else 482).
template <bool BF16, int BLOCK>
struct Across {
    static constexpr int ROWS = BLOCK == 1 ? 64 : 128;
    static constexpr int LANES = ROWS / 8;             // side by side along the rows
    static constexpr int THREADS = LANES * 32, WAVES = THREADS / 64;
};

template <bool BF16, int BLOCK>
__global__ void __launch_bounds__((Across<BF16, BLOCK>::THREADS), 4) fp8_quantize_across_kernel(F8QuantParams p)
{
    using Cf = Across<BF16, BLOCK>;
    constexpr int ROWS = Cf::ROWS, LANES = Cf::LANES, PITCH = 33;   // dwords of a row of codes: other banks for the next
    __shared__ unsigned out[ROWS * PITCH];
    __shared__ unsigned tops[BLOCK == 1 ? Cf::WAVES * ROWS : Cf::WAVES];
    __shared__ float scales[BLOCK == 1 ? 2 * ROWS : 1];             // and the reciprocals
    const int rl = threadIdx.x % LANES, team = threadIdx.x / LANES, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t Kp = (int64_t)p.chunks * 128, groups = (p.R + ROWS - 1) / ROWS;
    for (int64_t work = blockIdx.x; work < p.works; work += gridDim.x) {
        // neighbouring workgroups have neighbouring rows of the same k
        const int64_t mat = work / (groups * p.chunks), in = work - mat * groups * p.chunks;
        const int64_t chunk = in / groups, rb = in - chunk * groups;
        const int64_t r0 = rb * ROWS + 8 * rl, k0 = chunk * 128 + 4 * team, base = mat * p.R * p.K;
        const int n = (int)max((int64_t)0, min((int64_t)8, p.R - r0));
        const int left = (int)max((int64_t)0, min((int64_t)4, p.K - k0));
        // k past K read the last k: it is of this chunk
        Piece<BF16, 8> in4[4];
        auto from = [&](int q) {
            return static_cast<const char*>(p.x) + (base + min(k0 + q, p.K - 1) * p.R) * (BF16 ? 2 : 4);
        };
        if (p.R >= 8) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
                in4[q].template load<BF16>(from(q), r0, p.R);
        } else {
#pragma unroll
            for (int q = 0; q < 4; ++q)
                in4[q].load_short(from(q), r0, p.R);
        }
        float v[4][8];                                 // [k][row]
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            in4[q].arrived();
            in4[q].end(r0, p.R);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[q][e] = in4[q][e];
        }
        unsigned top[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            top[e] = 0;
#pragma unroll
            for (int q = 0; q < 4; ++q)
                top[e] = max(top[e], __float_as_uint(v[q][e]) & 0x7FFFFFFFu);
#pragma unroll
            for (int off = LANES; off < 64; off <<= 1)
                top[e] = max(top[e], (unsigned)__shfl_xor((int)top[e], off));
        }
        __syncthreads();                               // the last work's codes and tops are read
        if constexpr (BLOCK == 1) {
            if (lane < LANES)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    tops[wave * ROWS + 8 * rl + e] = top[e];
            __syncthreads();
            if (threadIdx.x < ROWS) {
                unsigned t = 0;
#pragma unroll
                for (int w = 0; w < Cf::WAVES; ++w)
                    t = max(t, tops[w * ROWS + threadIdx.x]);
                const Scale s(t);
                scales[threadIdx.x] = s.s;
                scales[ROWS + threadIdx.x] = s.inv;
                if (rb * ROWS + (int)threadIdx.x < p.R)
                    p.scales[(mat * p.R + rb * ROWS + threadIdx.x) * p.chunks + chunk] = s.s;
            }
            __syncthreads();
        } else {
            unsigned t = top[0];
#pragma unroll
            for (int e = 1; e < 8; ++e)
                t = max(t, top[e]);
            t = max16(t);
            if (lane == 0)
                tops[wave] = t;
            __syncthreads();
#pragma unroll
            for (int w = 0; w < Cf::WAVES; ++w)
                t = max(t, tops[w]);
            top[0] = t;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const Scale s = BLOCK == 1 ? Scale(scales[8 * rl + e], scales[ROWS + 8 * rl + e]) : Scale(top[0]);
            float x[4];
#pragma unroll
            for (int q = 0; q < 4; ++q)
                x[q] = v[q][e];
            unsigned c = encode4(x, s);
            c = left <= 0 ? 0u : left < 4 ? c & ((1u << (8 * left)) - 1) : c;      // k past K
            out[(8 * rl + e) * PITCH + team] = c;
            if (p.values) {
                decode4(c, s, x);
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    v[q][e] = x[q];
            }
            if (BLOCK == 128 && e == 0 && threadIdx.x == 0)
                p.scales[(mat * groups + rb) * p.chunks + chunk] = s.s;
        }
        if (p.values) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
                store8<BF16>(p.values, base + (k0 + q) * p.R + r0, q < left ? n : 0, v[q]);
        }
        __syncthreads();
        // eight threads a row, sixteen codes each
#pragma unroll
        for (int q = 0; q < ROWS * 8 / Cf::THREADS; ++q) {
            const int r = q * (Cf::THREADS / 8) + (threadIdx.x >> 3), at = r * PITCH + 4 * (threadIdx.x & 7);
            if (rb * ROWS + r < p.R)
                *reinterpret_cast<u32x4_t*>(p.codes + (mat * p.R + rb * ROWS + r) * Kp + chunk * 128 +
                                            16 * (threadIdx.x & 7)) = u32x4_t{out[at], out[at + 1], out[at + 2], out[at + 3]};
        }
    }
}

// Chunks of rows from which a lane takes four at a time (fewer fill the compute
// units only one by one).
constexpr int64_t kManyChunks = (int64_t)1 << 16;

template <bool BF16>
static int launch_quantize(F8QuantParams p, int64_t count, int block, bool along, hipStream_t s)
{
    const int64_t blocks = count * ceil_div(p.R, 128) * p.chunks, chunks = p.rows * p.chunks;
    if (block == 1 && along && chunks > 0xFFFFFF00ll)
        return set_error(TG_E_UNSUPPORTED, "fp8_quantize: more than 2^32 chunks of 128 elements");
    auto grid = [&](int64_t works) {
        p.works = works;
        return dim3((unsigned)std::min<int64_t>(works, 1 << 22));
    };
    if (!along && block == 1)
        hipLaunchKernelGGL((fp8_quantize_across_kernel<BF16, 1>), grid(count * ceil_div(p.R, 64) * p.chunks),
                           dim3((unsigned)Across<BF16, 1>::THREADS), 0, s, p);
    else if (!along)
        hipLaunchKernelGGL((fp8_quantize_across_kernel<BF16, 128>), grid(blocks), dim3((unsigned)Across<BF16, 128>::THREADS), 0, s,
                           p);
    else if (block == 128)
        hipLaunchKernelGGL((fp8_quantize_along_kernel<BF16, 128, 8>), grid(blocks), dim3(256), 0, s, p);
    else if (chunks < kManyChunks)
        hipLaunchKernelGGL((fp8_quantize_along_kernel<BF16, 1, 1>), grid(ceil_div(chunks, 16)), dim3(256), 0, s, p);
    else
        hipLaunchKernelGGL((fp8_quantize_along_kernel<BF16, 1, 4>), grid(ceil_div(chunks, 64)), dim3(256), 0, s, p);
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
    p.rows = count * R;
    p.R = R;
    p.K = K;
    p.chunks = (int)ceil_div(K, 128);
    return dtype == TG_BF16 ? launch_quantize<true>(p, count, block, rows_first != 0, current_stream())
                            : launch_quantize<false>(p, count, block, rows_first != 0, current_stream());
}

}  // extern "C"
