// Quantisation of weights to 4 bits with a scale, and optionally a zero
// point, for every group of rows of a column.
//
//   symmetric:   s = round(max |w| / 7),  z = 8
//   zero point:  lo = min(w, 0), hi = max(w, 0) over the group, hi - lo
//                rounded to fp32,
//                s = round((hi - lo) / 15),  z = clamp(rint(-lo / s), 0, 15)
//   code         q = clamp(rint(w / s) + z, 0, 15)
// where round() is to fp32 and then to the scales' type.  The quotients are
// rounded as if exact (ties to even): rint of a float estimate, corrected by
// the sign of the remainder that one FMA gives exactly.
//
// A wave takes 16 columns (a panel) and one group of rows, or 128 rows when
// groups are smaller; a workgroup's four waves take neighbouring panels.  A lane
// holds the 32 elements of its four words; lanes l, l + 16, l + 32 and l + 48
// share a column, so a group's extremes are those of a lane's own elements and
// two shuffles.  A matrix stored [N][K] has a lane's eight rows contiguous and
// is read straight into registers, and its values written back the same way; one
// stored [K][N] crosses LDS, which turns rows of 64 columns into columns.  The
// latter's accesses are of whole lines and carry the non-temporal policy; the
// former's are of parts of lines, which the caches join.
// Groups of more than 128 rows are read twice, first for the extremes.
#include <hip/hip_runtime.h>

#include <cmath>
#include <string>
#include <type_traits>

#include "w4.hpp"
#include "w4_host.hpp"

namespace tg {

struct QuantParams {
    const void* W;
    u32x4_t* words;
    void* scales;
    unsigned char* zeros;
    void* values;
    int K, N, group, groups, chunks, panels;
    int scale_f32, zero;
};

static constexpr int kQCols = 64, kQRows = 128;

// rint(w / s) for finite w and normal s > 0, q = rint(w * inv) given: the
// remainder against the two neighbouring half steps has its exact sign.
__device__ __forceinline__ float exact_quotient(float w, float s, float q)
{
    const float up = fmaf(-(q + 0.5f), s, w), down = fmaf(-(q - 0.5f), s, w);
    const bool odd = ((int)q & 1) != 0;
    if (up > 0.0f || (up == 0.0f && odd))
        return q + 1.0f;
    if (down < 0.0f || (down == 0.0f && odd))
        return q - 1.0f;
    return q;
}

// VEC: sixteen bytes at a time along the matrix's contiguous dimension.
template <bool BF16, bool ROWS, bool VEC>
__global__ void __launch_bounds__(256) w4_quantize_kernel(QuantParams p)
{
    // row r of the tile at r * STRIDE bytes: lanes 16 apart, eight rows, fall on other banks
    constexpr int EB = BF16 ? 2 : 4, STRIDE = kQCols * EB + 8;
    __shared__ __align__(16) char tile[ROWS ? kQRows * STRIDE : 16];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int n = lane & 15, kq = lane >> 4;
    const int col0 = blockIdx.x * kQCols;
    const int panel = blockIdx.x * (kQCols / 16) + wave, col = panel * 16 + n;
    const int64_t mat = blockIdx.z;
    const int span = max(p.group, kQRows);             // rows of this workgroup
    const int64_t row_first = (int64_t)blockIdx.y * span;
    const int nch = (int)((min((int64_t)p.K, row_first + span) - row_first + kQRows - 1) / kQRows);
    const char* W = static_cast<const char*>(p.W) + mat * (int64_t)p.K * p.N * EB;
    char* V = static_cast<char*>(p.values) + (p.values ? mat * (int64_t)p.K * p.N * EB : 0);

    auto element = [](const char* at) {
        if constexpr (BF16)
            return __uint_as_float((unsigned)*reinterpret_cast<const unsigned short*>(at) << 16);
        else
            return *reinterpret_cast<const float*>(at);
    };
    auto put = [](char* at, float x) {
        if constexpr (BF16)
            *reinterpret_cast<unsigned short*>(at) = f32_to_bf16_rne(x);
        else
            *reinterpret_cast<float*>(at) = x;
    };
    // pieces of 16 bytes of the tile's rows (ROWS), eight bytes aligned in LDS
    constexpr int PIECES = kQCols * EB / 16;
    auto piece = [&](int i, int& r, int& c) {
        r = i / PIECES;
        c = i % PIECES * (16 / EB);
    };
    typedef unsigned u32x2 __attribute__((ext_vector_type(2)));

    float v[4][8];
    auto load = [&](int64_t r0) {
        if constexpr (ROWS) {
            __syncthreads();
            for (int i = tid; i < kQRows * PIECES; i += 256) {
                int r, c;
                piece(i, r, c);
                char* to = tile + r * STRIDE + c * EB;
                const char* from = W + ((r0 + r) * p.N + col0 + c) * EB;
                u32x4_t x = splat4(0);
                if constexpr (VEC) {
                    if (r0 + r < p.K && col0 + c < p.N)
                        x = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(from));
                } else {
#pragma unroll
                    for (int e = 0; e < 16 / EB; ++e)
                        if (r0 + r < p.K && col0 + c + e < p.N) {
                            if constexpr (BF16)
                                x[e >> 1] |= (unsigned)reinterpret_cast<const unsigned short*>(from)[e]
                                             << (16 * (e & 1));
                            else
                                x[e & 3] = reinterpret_cast<const unsigned*>(from)[e];
                        }
                }
                reinterpret_cast<u32x2*>(to)[0] = u32x2{x[0], x[1]};
                reinterpret_cast<u32x2*>(to)[1] = u32x2{x[2], x[3]};
            }
            __syncthreads();
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    v[t][e] = element(tile + (32 * t + 8 * kq + e) * STRIDE + (wave * 16 + n) * EB);
        } else {
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const int64_t k = r0 + 32 * t + 8 * kq;
                const char* from = W + ((int64_t)col * p.K + k) * EB;
                if constexpr (VEC) {
                    constexpr int X = EB / 2;          // 16-byte loads
                    u32x4_t x[X];
#pragma unroll
                    for (int q = 0; q < X; ++q)
                        x[q] = col < p.N && k + q * 4 < p.K ? reinterpret_cast<const u32x4_t*>(from)[q] : splat4(0);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        if constexpr (BF16)
                            v[t][e] = __uint_as_float(e & 1 ? x[0][e >> 1] & 0xFFFF0000u : x[0][e >> 1] << 16);
                        else
                            v[t][e] = __uint_as_float(x[e >> 2][e & 3]);
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        v[t][e] = col < p.N && k + e < p.K ? element(from + e * EB) : 0.0f;
                }
            }
        }
    };
    // extremes of this lane's four runs of eight; size: of the magnitudes, as
    // bits, which order infinities and NaN last
    float lo[4] = {0.f, 0.f, 0.f, 0.f}, hi[4] = {0.f, 0.f, 0.f, 0.f};
    unsigned size[4] = {0, 0, 0, 0};
    for (int c = 0; c < nch; ++c) {
        load(row_first + (int64_t)c * kQRows);
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                size[t] = max(size[t], __float_as_uint(v[t][e]) & 0x7FFFFFFFu);
                if (p.zero) {
                    lo[t] = fminf(lo[t], v[t][e]);
                    hi[t] = fmaxf(hi[t], v[t][e]);
                }
            }
    }
    auto join = [&](int t, float l, float h, unsigned z) {
        lo[t] = fminf(lo[t], l);
        hi[t] = fmaxf(hi[t], h);
        size[t] = max(size[t], z);
    };
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int off = 16; off <= 32; off <<= 1)
            join(t, __shfl_xor(lo[t], off), __shfl_xor(hi[t], off), (unsigned)__shfl_xor((int)size[t], off));
    if (p.group >= 64)
#pragma unroll
        for (int t = 0; t < 4; t += 2) {
            join(t, lo[t + 1], hi[t + 1], size[t + 1]);
            join(t + 1, lo[t], hi[t], size[t]);
        }
    if (p.group >= 128)
#pragma unroll
        for (int t = 0; t < 4; ++t)
            join(t, lo[t ^ 2], hi[t ^ 2], size[t ^ 2]);

    // quotients are taken of w * up and s * up: up = 2^64 keeps the remainders
    // of groups near the smallest normal number from vanishing
    float s[4], z[4], inv[4], up[4], su[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        const bool bad = size[t] >= 0x7F800000u;
        s[t] = p.zero ? (hi[t] - lo[t]) / 15.0f : __uint_as_float(size[t]) / 7.0f;
        if (!p.scale_f32)
            s[t] = __uint_as_float((unsigned)f32_to_bf16_rne(s[t]) << 16);
        const bool usable = !bad && s[t] > 0.0f && s[t] < INFINITY;
        up[t] = s[t] < 0x1p-80f ? 0x1p64f : 1.0f;
        su[t] = s[t] * up[t];
        inv[t] = usable ? 1.0f / su[t] : 0.0f;
        z[t] = 8.0f;
        if (p.zero)
            z[t] = usable ? fminf(exact_quotient(-lo[t] * up[t], su[t], rintf(-lo[t] * up[t] * inv[t])), 15.0f) : 0.0f;
        // a group that is not finite, or whose range is not: an infinite scale
        // times a code's distance of zero, or of nearly zero in a product's sums
        if (bad || s[t] == INFINITY)
            s[t] = NAN;
    }
    // scales and zero points: one lane a column and group; columns past N hold zero
    if (kq == 0 && panel < p.panels) {
        const int per = p.group >= 128 ? 4 : p.group / 32;     // runs of 32 rows in a group
        const bool real = col < p.N;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const int64_t g = (row_first + 32 * t) / p.group;
            if (t % per != 0 || g >= p.groups)
                continue;
            const int64_t at = ((mat * p.panels + panel) * p.groups + g) * 16 + n;
            if (p.scale_f32)
                static_cast<float*>(p.scales)[at] = real ? s[t] : 0.0f;
            else
                static_cast<unsigned short*>(p.scales)[at] = real ? f32_to_bf16_rne(s[t]) : (unsigned short)0;
            if (p.zero)
                p.zeros[at] = real ? (unsigned char)z[t] : (unsigned char)0;
        }
    }

    for (int c = 0; c < nch; ++c) {
        const int64_t r0 = row_first + (int64_t)c * kQRows;
        if (nch > 1)
            load(r0);
        u32x4_t w;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            float q[8], off = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float x = v[t][e] * up[t] * inv[t];
                q[e] = rintf(x);
                off = fmaxf(off, fabsf(x - q[e]));
            }
            // x is off by less than 2^-18: only a quotient that near to the
            // middle of two codes can have been rounded to the wrong one
            if (off > 0.5f - 0x1p-18f && inv[t] != 0.0f)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    q[e] = exact_quotient(v[t][e] * up[t], su[t], q[e]);
            unsigned word = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float code = fminf(fmaxf(q[e] + z[t], 0.0f), 15.0f);
                if (inv[t] == 0.0f)
                    code = z[t];
                word |= (unsigned)code << (4 * (e >> 1) + 16 * (e & 1));
                v[t][e] = (code - z[t]) * s[t];
            }
            // nothing is stored past K and N
            const int64_t left = p.K - (r0 + 32 * t + 8 * kq);
            if (left < 8 || col >= p.N)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (e >= left || col >= p.N)
                        word &= ~(15u << (4 * (e >> 1) + 16 * (e & 1)));
            w[t] = word;
        }
        if (panel < p.panels)
            __builtin_nontemporal_store(w, p.words + ((mat * p.panels + panel) * p.chunks + r0 / kQRows) * 64 + lane);
        if (!p.values)
            continue;
        if constexpr (ROWS) {
            __syncthreads();
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    put(tile + (32 * t + 8 * kq + e) * STRIDE + (wave * 16 + n) * EB, v[t][e]);
            __syncthreads();
            for (int i = tid; i < kQRows * PIECES; i += 256) {
                int r, cc;
                piece(i, r, cc);
                const char* from = tile + r * STRIDE + cc * EB;
                char* to = V + ((r0 + r) * p.N + col0 + cc) * EB;
                if constexpr (VEC) {
                    const u32x2 a = reinterpret_cast<const u32x2*>(from)[0], b = reinterpret_cast<const u32x2*>(from)[1];
                    if (r0 + r < p.K && col0 + cc < p.N)
                        __builtin_nontemporal_store(u32x4_t{a[0], a[1], b[0], b[1]}, reinterpret_cast<u32x4_t*>(to));
                } else {
#pragma unroll
                    for (int e = 0; e < 16 / EB; ++e)
                        if (r0 + r < p.K && col0 + cc + e < p.N)
                            put(to + e * EB, element(from + e * EB));
                }
            }
        } else {
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const int64_t k = r0 + 32 * t + 8 * kq;
                char* to = V + ((int64_t)col * p.K + k) * EB;
                if constexpr (VEC) {
                    constexpr int X = EB / 2;
                    u32x4_t x[X];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        if constexpr (BF16) {
                            const unsigned h = f32_to_bf16_rne(v[t][e]);
                            x[0][e >> 1] = e & 1 ? x[0][e >> 1] | h << 16 : h;
                        } else {
                            x[e >> 2][e & 3] = __float_as_uint(v[t][e]);
                        }
                    }
#pragma unroll
                    for (int q = 0; q < X; ++q)
                        if (col < p.N && k + q * 4 < p.K)
                            reinterpret_cast<u32x4_t*>(to)[q] = x[q];
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (col < p.N && k + e < p.K)
                            put(to + e * EB, v[t][e]);
                }
            }
        }
    }
}

int check_weight(const tg_weight* w, const char* name)
{
    const std::string s(name);
    if (!w || !w->data)
        return set_error(TG_E_INVAL, s + ": NULL weight");
    if ((uintptr_t)w->data & 15u)
        return set_error(TG_E_INVAL, s + ": weights must be 16-byte aligned");
    if (w->format == TG_W_BF16)
        return TG_OK;
    if (w->format != TG_W_W4)
        return set_error(TG_E_INVAL, s + ": unknown weight format");
    if (!w->scales || ((uintptr_t)w->scales & 3u))
        return set_error(TG_E_INVAL, s + ": scales must be given, 4-byte aligned");
    if (w->scale_dtype != TG_F32 && w->scale_dtype != TG_BF16)
        return set_error(TG_E_INVAL, s + ": scales are fp32 or bf16");
    if (w->group != 32 && w->group != 64 && (w->group < 128 || w->group % 128 != 0))
        return set_error(TG_E_INVAL, s + ": group must be 32, 64 or a multiple of 128");
    return TG_OK;
}

}  // namespace tg

using namespace tg;

extern "C" int tg_w4_quantize(int64_t count, int64_t K, int64_t N, int group, const void* W, int dtype, int rows_first,
                              int scale_dtype, void* words, void* scales, void* zeros, void* values)
{
    if (count < 0 || K < 1 || N < 1)
        return set_error(TG_E_INVAL, "count must be >= 0, K and N >= 1");
    if (dtype != TG_F32 && dtype != TG_BF16)
        return set_error(TG_E_INVAL, "weights are fp32 or bf16");
    tg_weight w{};
    w.format = TG_W_W4;
    w.group = group;
    w.scale_dtype = scale_dtype;
    w.data = words;
    w.scales = scales;
    if (count == 0)
        w.data = w.scales = reinterpret_cast<void*>(16);   // nothing is read or written
    const int st = check_weight(&w, "w4_quantize");
    if (st != TG_OK)
        return st;
    const int64_t span = group > kQRows ? group : kQRows;
    if (K > (1 << 21) || N > (1 << 21) || count > 65535 || ceil_div(K, span) > 65535)
        return set_error(TG_E_UNSUPPORTED, "K and N are at most 2^21, count at most 65535");
    if (count == 0)
        return TG_OK;
    if (!W || ((uintptr_t)W % (dtype == TG_F32 ? 4 : 2)) || ((uintptr_t)values % (dtype == TG_F32 ? 4 : 2)))
        return set_error(TG_E_INVAL, "W and values must be aligned to their elements, W not NULL");
    if (!have_device())
        return set_error(TG_E_UNSUPPORTED, "no HIP device");
    QuantParams p{};
    p.W = W;
    p.words = static_cast<u32x4_t*>(words);
    p.scales = scales;
    p.zeros = static_cast<unsigned char*>(zeros);
    p.values = values;
    p.K = (int)K;
    p.N = (int)N;
    p.group = group;
    p.groups = (int)ceil_div(K, group);
    p.chunks = (int)ceil_div(K, 128);
    p.panels = (int)ceil_div(N, 16);
    p.scale_f32 = scale_dtype == TG_F32;
    p.zero = zeros != nullptr;
    const dim3 grid((unsigned)ceil_div(N, kQCols), (unsigned)ceil_div(K, span), (unsigned)count);
    hipStream_t s = current_stream();
    const int64_t run = rows_first ? N : K;            // contiguous elements
    const bool vec = run % (dtype == TG_BF16 ? 8 : 4) == 0 && (((uintptr_t)W | (uintptr_t)values) & 15u) == 0;
    auto go = [&](auto bf16, auto rows) {
        constexpr bool B = decltype(bf16)::value, R = decltype(rows)::value;
        if (vec)
            hipLaunchKernelGGL((w4_quantize_kernel<B, R, true>), grid, dim3(256), 0, s, p);
        else
            hipLaunchKernelGGL((w4_quantize_kernel<B, R, false>), grid, dim3(256), 0, s, p);
    };
    auto pick = [&](auto bf16) { rows_first ? go(bf16, std::true_type{}) : go(bf16, std::false_type{}); };
    dtype == TG_BF16 ? pick(std::true_type{}) : pick(std::false_type{});
    return launched("w4_quantize launch");
}
