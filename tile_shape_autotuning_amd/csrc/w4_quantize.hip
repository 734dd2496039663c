// Quantisation of weights to 4 bits with a scale, and optionally a zero
// point, for every group of rows of a column.
//
//   symmetric:   s = round(max |w| / 7),  z = 8
//   zero point:  lo = min(w, 0), hi = max(w, 0) over the group,
//                s = round((hi - lo) / 15),  z = clamp(rint(-lo / s), 0, 15)
//   code         q = clamp(rint(w / s) + z, 0, 15)
// where round() is to fp32 and then to the scales' type.  The quotients are
// rounded as if exact (ties to even): rint of a float estimate, corrected by
// the sign of the remainder that one FMA gives exactly.
//
// One 256-thread workgroup takes 64 columns (four panels, one a wave) and one
// group of rows, or 128 rows when groups are smaller.  Each chunk of 128 rows
// goes through LDS, so that global reads and writes follow the input's own
// order (either may be contiguous) and a lane then holds the 32 elements of
// its four words.  Lanes l, l + 16, l + 32, l + 48 share a column: a group's
// extremes are a maximum over a lane's own elements and two shuffles.  Groups
// of more than 128 rows are read twice, first for the extremes.
#include <hip/hip_runtime.h>

#include <cmath>
#include <string>

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

// rint(w * inv) made rint(w / s) for finite w and normal s > 0: the remainder
// against the two neighbouring half steps has its exact sign.
__device__ __forceinline__ float rint_quotient(float w, float s, float inv)
{
    float q = rintf(w * inv);
    const float up = fmaf(-(q + 0.5f), s, w), down = fmaf(-(q - 0.5f), s, w);
    const bool odd = ((int)q & 1) != 0;
    if (up > 0.0f || (up == 0.0f && odd))
        q += 1.0f;
    else if (down < 0.0f || (down == 0.0f && odd))
        q -= 1.0f;
    return q;
}

template <bool BF16, bool ROWS>
__global__ void __launch_bounds__(256) w4_quantize_kernel(QuantParams p)
{
    __shared__ float tile[kQRows * (kQCols + 1)];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int n = lane & 15, kq = lane >> 4;
    const int col0 = blockIdx.x * kQCols;
    const int panel = blockIdx.x * (kQCols / 16) + wave;
    const int64_t mat = blockIdx.z;
    const int span = max(p.group, kQRows);             // rows of this workgroup
    const int64_t row_first = (int64_t)blockIdx.y * span;
    const int nch = (int)((min((int64_t)p.K, row_first + span) - row_first + kQRows - 1) / kQRows);
    const int64_t base = mat * (int64_t)p.K * p.N;

    auto load = [&](int64_t r0) {
        __syncthreads();
        for (int i = tid; i < kQRows * kQCols; i += 256) {
            const int r = ROWS ? i / kQCols : i % kQRows, c = ROWS ? i % kQCols : i / kQRows;
            float v = 0.0f;
            if (r0 + r < p.K && col0 + c < p.N) {
                const int64_t at = base + (ROWS ? (r0 + r) * p.N + col0 + c : (int64_t)(col0 + c) * p.K + r0 + r);
                v = BF16 ? __uint_as_float((unsigned)static_cast<const unsigned short*>(p.W)[at] << 16)
                         : static_cast<const float*>(p.W)[at];
            }
            tile[r * (kQCols + 1) + c] = v;
        }
        __syncthreads();
    };
    float v[4][8];
    auto take = [&] {
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[t][e] = tile[(32 * t + 8 * kq + e) * (kQCols + 1) + wave * 16 + n];
    };
    // extremes of this lane's four runs of eight; `bad`: something not finite
    float lo[4] = {0.f, 0.f, 0.f, 0.f}, hi[4] = {0.f, 0.f, 0.f, 0.f};
    int bad[4] = {0, 0, 0, 0};
    auto widen = [&] {
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                lo[t] = fminf(lo[t], v[t][e]);
                hi[t] = fmaxf(hi[t], v[t][e]);
                bad[t] |= !(fabsf(v[t][e]) < INFINITY);
            }
    };
    for (int c = 0; c < nch; ++c) {
        load(row_first + (int64_t)c * kQRows);
        take();
        widen();
    }
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int off = 16; off <= 32; off <<= 1) {
            lo[t] = fminf(lo[t], __shfl_xor(lo[t], off));
            hi[t] = fmaxf(hi[t], __shfl_xor(hi[t], off));
            bad[t] |= __shfl_xor(bad[t], off);
        }
    if (p.group >= 64)
#pragma unroll
        for (int t = 0; t < 4; t += 2) {
            lo[t] = lo[t + 1] = fminf(lo[t], lo[t + 1]);
            hi[t] = hi[t + 1] = fmaxf(hi[t], hi[t + 1]);
            bad[t] = bad[t + 1] = bad[t] | bad[t + 1];
        }
    if (p.group >= 128) {
        const float l = fminf(lo[0], lo[2]), h = fmaxf(hi[0], hi[2]);
        const int b = bad[0] | bad[2];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            lo[t] = l;
            hi[t] = h;
            bad[t] = b;
        }
    }

    // quotients are taken of w * up and s * up: up = 2^64 keeps the remainders
    // of groups near the smallest normal number from vanishing
    float s[4], z[4], inv[4], up[4], su[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        s[t] = p.zero ? (hi[t] - lo[t]) / 15.0f : fmaxf(hi[t], -lo[t]) / 7.0f;
        if (!p.scale_f32)
            s[t] = __uint_as_float((unsigned)f32_to_bf16_rne(s[t]) << 16);
        const bool usable = !bad[t] && s[t] > 0.0f && s[t] < INFINITY;
        up[t] = s[t] < 0x1p-80f ? 0x1p64f : 1.0f;
        su[t] = s[t] * up[t];
        inv[t] = usable ? 1.0f / su[t] : 0.0f;
        z[t] = 8.0f;
        if (p.zero)
            z[t] = usable ? fminf(rint_quotient(-lo[t] * up[t], su[t], inv[t]), 15.0f) : 0.0f;
        if (bad[t])
            s[t] = NAN;
    }
    // scales and zero points: one lane a column and group; columns past N hold zero
    if (kq == 0 && panel < p.panels) {
        const int per = p.group >= 128 ? 4 : p.group / 32;     // runs of 32 rows in a group
        const bool real = panel * 16 + n < p.N;
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
        if (nch > 1) {
            load(r0);
            take();
        }
        u32x4_t w;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            unsigned word = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float q = z[t];
                if (inv[t] != 0.0f)
                    q = fminf(fmaxf(rint_quotient(v[t][e] * up[t], su[t], inv[t]) + z[t], 0.0f), 15.0f);
                const bool real = r0 + 32 * t + 8 * kq + e < p.K && panel * 16 + n < p.N;
                word |= (real ? (unsigned)q : 0u) << (4 * (e >> 1) + 16 * (e & 1));
                v[t][e] = (q - z[t]) * s[t];
            }
            w[t] = word;
        }
        if (panel < p.panels)
            p.words[((mat * p.panels + panel) * p.chunks + r0 / kQRows) * 64 + lane] = w;
        if (p.values) {
            __syncthreads();
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    tile[(32 * t + 8 * kq + e) * (kQCols + 1) + wave * 16 + n] = v[t][e];
            __syncthreads();
            for (int i = tid; i < kQRows * kQCols; i += 256) {
                const int r = ROWS ? i / kQCols : i % kQRows, cc = ROWS ? i % kQCols : i / kQRows;
                if (r0 + r >= p.K || col0 + cc >= p.N)
                    continue;
                const int64_t at = base + (ROWS ? (r0 + r) * p.N + col0 + cc : (int64_t)(col0 + cc) * p.K + r0 + r);
                const float x = tile[r * (kQCols + 1) + cc];
                if (BF16)
                    static_cast<unsigned short*>(p.values)[at] = f32_to_bf16_rne(x);
                else
                    static_cast<float*>(p.values)[at] = x;
            }
        }
    }
}

int check_weight(const tg_weight* w, int64_t K, int64_t N, const char* name)
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
    (void)K;
    (void)N;
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
    const int st = check_weight(&w, K, N, "w4_quantize");
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
    if (dtype == TG_BF16) {
        if (rows_first)
            hipLaunchKernelGGL((w4_quantize_kernel<true, true>), grid, dim3(256), 0, s, p);
        else
            hipLaunchKernelGGL((w4_quantize_kernel<true, false>), grid, dim3(256), 0, s, p);
    } else {
        if (rows_first)
            hipLaunchKernelGGL((w4_quantize_kernel<false, true>), grid, dim3(256), 0, s, p);
        else
            hipLaunchKernelGGL((w4_quantize_kernel<false, false>), grid, dim3(256), 0, s, p);
    }
    return launched("w4_quantize launch");
}
