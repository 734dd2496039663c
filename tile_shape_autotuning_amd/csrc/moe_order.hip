// Tokens in the order of their experts, and back: the sort of (token, choice)
// pairs, the copy of rows into that order, the weighted sum that brings them
// back, and its gradients.  Everything here is bound by memory, but for the
// sort's latency.  No atomics: the same call gives the same bits.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <string>

#include "kernels/common.hpp"
#include "w4_host.hpp"

namespace tg {

constexpr int kOrderExperts = 1024, kOrderChoices = 16;
constexpr int64_t kOrderTokens = (int64_t)1 << 24, kOrderWidth = (int64_t)1 << 24;

// ---------------------------------------------------------------- sort
// A workgroup takes one expert: it counts the pairs of the experts before it,
// then walks the pairs in order and numbers its own.  The last workgroup takes
// the pairs without an expert, and the rows behind the last one.
__global__ void __launch_bounds__(256) moe_sort_kernel(const int32_t* ids, int64_t n, int E, int32_t* position,
                                                       int32_t* source, int32_t* offsets)
{
    __shared__ int part[4];
    const int e = blockIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    auto total = [&](int v) {                          // over the workgroup
#pragma unroll
        for (int off = 1; off < 64; off <<= 1)
            v += __shfl_xor(v, off);
        __syncthreads();
        if (lane == 0)
            part[wave] = v;
        __syncthreads();
        return part[0] + part[1] + part[2] + part[3];
    };
    int before = 0;
    for (int64_t i = threadIdx.x; i < n; i += 256)
        before += ids[i] >= 0 && ids[i] < e;
    int at = total(before);
    if (threadIdx.x == 0)
        offsets[e] = at;
    if (e == E) {
        for (int64_t i = threadIdx.x; i < n; i += 256) {
            if (ids[i] < 0 || ids[i] >= E)
                position[i] = -1;
            if (i >= at)
                source[i] = -1;
        }
        return;
    }
    for (int64_t i0 = 0; i0 < n; i0 += 256) {
        const int64_t i = i0 + threadIdx.x;
        const bool mine = i < n && ids[i] == e;
        const unsigned long long has = __ballot(mine);
        __syncthreads();
        if (lane == 0)
            part[wave] = __popcll(has);
        __syncthreads();
        int to = at + __popcll(has & ((1ull << lane) - 1));
        for (int w = 0; w < wave; ++w)
            to += part[w];
        if (mine) {
            position[i] = to;
            source[to] = (int32_t)i;
        }
        at += part[0] + part[1] + part[2] + part[3];
    }
}

// ---------------------------------------------------------------- rows into order
struct GatherParams {
    const int32_t* position;
    int64_t T, rows;
    int k;
    const char* x[2];
    char* out[2];
    int64_t bytes[2];
};

// A workgroup takes a token: V bytes a step are read once and written to each of its rows.
template <class V>
__device__ __forceinline__ void gather_row(const GatherParams& p, int64_t t, const char* x, char* out, int64_t bytes)
{
    const V* from = reinterpret_cast<const V*>(x + t * bytes);
    for (int64_t i = threadIdx.x; i < bytes / (int64_t)sizeof(V); i += 256) {
        const V v = from[i];
        for (int j = 0; j < p.k; ++j) {
            const int64_t r = p.position[t * p.k + j];
            if (r >= 0 && r < p.rows)
                reinterpret_cast<V*>(out + r * bytes)[i] = v;
        }
    }
}

__global__ void __launch_bounds__(256) moe_gather_kernel(GatherParams p)
{
    for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x)
        for (int s = 0; s < 2; ++s) {
            if (p.bytes[s] == 0)
                continue;
            const uintptr_t a = (uintptr_t)p.x[s] | (uintptr_t)p.out[s] | (uintptr_t)p.bytes[s];
            if (a % 16 == 0)
                gather_row<u32x4_t>(p, t, p.x[s], p.out[s], p.bytes[s]);
            else if (a % 4 == 0)
                gather_row<unsigned>(p, t, p.x[s], p.out[s], p.bytes[s]);
            else
                gather_row<unsigned char>(p, t, p.x[s], p.out[s], p.bytes[s]);
        }
}

// ---------------------------------------------------------------- rows back
struct CombineParams {
    const void *x, *dy;
    const int32_t* position;
    const float* weights;
    void *y, *dx;
    float* dweights;
    int64_t T, rows, H;
    int k;
};

template <bool BF16>
__device__ __forceinline__ float element(const void* p, int64_t i)
{
    if constexpr (BF16)
        return __uint_as_float((unsigned)static_cast<const unsigned short*>(p)[i] << 16);
    else
        return static_cast<const float*>(p)[i];
}

template <bool BF16>
__device__ __forceinline__ void put(void* p, int64_t i, float v)
{
    if constexpr (BF16)
        static_cast<unsigned short*>(p)[i] = f32_to_bf16_rne(v);
    else
        static_cast<float*>(p)[i] = v;
}

template <bool BF16>
__global__ void __launch_bounds__(256) moe_combine_kernel(CombineParams p)
{
    for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x)
        for (int64_t h = threadIdx.x; h < p.H; h += 256) {
            float v = 0.0f;
            for (int j = 0; j < p.k; ++j) {
                const int64_t r = p.position[t * p.k + j];
                if (r >= 0 && r < p.rows)
                    v = fmaf(p.weights ? p.weights[t * p.k + j] : 1.0f, element<BF16>(p.x, r * p.H + h), v);
            }
            put<BF16>(p.y, t * p.H + h, v);
        }
}

template <bool BF16>
__global__ void __launch_bounds__(256) moe_combine_grad_kernel(CombineParams p)
{
    __shared__ float part[4];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x)
        for (int j = 0; j < p.k; ++j) {
            const int64_t r = p.position[t * p.k + j];
            float dot = 0.0f;
            if (r >= 0 && r < p.rows) {
                const float w = p.weights[t * p.k + j];
                for (int64_t h = threadIdx.x; h < p.H; h += 256) {
                    const float d = element<BF16>(p.dy, t * p.H + h);
                    dot = fmaf(d, element<BF16>(p.x, r * p.H + h), dot);
                    put<BF16>(p.dx, r * p.H + h, w * d);
                }
            }
#pragma unroll
            for (int off = 1; off < 64; off <<= 1)
                dot += __shfl_xor(dot, off);
            __syncthreads();
            if (lane == 0)
                part[wave] = dot;
            __syncthreads();
            if (threadIdx.x == 0)
                p.dweights[t * p.k + j] = part[0] + part[1] + part[2] + part[3];
        }
}

// ---------------------------------------------------------------- checks
static int check_order(int64_t T, int k)
{
    if (T < 0 || k < 1)
        return set_error(TG_E_INVAL, "T must be >= 0, k >= 1");
    if (k > kOrderChoices || T > kOrderTokens)
        return set_error(TG_E_UNSUPPORTED, "at most 16 choices and 2^24 tokens");
    return TG_OK;
}

static int check_sort(int64_t T, int64_t E, int k)
{
    const int st = check_order(T, k);
    if (st != TG_OK)
        return st;
    if (E < 1)
        return set_error(TG_E_INVAL, "E must be >= 1");
    if (E > kOrderExperts)
        return set_error(TG_E_UNSUPPORTED, "at most 1024 experts");
    return TG_OK;
}

static int check_rows(int64_t T, int k, int64_t rows, const int32_t* position)
{
    const int st = check_order(T, k);
    if (st != TG_OK)
        return st;
    if (rows < 0)
        return set_error(TG_E_INVAL, "rows must be >= 0");
    if (rows > 0x7FFFFFFF)
        return set_error(TG_E_UNSUPPORTED, "rows must be below 2^31");
    if (T > 0 && (!position || ((uintptr_t)position & 3u)))
        return set_error(TG_E_INVAL, "position must be given, 4-byte aligned");
    return TG_OK;
}

static int check_combine(int64_t T, int k, int64_t rows, int64_t H, int dtype, const int32_t* position)
{
    const int st = check_rows(T, k, rows, position);
    if (st != TG_OK)
        return st;
    if (H < 1)
        return set_error(TG_E_INVAL, "H must be >= 1");
    if (H > kOrderWidth)
        return set_error(TG_E_UNSUPPORTED, "H is at most 2^24");
    if (dtype != TG_F32 && dtype != TG_BF16)
        return set_error(TG_E_INVAL, "rows are fp32 or bf16");
    return TG_OK;
}

static unsigned grid_of(int64_t n) { return (unsigned)std::min<int64_t>(n, 1 << 20); }

}  // namespace tg

using namespace tg;

extern "C" {

int tg_moe_sort_workspace_bytes(int64_t T, int64_t E, int k, size_t* bytes)
{
    const int st = check_sort(T, E, k);
    if (st != TG_OK)
        return st;
    if (!bytes)
        return set_error(TG_E_INVAL, "bytes is NULL");
    *bytes = 0;
    return TG_OK;
}

int tg_moe_sort(int64_t T, int64_t E, int k, const int32_t* ids, int32_t* position, int32_t* source,
                int32_t* offsets, void* workspace, size_t workspace_bytes)
{
    (void)workspace, (void)workspace_bytes;
    const int st = check_sort(T, E, k);
    if (st != TG_OK)
        return st;
    if (!offsets || (T > 0 && (!ids || !position || !source)) ||
        (((uintptr_t)ids | (uintptr_t)position | (uintptr_t)source | (uintptr_t)offsets) & 3u))
        return set_error(TG_E_INVAL, "ids, position, source and offsets must be given, 4-byte aligned");
    if (!have_device())
        return set_error(TG_E_UNSUPPORTED, "no HIP device");
    hipLaunchKernelGGL(moe_sort_kernel, dim3((unsigned)E + 1), dim3(256), 0, current_stream(), ids, T * k, (int)E,
                       position, source, offsets);
    return launched("moe_sort launch");
}

int tg_moe_gather(int64_t T, int k, int64_t rows, const int32_t* position, int64_t row_bytes, const void* x,
                  void* out, int64_t row2_bytes, const void* x2, void* out2)
{
    const int st = check_rows(T, k, rows, position);
    if (st != TG_OK)
        return st;
    if (row_bytes < 1 || row2_bytes < 0)
        return set_error(TG_E_INVAL, "row_bytes must be >= 1, row2_bytes >= 0");
    if (row_bytes > kOrderWidth || row2_bytes > kOrderWidth)
        return set_error(TG_E_UNSUPPORTED, "rows are at most 2^24 bytes");
    if (T == 0 || rows == 0)
        return TG_OK;
    if (!x || !out || (row2_bytes > 0 && (!x2 || !out2)))
        return set_error(TG_E_INVAL, "x and out must be given");
    if (!have_device())
        return set_error(TG_E_UNSUPPORTED, "no HIP device");
    const GatherParams p{position, T, rows, k, {static_cast<const char*>(x), static_cast<const char*>(x2)},
                         {static_cast<char*>(out), static_cast<char*>(out2)}, {row_bytes, row2_bytes}};
    hipLaunchKernelGGL(moe_gather_kernel, dim3(grid_of(T)), dim3(256), 0, current_stream(), p);
    return launched("moe_gather launch");
}

int tg_moe_combine(int64_t T, int k, int64_t rows, int64_t H, const void* x, int dtype, const int32_t* position,
                   const float* weights, void* y)
{
    const int st = check_combine(T, k, rows, H, dtype, position);
    if (st != TG_OK || T == 0)
        return st;
    const uintptr_t mask = dtype == TG_F32 ? 3u : 1u;
    if ((rows > 0 && !x) || !y || (((uintptr_t)x | (uintptr_t)y) & mask) || ((uintptr_t)weights & 3u))
        return set_error(TG_E_INVAL, "x and y must be given; x, y and weights aligned to their elements");
    if (!have_device())
        return set_error(TG_E_UNSUPPORTED, "no HIP device");
    const CombineParams p{x, nullptr, position, weights, y, nullptr, nullptr, T, rows, H, k};
    if (dtype == TG_BF16)
        hipLaunchKernelGGL(moe_combine_kernel<true>, dim3(grid_of(T)), dim3(256), 0, current_stream(), p);
    else
        hipLaunchKernelGGL(moe_combine_kernel<false>, dim3(grid_of(T)), dim3(256), 0, current_stream(), p);
    return launched("moe_combine launch");
}

int tg_moe_combine_grad(int64_t T, int k, int64_t rows, int64_t H, const void* dy, const void* x, int dtype,
                        const int32_t* position, const float* weights, void* dx, float* dweights)
{
    const int st = check_combine(T, k, rows, H, dtype, position);
    if (st != TG_OK || T == 0)
        return st;
    const uintptr_t mask = dtype == TG_F32 ? 3u : 1u;
    if (!dy || (rows > 0 && (!x || !dx)) || !weights || !dweights ||
        (((uintptr_t)dy | (uintptr_t)x | (uintptr_t)dx) & mask) || (((uintptr_t)weights | (uintptr_t)dweights) & 3u))
        return set_error(TG_E_INVAL, "dy, x, weights, dx and dweights must be given, aligned to their elements");
    if (!have_device())
        return set_error(TG_E_UNSUPPORTED, "no HIP device");
    const CombineParams p{x, dy, position, weights, nullptr, dx, dweights, T, rows, H, k};
    if (dtype == TG_BF16)
        hipLaunchKernelGGL(moe_combine_grad_kernel<true>, dim3(grid_of(T)), dim3(256), 0, current_stream(), p);
    else
        hipLaunchKernelGGL(moe_combine_grad_kernel<false>, dim3(grid_of(T)), dim3(256), 0, current_stream(), p);
    return launched("moe_combine_grad launch");
}

}  // extern "C"
