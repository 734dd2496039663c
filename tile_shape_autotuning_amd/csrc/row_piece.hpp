// N neighbouring elements of a row, loaded 16 bytes at a time at any alignment.
//
// A load and its conversion are kept apart.  Converted where it is loaded, under
// the branch for a row's end or for a row that isn't there, each piece is waited
// for before the next load is issued; so the loads have no branch for the
// end (the last N elements of the row, moved down by those before the piece), rows
// shorter than a piece are a branch of the whole call, and arrived() stands
// between loads and the first use.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kernels/common.hpp"

namespace tg {

// Sixteen bytes of any alignment: the memory takes them as they are.
typedef u32x4_t u32x4_any __attribute__((aligned(1)));

template <bool BF16, int N>
struct Piece {
    static constexpr int D = N / (BF16 ? 2 : 1);       // dwords
    static_assert(D == 4 || D == 8, "whole loads");
    u32x4_t v[D / 4];                                  // whole, so that a load needs no moves

    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int q = 0; q < D / 4; ++q)
            v[q] = u32x4_t{0, 0, 0, 0};
    }
    // Elements h .. h + N - 1 of `row`, which has H >= N; arrived() and end(h, H) have to follow.
    // ONCE: it is not read again soon, and need not stay in the caches.
    template <bool ONCE = false>
    __device__ __forceinline__ void load(const void* row, int64_t h, int64_t H)
    {
        const int64_t at = min(h, H - N) * (BF16 ? 2 : 4);
        const u32x4_any* from = reinterpret_cast<const u32x4_any*>(static_cast<const char*>(row) + at);
#pragma unroll
        for (int q = 0; q < D / 4; ++q)
            v[q] = ONCE ? __builtin_nontemporal_load(from + q) : from[q];
    }
    // The same of a row with H < N.
    __device__ __forceinline__ void load_short(const void* row, int64_t h, int64_t H)
    {
        clear();
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (h + i < H) {
                if constexpr (BF16)
                    v[0][i / 2] |= (unsigned)static_cast<const unsigned short*>(row)[h + i] << (16 * (i & 1));
                else
                    v[i / 4][i % 4] = static_cast<const unsigned*>(row)[h + i];
            }
    }
    __device__ __forceinline__ void arrived()
    {
#pragma unroll
        for (int q = 0; q < D / 4; ++q)
            __asm__ __volatile__("" : "+v"(v[q]));
    }
    // Elements from H on become zero.
    __device__ __forceinline__ void end(int64_t h, int64_t H)
    {
        if (H < N || h + N <= H)
            return;
        const int skip = (int)min((int64_t)N, h - (H - N));
        unsigned w[D];
#pragma unroll
        for (int i = 0; i < D; ++i)
            w[i] = v[i / 4][i % 4];
        if constexpr (BF16)
            if (skip & 1) {
#pragma unroll
                for (int i = 0; i < D; ++i)
                    w[i] = w[i] >> 16 | (i + 1 < D ? w[i + 1 < D ? i + 1 : i] << 16 : 0u);
            }
#pragma unroll
        for (int by = 1; by <= D; by <<= 1)            // dwords
            if (skip / (BF16 ? 2 : 1) & by) {
#pragma unroll
                for (int i = 0; i < D; ++i)
                    w[i] = i + by < D ? w[i + by < D ? i + by : i] : 0u;
            }
#pragma unroll
        for (int i = 0; i < D; ++i)
            v[i / 4][i % 4] = w[i];
    }
    __device__ __forceinline__ float operator[](int i) const
    {
        if constexpr (BF16)
            return __uint_as_float(i & 1 ? v[0][i / 2] & 0xFFFF0000u : v[0][i / 2] << 16);
        else
            return __uint_as_float(v[i / 4][i % 4]);
    }
};

}  // namespace tg
