// Products of 8-bit matrices for few rows: the work is the stream of B
// (gemm_fp8.hip has the formula).
//
// A workgroup takes P panels of 16 columns and up to 16 MT rows; its W waves cut
// the chunks of 128 k into W neighbouring ranges, and their sums meet in LDS at
// the end.  Each wave has a ring of R chunks in LDS to itself, panels, rows and
// scales, which it fills R chunks ahead without registers and without barriers.  The
// products are the exact form in every call: the conversions are hidden behind
// the stream (16 x 28672 x 8192 44.7 us, with the fast form 44.2).
#pragma once

#include "fp8.hpp"
#include "kernels/gemm_tiled_dma.hpp"

namespace tg {

// Four neighbouring results from element `at` of C, of which the first `left` are there.
__device__ __forceinline__ void store_four(const F8Params& p, int64_t at, int64_t left, const f32x4_t& v)
{
    if (p.out_bf16) {
        unsigned short* to = static_cast<unsigned short*>(p.C) + at;
        if (p.vec_out && left >= 4) {
            typedef unsigned short u16x4 __attribute__((ext_vector_type(4)));
            *reinterpret_cast<u16x4*>(to) = u16x4{f32_to_bf16_rne(v[0]), f32_to_bf16_rne(v[1]), f32_to_bf16_rne(v[2]),
                                                  f32_to_bf16_rne(v[3])};
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (e < left)
                    to[e] = f32_to_bf16_rne(v[e]);
        }
    } else {
        float* to = static_cast<float*>(p.C) + at;
        if (p.vec_out && left >= 4) {
            *reinterpret_cast<f32x4_t*>(to) = f32x4_t{v[0], v[1], v[2], v[3]};
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (e < left)
                    to[e] = v[e];
        }
    }
}

// The same of a row.
__device__ __forceinline__ void store_results(const F8Params& p, int64_t row, int64_t col, const f32x4_t& v)
{
    store_four(p, row * p.N + col, p.N - col, v);
}

// One wave-wide load of 4 bytes a lane straight into LDS (lane l writes lds_addr
// + 4 l; as dma16).
__device__ __forceinline__ void dma4(i32x4_t rsrc, int voff, unsigned lds_addr)
{
    __asm__ __volatile__("s_nop 4\n\tbuffer_load_dword %0, %1, 0 offen lds" ::"v"(voff), "s"(rsrc), "{m0}"(lds_addr)
                         : "memory");
}

template <int MT, int P, int R, int W, bool BROWS>
struct F8Stream {
    static constexpr int SB = BROWS ? (16 * P + 63) / 64 : 1;      // transfers of B's scales
    static constexpr int INST = 2 * (P + MT) + 1 + SB;             // transfers of a chunk
    static constexpr int SLOT = (P + MT) * 2048 + 256 * (1 + SB);
    static constexpr int RING = W * R * SLOT, SUMS = W * P * MT * 1024;
    static constexpr int LDS = RING > SUMS ? RING : SUMS;
    static_assert(LDS <= 160 * 1024 && (R - 1) * INST <= 63 && P <= 8 && MT <= 4, "LDS, counted transfers, scales");
};

template <int MT, int P, int R, int W, bool BROWS>
__device__ __forceinline__ void f8_stream(const F8Params& p, char* lds, int64_t m0, int64_t m1, int64_t n0, int expert)
{
    using Cf = F8Stream<MT, P, R, W, BROWS>;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int l16 = lane & 15, g = lane >> 4;
    const int chunks = p.chunks, each = (chunks + W - 1) / W;
    const int first = wave * each, last = min(chunks, first + each);
    const int64_t Kp = (int64_t)chunks * 128, groups = (p.N + p.b_rows - 1) / p.b_rows;
    const int rows = (int)min(m1 - m0, (int64_t)(16 * MT)), cols = (int)min(p.N - n0, (int64_t)(16 * P));
    const i32x4_t ra = rsrc_words(p.A + m0 * Kp, kMaxRecords);
    const i32x4_t rb = rsrc_words(p.B + ((int64_t)expert * p.N + n0) * Kp, kMaxRecords);
    const i32x4_t rsa = rsrc_words(p.sA + m0 * chunks, kMaxRecords);
    const i32x4_t rsb = rsrc_words(p.sB + ((int64_t)expert * groups + n0 / p.b_rows) * chunks, kMaxRecords);
    const unsigned ring = (unsigned)(uintptr_t)(__attribute__((address_space(3))) char*)lds + (unsigned)(wave * R * Cf::SLOT);

    // a transfer brings eight rows, whole lines of 128 bytes (half lines, the
    // fragments' own order, come at half the rate); piece q of row r at q ^ ((r >> 1) & 7)
    int oa[2 * MT], ob[2 * P], osb[Cf::SB];
#pragma unroll
    for (int q = 0; q < 2 * P; ++q) {
        const int r = 8 * q + (lane >> 3);
        ob[q] = min(r, cols - 1) * (int)Kp + 16 * ((lane & 7) ^ ((r >> 1) & 7));
    }
#pragma unroll
    for (int q = 0; q < 2 * MT; ++q) {
        const int r = 8 * q + (lane >> 3);
        oa[q] = min(r, rows - 1) * (int)Kp + 16 * ((lane & 7) ^ ((r >> 1) & 7));
    }
    const int osa = min(lane, rows - 1) * chunks * 4;
#pragma unroll
    for (int q = 0; q < Cf::SB; ++q)
        osb[q] = BROWS ? min(64 * q + lane, cols - 1) * chunks * 4 : 0;
    // chunks past the range: zeros, scales too
    auto fetch = [&](int c, int slot) {
        const bool in = c < last;
        const unsigned to = ring + (unsigned)(slot * Cf::SLOT);
#pragma unroll
        for (int q = 0; q < 2 * P; ++q)
            dma16(rb, in ? ob[q] + c * 128 : kOOB, to + (unsigned)(q * 1024));
#pragma unroll
        for (int q = 0; q < 2 * MT; ++q)
            dma16(ra, in ? oa[q] + c * 128 : kOOB, to + (unsigned)((2 * P + q) * 1024));
        const unsigned scales = to + (P + MT) * 2048;
        dma4(rsa, in ? osa + c * 4 : kOOB, scales);
#pragma unroll
        for (int q = 0; q < Cf::SB; ++q)
            dma4(rsb, in ? osb[q] + c * 4 : kOOB, scales + 256u * (1 + q));
    };
    f32x4_t acc[P][MT];
#pragma unroll
    for (int j = 0; j < P; ++j)
#pragma unroll
        for (int i = 0; i < MT; ++i)
            acc[j][i] = f32x4_t{0.f, 0.f, 0.f, 0.f};

    const unsigned sw = (unsigned)(l16 >> 1) & 7u;
    const unsigned rd[2] = {(unsigned)l16 * 128u + ((unsigned)g ^ sw) * 16u, (unsigned)l16 * 128u + (((unsigned)g + 4) ^ sw) * 16u};
    auto multiply = [&](int slot) {
        const unsigned at = ring + (unsigned)(slot * Cf::SLOT), scales = at + (P + MT) * 2048;
        float sa[MT];
        Expanded a[MT];
        const float s = BROWS ? 1.0f : __uint_as_float(lds_read_b32(scales + 256));
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            a[i] = expand(lds_read_b128(at + (unsigned)((P + i) * 2048) + rd[0]),
                          lds_read_b128(at + (unsigned)((P + i) * 2048) + rd[1]));
            sa[i] = __uint_as_float(lds_read_b32(scales + (unsigned)(16 * i + l16) * 4)) * s;
        }
#pragma unroll
        for (int j = 0; j < P; ++j) {
            const Expanded b = expand(lds_read_b128(at + (unsigned)(j * 2048) + rd[0]),
                                      lds_read_b128(at + (unsigned)(j * 2048) + rd[1]));
            u32x4_t sb;
            if constexpr (BROWS)
                sb = lds_read_b128(scales + 256 + (unsigned)(16 * j + 4 * g) * 4);
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const f32x4_t d = mfma_exact(b, a[i]);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    // element first, then reinterpreted
                    const unsigned w = BROWS ? sb[e] : 0u;
                    acc[j][i][e] = fmaf(d[e], BROWS ? sa[i] * __uint_as_float(w) : sa[i], acc[j][i][e]);
                }
            }
        }
    };
#pragma unroll
    for (int d = 0; d < R; ++d)
        fetch(first + d, d);
    int slot = 0;
    for (int c = 0; c < each; ++c) {
        wait_vmcnt<(R - 1) * Cf::INST>();              // chunk c has landed
        __asm__ __volatile__("" ::: "memory");
        multiply(slot);
        wait_lgkm0();                                  // and is in registers
        fetch(first + c + R, slot);
        slot = slot + 1 == R ? 0 : slot + 1;
    }
    wait_vm_all();
    __syncthreads();

    f32x4_t* const sums = reinterpret_cast<f32x4_t*>(lds);
#pragma unroll
    for (int j = 0; j < P; ++j)
#pragma unroll
        for (int i = 0; i < MT; ++i)
            sums[(wave * P * MT + j * MT + i) * 64 + lane] = acc[j][i];
    __syncthreads();
    for (int t = tid; t < P * MT * 64; t += 64 * W) {
        f32x4_t sum = sums[t];
#pragma unroll
        for (int w = 1; w < W; ++w)
            sum += sums[w * P * MT * 64 + t];
        const int j = t / (MT * 64), i = t / 64 % MT, l = t % 64;
        const int64_t row = m0 + 16 * i + l % 16, col = n0 + 16 * j + l / 16 * 4;
        if (row < m1 && col < p.N) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                sum[e] = activate(sum[e] + (p.bias && col + e < p.N ? p.bias[col + e] : 0.0f), p.act);
            store_results(p, row, col, sum);
        }
    }
}

template <int MT, int P, int R, int W, bool BROWS>
__global__ void __launch_bounds__(64 * W) gemm_fp8_stream_kernel(F8Params p)
{
    extern __shared__ __align__(16) char lds[];
    const int tiles_n = (int)((p.N + 16 * P - 1) / (16 * P));
    int64_t m0 = 0, m1 = p.M;
    int tn = blockIdx.x, expert = 0;
    if (p.offsets && !expert_tile<16 * MT>(p, tiles_n, m0, m1, tn, expert))
        return;
    f8_stream<MT, P, R, W, BROWS>(p, lds, m0, m1, (int64_t)tn * 16 * P, expert);
}

}  // namespace tg
