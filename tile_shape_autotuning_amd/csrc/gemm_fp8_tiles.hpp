// Tiles of the products of 8-bit matrices, for many rows (gemm_fp8.hip has the
// formula).
//
// A workgroup of WGM x WGN waves takes BM rows and BN columns.  Chunks of 128 k
// of both operands travel global -> LDS without registers, two chunks deep; a
// row of a chunk is 128 bytes, eight 16-byte pieces, piece p of row r at
// p ^ ((r >> 1) & 7), so that 16 rows that read one piece hit 16 slots of a
// 256-byte window.  A wave multiplies a chunk's fragments from zero and adds
// each 16 x 16 result, times its scales, to its sums.  There is one barrier a
// chunk: all of its fragments are in registers and the next chunk has landed,
// so its buffer can be filled again.  Scales come eight chunks at a time through
// registers into LDS, [chunk][row].
#pragma once

#include <type_traits>

#include "fp8.hpp"
#include "kernels/gemm_tiled_dma.hpp"

namespace tg {

template <int BM, int BN, int WGM, int WGN, bool BROWS>
struct F8Tile {
    static constexpr int W = WGM * WGN, T = 64 * W;
    static constexpr int WM = BM / WGM, WN = BN / WGN, FM = WM / 16, FN = WN / 16;
    static constexpr int CHUNK = 128;                  // bytes of a row in LDS
    static constexpr int STAGE = (BM + BN) * CHUNK;
    static constexpr int INST = STAGE / 1024 / W;      // transfers a wave and chunk, eight rows each
    static constexpr int NS = 8;                       // chunks of a batch of scales
    static constexpr int SB = BROWS ? BN : (BN + 127) / 128;
    static constexpr int SROW = BM + SB;               // floats of one chunk's scales
    static constexpr int SLOADS = (BM + SB) * NS / T + ((BM + SB) * NS % T != 0);
    static constexpr int LDS = 2 * STAGE + 2 * NS * SROW * 4;
    static_assert(STAGE % (1024 * W) == 0 && BM % 8 == 0, "whole transfers a wave, each of one operand");
    static_assert(LDS <= 160 * 1024, "LDS");
    static_assert(WN <= 128 && 128 % WN == 0, "a wave's columns share a block's scale");
};

// Rows m0 .. m1 - 1 of A (at most BM of them matter), columns n0 .. of B.
template <int BM, int BN, int WGM, int WGN, bool BROWS, bool EXACT>
__device__ __forceinline__ void f8_tile(const F8Params& p, char* lds, int64_t m0, int64_t m1, int64_t n0, int expert)
{
    using Cf = F8Tile<BM, BN, WGM, WGN, BROWS>;
    constexpr int FM = Cf::FM, FN = Cf::FN;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int l16 = lane & 15, g = lane >> 4;
    const int wm = wave / WGN, wn = wave % WGN;
    const int chunks = p.chunks;
    const int64_t Kp = (int64_t)chunks * 128;
    const int64_t groups = (p.N + p.b_rows - 1) / p.b_rows;
    const unsigned char* A = p.A + m0 * Kp;
    const unsigned char* B = p.B + ((int64_t)expert * p.N + n0) * Kp;
    const int rows = (int)min(m1 - m0, (int64_t)BM), cols = (int)min(p.N - n0, (int64_t)BN);
    const unsigned lds_base = (unsigned)(uintptr_t)(__attribute__((address_space(3))) char*)lds;

    // transfer q of this wave: rows 8 j .. 8 j + 7 of the stage, j = wave + q W
    // (rows of A, then of B); rows past the matrix read as its last
    int vo[Cf::INST];
#pragma unroll
    for (int q = 0; q < Cf::INST; ++q) {
        const int r = (wave + q * Cf::W) * 8 + (lane >> 3);
        const int piece = (lane & 7) ^ ((r >> 1) & 7);
        vo[q] = (r < BM ? min(r, rows - 1) : min(r - BM, cols - 1)) * (int)Kp + piece * 16;
    }
    auto fetch = [&](int c, int buf) {
        const i32x4_t ra = rsrc_words(A + (int64_t)c * 128, kMaxRecords);
        const i32x4_t rb = rsrc_words(B + (int64_t)c * 128, kMaxRecords);
#pragma unroll
        for (int q = 0; q < Cf::INST; ++q) {
            const int j = wave + q * Cf::W;
            dma16(j * 8 < BM ? ra : rb, vo[q], lds_base + (unsigned)(buf * Cf::STAGE + j * 1024));
        }
    };

    // scales of chunks 8 b .. 8 b + 7: value i is chunk i % 8 of row i / 8 (A, then B)
    float* const scales = reinterpret_cast<float*>(lds + 2 * Cf::STAGE);
    const float* sA = p.sA + m0 * chunks;
    const float* sB = p.sB + ((int64_t)expert * groups + n0 / p.b_rows) * chunks;
    const int sb_rows = BROWS ? cols : (cols + 127) / 128;
    float held[Cf::SLOADS];
    auto load_scales = [&](int b) {
#pragma unroll
        for (int q = 0; q < Cf::SLOADS; ++q) {
            const int i = tid + q * Cf::T, r = i / Cf::NS, c = min(b * Cf::NS + i % Cf::NS, chunks - 1);
            held[q] = r < BM ? sA[(int64_t)min(r, rows - 1) * chunks + c]
                             : sB[(int64_t)min(r - BM, sb_rows - 1) * chunks + c];
        }
    };
    auto keep_scales = [&](int b) {
#pragma unroll
        for (int q = 0; q < Cf::SLOADS; ++q) {
            const int i = tid + q * Cf::T;
            if (Cf::SROW * Cf::NS % Cf::T == 0 || i < Cf::SROW * Cf::NS)
                scales[(b & 1) * Cf::NS * Cf::SROW + i % Cf::NS * Cf::SROW + i / Cf::NS] = held[q];
        }
    };

    f32x4_t acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
            acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};

    // fragment reads: piece h 4 + g of the row
    const unsigned sw = (unsigned)(l16 >> 1) & 7u;
    const unsigned rd[2] = {(unsigned)l16 * 128u + ((unsigned)g ^ sw) * 16u, (unsigned)l16 * 128u + (((unsigned)g + 4) ^ sw) * 16u};
    auto fragment = [&](unsigned at, u32x4_t (&f)[2]) {
        f[0] = lds_read_b128(at + rd[0]);
        f[1] = lds_read_b128(at + rd[1]);
    };

    fetch(0, 0);
    load_scales(0);
    keep_scales(0);
    fetch(min(1, chunks - 1), 1);
    wait_vmcnt<Cf::INST>();
    wait_lgkm0();
    block_barrier();

    for (int c = 0; c < chunks; ++c) {
        const unsigned st = lds_base + (unsigned)((c & 1) * Cf::STAGE);
        const unsigned at_a = st + (unsigned)(wm * Cf::WM * 128), at_b = st + (unsigned)((BM + wn * Cf::WN) * 128);
        const float* sc = scales + ((c / Cf::NS & 1) * Cf::NS + c % Cf::NS) * Cf::SROW;
        if (c % Cf::NS == 0 && c + Cf::NS < chunks)
            load_scales(c / Cf::NS + 1);
        if (c % Cf::NS == Cf::NS / 2 && c + Cf::NS / 2 < chunks)
            keep_scales(c / Cf::NS + 1);

        float sa[FM];
        f32x4_t sb[FN];
#pragma unroll
        for (int i = 0; i < FM; ++i)
            sa[i] = sc[wm * Cf::WM + 16 * i + l16];
        if constexpr (BROWS) {
#pragma unroll
            for (int j = 0; j < FN; ++j)
                sb[j] = *reinterpret_cast<const f32x4_t*>(sc + BM + wn * Cf::WN + 16 * j + 4 * g);
        } else {
            const float s = sc[BM + wn * Cf::WN / 128];
#pragma unroll
            for (int i = 0; i < FM; ++i)
                sa[i] *= s;
        }
        u32x4_t b[FN][2], a[2][2];
#pragma unroll
        for (int j = 0; j < FN; ++j)
            fragment(at_b + (unsigned)(j * 16 * 128), b[j]);
        fragment(at_a, a[0]);
        if (FM > 1)
            fragment(at_a + 16 * 128, a[1]);
        Expanded be[EXACT ? FN : 1];
        if constexpr (EXACT) {
#pragma unroll
            for (int j = 0; j < FN; ++j)
                be[j] = expand(b[j][0], b[j][1]);
        }
        f32x4_t d[2][FN];
        auto add = [&](int i, int j) {
#pragma unroll
            for (int r = 0; r < 4; ++r)
                acc[i][j][r] = fmaf(d[i & 1][j][r], BROWS ? sa[i] * sb[j][r] : sa[i], acc[i][j][r]);
        };
        // row i's products, and the sums of the row before
#pragma unroll
        for (int i = 0; i < FM; ++i) {
            if (i == FM - 1) {
                // every fragment of this chunk is in registers, the next chunk has landed
                wait_lgkm0();
                wait_vmcnt<0>();
                block_barrier();
                // past the end a chunk that nothing reads: no branch, across which the
                // compiler would move the sums and spill them
                fetch(min(c + 2, chunks - 1), c & 1);
            }
            Expanded ae;
            if constexpr (EXACT)
                ae = expand(a[i & 1][0], a[i & 1][1]);
#pragma unroll
            for (int j = 0; j < FN; ++j) {
                if constexpr (EXACT)
                    d[i & 1][j] = mfma_exact(be[j], ae);
                else
                    d[i & 1][j] = mfma_fp8(join8(b[j][0], b[j][1]), join8(a[i & 1][0], a[i & 1][1]),
                                           f32x4_t{0.f, 0.f, 0.f, 0.f});
                if (i > 0)
                    add(i - 1, j);
                __builtin_amdgcn_sched_barrier(0);
            }
            if (i + 2 < FM)
                fragment(at_a + (unsigned)((i + 2) * 16 * 128), a[i & 1]);
            __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int j = 0; j < FN; ++j)
            add(FM - 1, j);
    }
    wait_vm_all();                                     // transfers still on their way to LDS

#pragma unroll
    for (int i = 0; i < FM; ++i) {
        const int r = wm * Cf::WM + 16 * i + l16;
        if (r >= rows)
            continue;
#pragma unroll
        for (int j = 0; j < FN; ++j) {
            const int col = wn * Cf::WN + 16 * j + 4 * g;
            if (col < cols)
                store_results(p, m0 + r, n0 + col, acc[i][j]);
        }
    }
}

template <int BM, int BN, int WGM, int WGN, bool BROWS, bool EXACT>
__global__ void __launch_bounds__(64 * WGM * WGN, 2) gemm_fp8_tiles_kernel(F8Params p)
{
    extern __shared__ __align__(16) char lds[];
    const int tiles_n = (int)((p.N + BN - 1) / BN);
    int64_t m0, m1;
    int tn, expert = 0;
    if (p.offsets) {
        if (!expert_tile<BM>(p, tiles_n, m0, m1, tn, expert))
            return;
    } else {
        const int tiles_m = (int)((p.M + BM - 1) / BM);
        int tile, tm, split;
        map_block(blockIdx.x, gridDim.x, tiles_m, tiles_n, p.group_m, tile, tm, tn, split);
        m0 = (int64_t)tm * BM;
        m1 = p.M;
    }
    f8_tile<BM, BN, WGM, WGN, BROWS, EXACT>(p, lds, m0, m1, (int64_t)tn * BN, expert);
}

}  // namespace tg
