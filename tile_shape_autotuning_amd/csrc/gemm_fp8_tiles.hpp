// Tiles of the products of 8-bit matrices, for many rows (gemm_fp8.hip has the
// formula).
//
// A workgroup of WGM x WGN waves takes BM rows and BN columns.  Chunks of 128 k
// of both operands travel global -> LDS without registers, ST chunks deep; a
// row of a chunk is 128 bytes, eight 16-byte pieces, piece p of row r at
// p ^ ((r >> 1) & 7), so that 16 rows that read one piece hit 16 slots of a
// 256-byte window.  A wave multiplies a chunk's fragments from zero and adds
// each 16 x 16 result, times its scales, to its sums: with fast sums four FMAs a
// lane beside a matrix instruction of 32 cycles, in whose shadow they fit if they are
// issued between the instructions and take a result some instructions old.  In the
// exact form they stand beside four instructions of 16 cycles, and the expansion of
// the codes, sixteen conversions a fragment, with them (8192 x 8192 x 8192: 929 us,
// matrix cores busy 53 % and vector instructions 58 % of the SIMDs' cycles; fast
// sums 468 us, 66 % and 49 %).
//
// Order of a chunk.  Rows of 16 x 16 results one after the other, but for the
// last two, whose columns alternate: a column's fragments of B are then free early,
// and those of the next chunk, with its first rows', are read while the rest is
// multiplied.  The one barrier of a chunk stands before these two rows: all of its
// fragments are in registers and the next chunk has landed, so its buffer can be
// filled again, a transfer after each instruction.  Scales come eight or four
// chunks at a time through registers into LDS, [chunk][row].
#pragma once

#include <type_traits>

#include "fp8.hpp"
#include "kernels/gemm_tiled_dma.hpp"

namespace tg {

template <int BM, int BN, int WGM, int WGN, int ST, bool BROWS>
struct F8Tile {
    static constexpr int W = WGM * WGN, T = 64 * W;
    static constexpr int WM = BM / WGM, WN = BN / WGN, FM = WM / 16, FN = WN / 16;
    static constexpr int CHUNK = 128;                  // bytes of a row in LDS
    static constexpr int STAGE = (BM + BN) * CHUNK;
    static constexpr int INST = STAGE / 1024 / W;      // transfers a wave and chunk, eight rows each
    static constexpr int SB = BROWS ? BN : (BN + 127) / 128;
    static constexpr int SROW = BM + SB;               // floats of one chunk's scales
    // chunks of a batch of scales
    static constexpr int NS = ST * STAGE + 2 * 8 * SROW * 4 <= 160 * 1024 ? 8 : 4;
    static constexpr int SLOADS = (BM + SB) * NS / T + ((BM + SB) * NS % T != 0);
    static constexpr int LDS = ST * STAGE + 2 * NS * SROW * 4;
    static constexpr int AR = FM < 4 ? FM : 4;         // rows' fragments in registers
    static_assert(STAGE % (1024 * W) == 0 && BM % 8 == 0, "whole transfers a wave, each of one operand");
    static_assert(LDS <= 160 * 1024 && ST >= 2 && (ST - 1) * INST <= 63, "LDS, counted transfers");
    static_assert(FM == 2 || FM % 4 == 0, "rows' fragments of neighbouring chunks in the same registers");
    static_assert(WN <= 128 && 128 % WN == 0, "a wave's columns share a block's scale");
};

// Rows m0 .. m1 - 1 of A (at most BM of them matter), columns n0 .. of B, chunks
// c0 .. c1 - 1 of the reduction.
template <int BM, int BN, int WGM, int WGN, int ST, bool BROWS, bool EXACT>
__device__ __forceinline__ void f8_tile(const F8Params& p, char* lds, int64_t m0, int64_t m1, int64_t n0, int expert, int c0, int c1)
{
    using Cf = F8Tile<BM, BN, WGM, WGN, ST, BROWS>;
    constexpr int FM = Cf::FM, FN = Cf::FN;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int l16 = lane & 15, g = lane >> 4;
    const int wm = wave / WGN, wn = wave % WGN;
    const int chunks = c1 - c0;
    const int64_t Kp = (int64_t)p.chunks * 128;
    const int64_t groups = (p.N + p.b_rows - 1) / p.b_rows;
    const unsigned char* A = p.A + m0 * Kp + (int64_t)c0 * 128;
    const unsigned char* B = p.B + ((int64_t)expert * p.N + n0) * Kp + (int64_t)c0 * 128;
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
    // past the end the last chunk once more, which nothing reads: no branch, across
    // which the compiler would move sums and spill them
    struct Source {
        i32x4_t a, b;
        unsigned to;
    };
    auto source = [&](int c, int buf) {
        const int64_t at = (int64_t)min(c, chunks - 1) * 128;
        return Source{rsrc_words(A + at, kMaxRecords), rsrc_words(B + at, kMaxRecords),
                      lds_base + (unsigned)(buf * Cf::STAGE)};
    };
    auto fetch = [&](const Source& s, int q) {
        const int j = wave + q * Cf::W;
        const bool of_a = BM % (8 * Cf::W) == 0 ? q * Cf::W * 8 < BM : j * 8 < BM;
        dma16(of_a ? s.a : s.b, vo[q], s.to + (unsigned)(j * 1024));
    };

    // scales of chunks NS b .. NS b + NS - 1: value i is chunk i % NS of row i / NS (A, then B)
    float* const scales = reinterpret_cast<float*>(lds + ST * Cf::STAGE);
    const float* sA = p.sA + m0 * p.chunks + c0;
    const float* sB = p.sB + ((int64_t)expert * groups + n0 / p.b_rows) * p.chunks + c0;
    const int sb_rows = BROWS ? cols : (cols + 127) / 128;
    float held[Cf::SLOADS];
    auto load_scales = [&](int b) {
#pragma unroll
        for (int q = 0; q < Cf::SLOADS; ++q) {
            const int i = tid + q * Cf::T, r = i / Cf::NS, c = min(b * Cf::NS + i % Cf::NS, chunks - 1);
            held[q] = r < BM ? sA[(int64_t)min(r, rows - 1) * p.chunks + c]
                             : sB[(int64_t)min(r - BM, sb_rows - 1) * p.chunks + c];
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

    // fragments: pieces g and g + 4 of the lane's row; bases of both and constant offsets
    const unsigned sw = (unsigned)(l16 >> 1) & 7u;
    const unsigned piece0 = (unsigned)l16 * 128u + ((unsigned)g ^ sw) * 16u;
    const unsigned piece1 = (unsigned)l16 * 128u + (((unsigned)g + 4) ^ sw) * 16u;
    struct Base {
        unsigned a0, a1, b0, b1;
    };
    auto base_of = [&](int buf) {
        const unsigned a = lds_base + (unsigned)(buf * Cf::STAGE + wm * Cf::WM * 128);
        const unsigned b = lds_base + (unsigned)(buf * Cf::STAGE + (BM + wn * Cf::WN) * 128);
        Base r{a + piece0, a + piece1, b + piece0, b + piece1};
        __asm__ __volatile__("" : "+v"(r.a0), "+v"(r.a1), "+v"(r.b0), "+v"(r.b1));
        return r;
    };
    u32x4_t a[Cf::AR][2], b[FN][2];
    auto read_a = [&](const Base& s, int i) {
        a[i % Cf::AR][0] = lds_read_b128(s.a0 + (unsigned)(i * 2048));
        a[i % Cf::AR][1] = lds_read_b128(s.a1 + (unsigned)(i * 2048));
    };
    auto read_b = [&](const Base& s, int j) {
        b[j][0] = lds_read_b128(s.b0 + (unsigned)(j * 2048));
        b[j][1] = lds_read_b128(s.b1 + (unsigned)(j * 2048));
    };

    constexpr int NM = FM * FN, TAIL = (FM - 2) * FN;
    constexpr int LAG = EXACT ? 1 : NM < 3 ? 1 : 3;    // results between one and the addition of it
    constexpr int DR = LAG + 1;
    auto row_of = [](int x) { return x < TAIL ? x / FN : FM - 2 + ((x - TAIL) & 1); };
    auto col_of = [](int x) { return x < TAIL ? x % FN : (x - TAIL) / 2; };

    load_scales(0);
#pragma unroll
    for (int t = 0; t < ST; ++t) {
        const Source s = source(t, t);
#pragma unroll
        for (int q = 0; q < Cf::INST; ++q)
            fetch(s, q);
    }
    keep_scales(0);
    wait_vmcnt<(ST - 1) * Cf::INST>();
    wait_lgkm0();
    block_barrier();
    Base cur = base_of(0);
    // in the order in which a chunk reads the next one's: the first product then
    // waits for its own fragments only
    read_a(cur, 0);
    read_a(cur, 1);
#pragma unroll
    for (int j = 0; j < FN; ++j)
        read_b(cur, j);

    int buf = 0;
    for (int c = 0; c < chunks; ++c) {
        const float* sc = scales + ((c / Cf::NS & 1) * Cf::NS + c % Cf::NS) * Cf::SROW;
        if (c % Cf::NS == 0 && c + Cf::NS < chunks)
            load_scales(c / Cf::NS + 1);
        if (c % Cf::NS == Cf::NS / 2 && c + Cf::NS / 2 < chunks)
            keep_scales(c / Cf::NS + 1);
        const int nbuf = buf + 1 == ST ? 0 : buf + 1;
        const Base nxt = base_of(nbuf);
        const Source src = source(c + ST, buf);

        float sa[FM], s = 1.0f;
        f32x4_t sb[FN];
        if constexpr (BROWS) {
#pragma unroll
            for (int j = 0; j < FN; ++j)
                sb[j] = *reinterpret_cast<const f32x4_t*>(sc + BM + wn * Cf::WN + 16 * j + 4 * g);
        } else {
            s = sc[BM + wn * Cf::WN / 128];
        }
#pragma unroll
        for (int i = 0; i < FM; ++i)
            sa[i] = sc[wm * Cf::WM + 16 * i + l16];
        __builtin_amdgcn_sched_barrier(0);             // on their way before the first product, not waited for
        Expanded be[EXACT ? FN : 1], ae[EXACT ? 2 : 1];
        if constexpr (EXACT) {
#pragma unroll
            for (int j = 0; j < FN; ++j)
                be[j] = expand(b[j][0], b[j][1]);
        }
        f32x4_t d[DR];
        auto add = [&](int x) {
            const int i = row_of(x), j = col_of(x);
            if (!BROWS && j == 0)
                sa[i] *= s;
#pragma unroll
            for (int r = 0; r < 4; ++r)
                acc[i][j][r] = fmaf(d[x % DR][r], BROWS ? sa[i] * sb[j][r] : sa[i], acc[i][j][r]);
        };
#pragma unroll
        for (int x = 0; x < NM; ++x) {
            const int i = row_of(x), j = col_of(x);
            if (x == TAIL) {
                // every fragment of this chunk is in registers, the next chunk has landed
                wait_lgkm0();
                wait_vmcnt<(ST - 2) * Cf::INST>();
                block_barrier();
            }
            if constexpr (EXACT) {
                if (j == 0)
                    ae[i & 1] = expand(a[i % Cf::AR][0], a[i % Cf::AR][1]);
                d[x % DR] = mfma_exact(be[j], ae[i & 1]);
            } else {
                d[x % DR] = mfma_fp8(join8(b[j][0], b[j][1]), join8(a[i % Cf::AR][0], a[i % Cf::AR][1]),
                                     f32x4_t{0.f, 0.f, 0.f, 0.f});
            }
            if (x >= LAG)
                add(x - LAG);
            __builtin_amdgcn_sched_barrier(0);
            if (x < TAIL) {
                if (j == 0 && i + 2 < FM)
                    read_a(cur, i + 2);
            } else {
                const int y = x - TAIL;                // 0 .. 2 FN - 1
                // the next chunk's first rows' fragments where theirs are free, and its columns'
                if (FM > 2 && y < 2)
                    read_a(nxt, y);
                if (y & 1)
                    read_b(nxt, j);
#pragma unroll
                for (int q = y * Cf::INST / (2 * FN); q < (y + 1) * Cf::INST / (2 * FN); ++q)
                    fetch(src, q);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        if constexpr (FM == 2) {
            read_a(nxt, 0);
            read_a(nxt, 1);
        }
#pragma unroll
        for (int x = NM - LAG; x < NM; ++x)
            add(x);
        cur = nxt;
        buf = nbuf;
    }
    wait_vm_all();                                     // transfers still on their way to LDS

    f32x4_t bias[FN];
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int col = wn * Cf::WN + 16 * j + 4 * g + e;
            bias[j][e] = p.bias && col < cols ? p.bias[n0 + col] : 0.0f;
        }
    // a row of results at a time: more would not fit the registers
    auto finish = [&](int i) {
#pragma unroll
        for (int j = 0; j < FN; ++j)
            acc[i][j] += bias[j];
        if (p.act == TG_ACT_RELU) {
#pragma unroll
            for (int j = 0; j < FN; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    acc[i][j][e] = activate(acc[i][j][e], TG_ACT_RELU);
        } else if (p.act == TG_ACT_GELU) {
#pragma unroll
            for (int j = 0; j < FN; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    acc[i][j][e] = activate(acc[i][j][e], TG_ACT_GELU);
        }
        __builtin_amdgcn_sched_barrier(0);
    };
    if constexpr (Cf::WN % 64 == 0) {
        if (p.out_bf16 && p.line_out) {
            // whole lines of bf16 through the wave's own part of the ring: eight
            // columns, 16 bytes, of row r at unit u ^ (r & 7) of each 128 bytes
            block_barrier();                           // every wave's transfers and reads are done
            constexpr int ROW = Cf::WN * 2, UNITS = ROW / 16, RPI = 64 / UNITS;
            static_assert(Cf::W * Cf::WM * ROW <= ST * Cf::STAGE && Cf::WM % RPI == 0, "the tile fits the ring");
            char* const mine = lds + wave * Cf::WM * ROW;
            typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
#pragma unroll
            for (int i = 0; i < FM; ++i) {
                finish(i);
#pragma unroll
                for (int j = 0; j < FN; ++j) {
                    const int r = 16 * i + l16, u = 2 * j + (g >> 1);
                    const f32x4_t v = acc[i][j];
                    *reinterpret_cast<u32x2*>(mine + r * ROW + (u ^ (l16 & 7)) * 16 + (g & 1) * 8) =
                        u32x2{f32_to_bf16_rne(v[0]) | (unsigned)f32_to_bf16_rne(v[1]) << 16,
                              f32_to_bf16_rne(v[2]) | (unsigned)f32_to_bf16_rne(v[3]) << 16};
                }
            }
            wait_lgkm0();
            __asm__ __volatile__("" ::: "memory");
            // RPI rows an instruction
            const int u = lane % UNITS, col = wn * Cf::WN + 8 * u;
            unsigned short* const to = static_cast<unsigned short*>(p.C) + (m0 + wm * Cf::WM) * p.N + n0 + col;
#pragma unroll 4
            for (int q = 0; q < Cf::WM / RPI; ++q) {
                const int r = q * RPI + lane / UNITS;
                const u32x4_t v = *reinterpret_cast<const u32x4_t*>(mine + r * ROW + (u ^ (r & 7)) * 16);
                if (wm * Cf::WM + r < rows && col < cols)
                    *reinterpret_cast<u32x4_t*>(to + (int64_t)r * p.N) = v;
            }
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < FM; ++i) {
        finish(i);
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

template <int BM, int BN, int WGM, int WGN, int ST, bool BROWS, bool EXACT>
__global__ void __launch_bounds__(64 * WGM * WGN, 2) gemm_fp8_tiles_kernel(F8Params p)
{
    extern __shared__ __align__(16) char lds[];
    const int tiles_n = (int)((p.N + BN - 1) / BN);
    int64_t m0, m1;
    int tn, expert = 0, c0 = 0, c1 = p.chunks;
    if (p.offsets) {
        if (!expert_tile<BM>(p, tiles_n, m0, m1, tn, expert))
            return;
    } else {
        const int tiles_m = (int)((p.M + BM - 1) / BM);
        int tile, tm, split;
        map_block(blockIdx.x, gridDim.x, tiles_m, tiles_n, p.group_m, tile, tm, tn, split);
        m0 = (int64_t)tm * BM;
        m1 = p.M;
        if (p.split > 1) {                             // sums of a part of the chunks, to its slab
            c0 = split * p.each;
            c1 = min(p.chunks, c0 + p.each);
            p.C = p.slabs + split * p.slab;
        }
    }
    f8_tile<BM, BN, WGM, WGN, ST, BROWS, EXACT>(p, lds, m0, m1, (int64_t)tn * BN, expert, c0, c1);
}

}  // namespace tg
