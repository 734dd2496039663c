// The product of a few rows with panel after panel of streamed weights: the
// core of the 4-bit product and of the expert layers (storage and arithmetic of
// 4-bit weights: w4.hpp).
//
// A few rows use every weight once, so the weights' stream from HBM is the
// bound, and what decides is how many bytes are on their way at any time.  The
// reduction is therefore cut among the W waves of a workgroup: a wave keeps
// its rows' fragments of CW chunks (128 k each) in registers, for all panels
// that the workgroup works on, and a step is the CW chunks of the next panel,
// whose loads are all issued one to three steps ahead.  A is read once a
// workgroup rather than once a panel.  The waves' sums meet in LDS and are added
// in wave order.  One barrier, which leaves the loads in flight, serves up to
// four panels: their tiles are then added up by as many waves at once, while
// the others go on in the other half of the buffer.  For 16 rows of 28672 x
// 8192 in 4 bits: loads of a panel for every wave's own A 79 us, rows kept and
// panels streamed 42, scales left as loaded until their step 30, a barrier for
// four panels and the next block's words ahead 27 on one card, 31 on
// others (with zero points 31 to 34, 3.6 to 4.0 TB/s).  What is left over the 24
// us of a copy is the start of the stream, the meeting of the sums and 36 VALU
// instructions a KiB of codes.
//
// The constant parts of the 4-bit sums (the two brackets of w4.hpp that do not
// depend on the column) are computed once for each chunk when the fragments
// arrive, by MFMAs against constant operands, and kept in LDS; the first enters
// as the initial accumulator.
#pragma once

#include "w4.hpp"

namespace tg {

// Waits for this wave's LDS accesses only, then for the other waves.
__device__ __forceinline__ void lds_barrier()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// A matrix of 4-bit weights of `panels` panels from panel `first` on; the byte
// counts are what buffer loads are checked against.
struct W4Source {
    const void *words, *scales, *zeros;
    int word_bytes, scale_bytes, zero_bytes;
    float per_chunk;                                   // groups a chunk
    int chunks, groups, scale_f32;

    __device__ __forceinline__ W4Source(const W4View& v, int first, int panels)
        : words(v.words + (int64_t)first * v.chunks * 64),
          scales(static_cast<const char*>(v.scales) + (int64_t)first * v.groups * (v.scale_f32 ? 64 : 32)),
          zeros(v.zeros ? v.zeros + (int64_t)first * v.groups * 16 : nullptr),
          word_bytes(bytes((int64_t)(panels - first) * v.chunks * 1024)),
          scale_bytes(bytes((int64_t)(panels - first) * v.groups * (v.scale_f32 ? 64 : 32))),
          zero_bytes(v.zeros ? bytes((int64_t)(panels - first) * v.groups * 16) : 0),
          per_chunk(128.0f / (float)v.group), chunks(v.chunks), groups(v.groups), scale_f32(v.scale_f32)
    {
    }

private:
    static __device__ __forceinline__ int bytes(int64_t n)
    {
        return (int)(n < kMaxRecords ? n : kMaxRecords);
    }
};

// MT: tiles of 16 rows; NT: matrices that share the rows (their panels advance
// together); NA: A is the sum of NA bf16; W: waves; CW: chunks a wave; GS: MFMA
// steps of 32 k between two scales (4 for groups of 128 and more, else group / 32).
// HALF: KiB of LDS for the sums of the panels between two barriers (held twice).
template <bool W4F, bool ZERO, int MT, int NT, int NA, int W, int CW, int GS, int HALF>
struct PanelStream {
    static constexpr int SC = W4F ? 4 / GS : 1;
    static constexpr int GL = (CW * SC + 3) / 4;                               // loads of four scales each
    // panels between two barriers: as many as HALF KiB of LDS hold, four at most
    static constexpr int R0 = HALF / (W * MT * NT), R = R0 < 1 ? 1 : R0 > 4 ? 4 : R0;
    static constexpr int RED = 2 * R * W * MT * NT * 64;                       // f32x4 of LDS
    static constexpr int MID = W4F ? W * CW * SC * MT * 4 * (ZERO ? 2 : 1) : 1;

    struct Words {
        u32x4_t w[NT][CW][W4F ? 1 : 4];
        unsigned s[NT][GL];                            // lane (i, column): the dword that holds scale i, as loaded
        unsigned char z[NT][ZERO ? GL : 1];            // its zero point
    };
    struct Rows {
        u32x4_t a[CW][MT][NA][4];
    };

    f32x4_t* red;
    f32x4_t* mid;                                      // this wave's part
    int lane, wave, turn;
    unsigned up, keep;                                 // a scale's bits within its dword: (dword << up) & keep
    CodeConsts code;

    __device__ __forceinline__ PanelStream(f32x4_t* r, f32x4_t* m, int scale_f32)
        : red(r), lane(threadIdx.x & 63), wave(__builtin_amdgcn_readfirstlane(threadIdx.x >> 6)), turn(0),
          up(scale_f32 || (lane & 1) ? 0 : 16), keep(scale_f32 ? ~0u : 0xFFFF0000u)
    {
        mid = m + (W4F ? wave * (MID / W) : 0);
    }

    // The wave's chunks c0 .. c0 + CW - 1 of the source's panel `index`, for
    // matrix j of the step.  What lies past the chunks, the groups or, with
    // `some` false, all of it, gets an offset out of the buffers' ranges: read
    // as zero, without a fetch.  One load brings four scales of the column, one
    // to each quarter of the wave.
    __device__ __forceinline__ void load_w4(Words& b, int j, const W4Source& v, int index, int c0, bool some) const
    {
        const __amdgpu_buffer_rsrc_t rw = wave_rsrc(v.words, v.word_bytes);
        const __amdgpu_buffer_rsrc_t rs = wave_rsrc(v.scales, v.scale_bytes);
        const __amdgpu_buffer_rsrc_t rz = wave_rsrc(v.zeros, v.zero_bytes);
#pragma unroll
        for (int i = 0; i < CW; ++i) {
            const int at = some && c0 + i < v.chunks ? (index * v.chunks + c0 + i) * 1024 : kOOB;
            b.w[j][i][0] = load16_stream(rw, (int)((unsigned)at + (unsigned)(lane * 16)));
        }
#pragma unroll
        for (int l = 0; l < GL; ++l) {
            const int i = CW * SC == 1 ? 0 : 4 * l + (lane >> 4);
            // groups of whole chunks by a product: off by 2^-23 of a number that is half a chunk from any border
            const int g = GS == 4 ? (int)(((float)(c0 + i) + 0.5f) * v.per_chunk) : c0 * SC + i;
            const bool in = some && g < v.groups;
            const int at = (index * v.groups + g) * 16 + (lane & 15);
            b.s[j][l] = load4(rs, in ? (v.scale_f32 ? at * 4 : at / 2 * 4) : kOOB);
            if constexpr (ZERO)
                b.z[j][l] = __builtin_amdgcn_raw_buffer_load_b8(rz, in ? at : kOOB, 0, 0);
        }
    }

    // The same of a bf16 matrix stored [N][K].  VEC: K a multiple of 8, rows on
    // 16 bytes; otherwise a skipped panel repeats itself and a ragged last
    // chunk is read element by element.
    template <bool VEC>
    __device__ __forceinline__ void load_bf16(Words& b, int j, const unsigned short* m, int N, int K, int panel, int c0,
                                              bool some) const
    {
        const int l16 = lane & 15, rows = min(16, N - panel * 16);
        const unsigned short* base = m + (int64_t)panel * 16 * K;
        if constexpr (VEC) {
            const __amdgpu_buffer_rsrc_t r = wave_rsrc(base, some ? (int64_t)rows * K * 2 : 0);
#pragma unroll
            for (int i = 0; i < CW; ++i)
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    const int k = (c0 + i) * 128 + 32 * t + 8 * (lane >> 4);
                    b.w[j][i][t] = load16(r, k < K ? (l16 * K + k) * 2 : kOOB);
                }
        } else {
#pragma unroll
            for (int i = 0; i < CW; ++i) {
                if (c0 + i < (K + 127) / 128)
                    load_chunk(b.w[j][i], base + (int64_t)min(l16, rows - 1) * K, c0 + i, lane >> 4, K);
                else
#pragma unroll
                    for (int t = 0; t < 4; ++t)
                        b.w[j][i][t] = splat4(0);
            }
        }
    }

    // The wave's fragments of row tile m: `off` bytes to the lane's row of K bf16
    // in r, kOOB if it has none.
    __device__ __forceinline__ void load_rows(Rows& x, int m, __amdgpu_buffer_rsrc_t r, int off, int K, int c0) const
    {
#pragma unroll
        for (int i = 0; i < CW; ++i)
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const int k = (c0 + i) * 128 + 32 * t + 8 * (lane >> 4);
                x.a[i][m][0][t] = load16(r, off != kOOB && k < K ? off + k * 2 : kOOB);
            }
    }
    // Of a row that starts anywhere, with any K (NULL: none).
    __device__ __forceinline__ void load_rows(Rows& x, int m, const unsigned short* row, int K, int c0) const
    {
#pragma unroll
        for (int i = 0; i < CW; ++i) {
#pragma unroll
            for (int t = 0; t < 4; ++t)
                x.a[i][m][0][t] = splat4(0);
            if (row && c0 + i < (K + 127) / 128)
                load_chunk(x.a[i][m][0], row, c0 + i, lane >> 4, K);
        }
    }
    // Of a row of K fp32 (NA = 3): as stored, for settle to part.
    __device__ __forceinline__ void load_floats(Rows& x, int m, __amdgpu_buffer_rsrc_t r, int off, int K, int c0) const
    {
#pragma unroll
        for (int i = 0; i < CW; ++i)
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const int k = (c0 + i) * 128 + 32 * t + 8 * (lane >> 4);
                const int at = off != kOOB && k < K ? off + k * 4 : kOOB;
                x.a[i][m][0][t] = load16(r, at);
                x.a[i][m][1][t] = load16(r, at == kOOB ? kOOB : at + 16);
            }
    }

    // Parts eight fp32, two fragments as loaded, into three fragments of bf16
    // whose sum they are: each takes the upper half, the sign and eight bits of
    // mantissa, of what the ones before leave, and 24 bits are three times eight
    // (but for what lies under 2^-133).  An infinity is its own first part and
    // leaves nothing.
    static __device__ __forceinline__ void part(u32x4_t (&a)[NA][4], int t)
    {
        const u32x4_t in[2] = {a[0][t], a[1][t]};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            unsigned v[2] = {in[e >> 1][e % 2 * 2], in[e >> 1][e % 2 * 2 + 1]};
#pragma unroll
            for (int n = 0; n < 3; ++n) {
                a[n][t][e] = __builtin_amdgcn_perm(v[1], v[0], 0x07060302u);
#pragma unroll
                for (int q = 0; q < 2 && n < 2; ++q) {
                    const float x = __uint_as_float(v[q]);
                    const float rest = x - __uint_as_float(v[q] & 0xFFFF0000u);
                    v[q] = n > 0 || __builtin_isfinite(x) ? __float_as_uint(rest) : 0u;
                }
            }
        }
    }

    // Makes loaded rows ready: parts fp32, computes the constant sums.
    __device__ __forceinline__ void settle(Rows& x)
    {
        if constexpr (NA == 3) {
#pragma unroll
            for (int i = 0; i < CW; ++i)
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int t = 0; t < 4; ++t)
                        part(x.a[i][m], t);
        }
        if constexpr (W4F) {
            const f32x4_t none = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < CW; ++i)
#pragma unroll
                for (int q = 0; q < SC; ++q)
#pragma unroll
                    for (int m = 0; m < MT; ++m) {
                        f32x4_t c = none, s = none;
#pragma unroll
                        for (int t = q * GS; t < (q + 1) * GS; ++t)
#pragma unroll
                            for (int n = 0; n < NA; ++n) {
                                c = mfma_bf16(x.a[i][m][n][t], splat4(kCentre), c);
                                if constexpr (ZERO)
                                    s = mfma_bf16(x.a[i][m][n][t], splat4(kOnes), s);
                            }
                        // the same in every column: lanes 0, 16, 32, 48 have all rows
                        const int at = ((i * SC + q) * MT + m) * 4 + (lane >> 4);
                        if ((lane & 15) == 0) {
                            mid[at] = c;
                            if constexpr (ZERO)
                                mid[CW * SC * MT * 4 + at] = s;
                        }
                    }
            // read back by this wave alone
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
            __builtin_amdgcn_wave_barrier();
            __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
        }
    }

    __device__ __forceinline__ void multiply(f32x4_t (&total)[MT][NT], const Rows& x, const Words& b) const
    {
        if constexpr (W4F) {
            // scales and shifts, still with the quarter that loaded them
            float scale[NT][GL], shift[NT][GL];
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int l = 0; l < GL; ++l) {
                    scale[j][l] = __uint_as_float((b.s[j][l] << up) & keep);
                    shift[j][l] = ZERO ? 8.0f - (float)b.z[j][ZERO ? l : 0] : 0.0f;
                }
            auto from = [&](float v, int i) {
                if constexpr (CW * SC == 1)
                    return v;
                return __int_as_float(
                    __builtin_amdgcn_ds_bpermute(4 * (16 * (i & 3) + (lane & 15)), __float_as_int(v)));
            };
#pragma unroll
            for (int i = 0; i < CW; ++i) {
                f32x4_t acc[MT][NT];
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    const int q = i * SC + t / GS;
                    if (t % GS == 0) {
#pragma unroll
                        for (int m = 0; m < MT; ++m) {
                            const f32x4_t c = mid[(q * MT + m) * 4 + (lane >> 4)];
#pragma unroll
                            for (int j = 0; j < NT; ++j)
                                acc[m][j] = c;
                        }
                    }
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        const u32x4_t w = w4_expand(b.w[j][i][0][t], code);
#pragma unroll
                        for (int m = 0; m < MT; ++m)
#pragma unroll
                            for (int n = 0; n < NA; ++n)
                                acc[m][j] = mfma_bf16(x.a[i][m][n][t], w, acc[m][j]);
                    }
                    if (t % GS == GS - 1) {
                        float sc[NT], d[NT];
#pragma unroll
                        for (int j = 0; j < NT; ++j) {
                            sc[j] = from(scale[j][q / 4], q);
                            d[j] = ZERO ? from(shift[j][q / 4], q) : 0.0f;
                        }
#pragma unroll
                        for (int m = 0; m < MT; ++m) {
                            f32x4_t s = {0.f, 0.f, 0.f, 0.f};
                            if constexpr (ZERO)
                                s = mid[CW * SC * MT * 4 + (q * MT + m) * 4 + (lane >> 4)];
#pragma unroll
                            for (int j = 0; j < NT; ++j)
#pragma unroll
                                for (int r = 0; r < 4; ++r)
                                    total[m][j][r] =
                                        fmaf(sc[j], ZERO ? fmaf(d[j], s[r], acc[m][j][r]) : acc[m][j][r], total[m][j][r]);
                        }
                    }
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < CW; ++i)
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int m = 0; m < MT; ++m)
#pragma unroll
                        for (int n = 0; n < NA; ++n)
#pragma unroll
                            for (int j = 0; j < NT; ++j)
                                total[m][j] = mfma_bf16(x.a[i][m][n][t], b.w[j][i][t], total[m][j]);
        }
    }

    __device__ __forceinline__ void clear(f32x4_t (&total)[MT][NT]) const
    {
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int j = 0; j < NT; ++j)
                total[m][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    }

    // The wave's sums of panel `index` to LDS.  After every R panels, and the
    // last, a barrier; then the waves share out the tiles and pass the sums over
    // all waves to done(index, m, sums).
    template <class Done>
    __device__ __forceinline__ void meet(int index, int n, const f32x4_t (&total)[MT][NT], const Done& done)
    {
        f32x4_t* half = red + (turn & 1) * (RED / 2);
        f32x4_t* r = half + index % R * (W * MT * NT * 64);
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int j = 0; j < NT; ++j)
                r[((m * NT + j) * W + wave) * 64 + lane] = total[m][j];
        if (index % R != R - 1 && index != n - 1)
            return;
        lds_barrier();
        const int first = index / R * R;
        for (int t = wave; t < (index - first + 1) * MT; t += W) {
            f32x4_t sum[NT];
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const f32x4_t* from = half + (t * NT + j) * W * 64 + lane;
                sum[j] = from[0];
#pragma unroll
                for (int q = 1; q < W; ++q)
                    sum[j] += from[q * 64];
            }
            done(first + t / MT, t % MT, sum);
        }
        ++turn;
    }

    // Panels 0 .. n - 1 of the workgroup, in each of `blocks` blocks of the
    // reduction (both the same for all its waves): load(block, index, words,
    // some) fills the wave's chunks and rows(block, rows, some) its fragments,
    // or skip them if !some; done(block, index, m, sums) as in meet.  The words
    // of the next D - 1 steps are on their way, across the change of blocks
    // too.  No other branch goes round a load, and nothing is computed from a
    // loaded value before its step: where two paths meet, or where a value is
    // first used, the wait for it would come before the younger loads are out.
    // (Scales shifted into place as they were loaded: 42 us instead of 30 for
    // 16 x 28672 x 8192.)
    template <int D, class RowsOf, class Load, class Done>
    __device__ __forceinline__ void run(int blocks, int n, const RowsOf& rows, const Load& load, const Done& done)
    {
        static_assert(D >= 2 && D <= 4, "steps");
        Words b[D];
        Rows x;
        int block = 0, index = 0, ahead_block = 0, ahead = 0;
        auto fetch = [&](Words& to) {
            load(ahead_block, ahead, to, ahead_block < blocks);
            if (++ahead == n) {
                ahead = 0;
                ++ahead_block;
            }
        };
#pragma unroll
        for (int d = 0; d < D - 1; ++d)
            fetch(b[d]);
        rows(0, x, true);
        settle(x);
        auto one = [&](int d) {
            fetch(b[(d + D - 1) % D]);
            f32x4_t total[MT][NT];
            clear(total);
            multiply(total, x, b[d]);
            meet(index, n, total, [&](int i, int m, f32x4_t (&sum)[NT]) { done(block, i, m, sum); });
            if (++index < n)
                return true;
            index = 0;
            if (++block == blocks)
                return false;
            rows(block, x, true);
            settle(x);
            return true;
        };
        if constexpr (D == 2)
            while (one(0) && one(1)) {
            }
        else if constexpr (D == 3)
            while (one(0) && one(1) && one(2)) {
            }
        else
            while (one(0) && one(1) && one(2) && one(3)) {
            }
    }

    // The same for a single panel and many blocks: the next block's rows are on
    // their way with its words, and the sums meet once, at the end.
    template <class RowsOf, class Load, class Done>
    __device__ __forceinline__ void run_one(int blocks, const RowsOf& rows, const Load& load, const Done& done)
    {
        Words b[2];
        Rows x[2];
        f32x4_t total[MT][NT];
        clear(total);
        int block = 0;
        load(0, 0, b[0], true);
        rows(0, x[0], true);
        auto one = [&](const Words& now, Words& next, Rows& mine, Rows& after) {
            const bool more = block + 1 < blocks;
            load(block + 1, 0, next, more);
            rows(block + 1, after, more);
            settle(mine);
            multiply(total, mine, now);
            ++block;
            return more;
        };
        while (one(b[0], b[1], x[0], x[1]) && one(b[1], b[0], x[1], x[0])) {
        }
        meet(0, 1, total, [&](int, int m, f32x4_t (&sum)[NT]) { done(0, 0, m, sum); });
    }
};

// The lane number, computed anew: what is derived from it is not kept in
// registers across the loop that the caller sits in.
__device__ __forceinline__ int fresh(int lane)
{
    __asm__ __volatile__("" : "+v"(lane));
    return lane;
}

}  // namespace tg
