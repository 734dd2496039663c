// The product of a few rows with panel after panel of streamed weights: the
// core of the 4-bit product and of the expert layers (storage and arithmetic of
// 4-bit weights: w4.hpp).
//
// A few rows use every weight once, so the weights' stream from HBM is the
// bound, and what decides is how many bytes are on their way at any time.  The
// reduction is therefore cut among the W waves of a workgroup: a wave keeps
// its rows' fragments of CW chunks (128 k each) in registers, for all panels
// that the workgroup works on, and a step is the CW chunks of the next panel,
// whose loads are all issued one step ahead.  In flight are CW KiB a wave in 4
// bits, four times that in bf16, and A is read once a workgroup rather than
// once a panel.  The waves' sums of a panel meet in LDS, in wave order, after one
// barrier that leaves the loads in flight; the buffer is doubled, and the wave
// that adds a tile up takes turns, so nobody waits for the adding.
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

// MT: tiles of 16 rows; NT: matrices that share the rows (their panels advance
// together); NA: A is the sum of NA bf16; W: waves; CW: chunks a wave; GS: MFMA
// steps of 32 k between two scales (4: groups of 128 and more, 1: smaller).
// HALF: KiB of LDS for the sums of the panels between two barriers (held twice).
template <bool W4F, bool ZERO, int MT, int NT, int NA, int W, int CW, int GS, int HALF>
struct PanelStream {
    static constexpr int SC = W4F ? 4 / GS : 1;
    // panels between two barriers: as many as HALF KiB of LDS hold, four at most
    static constexpr int R0 = HALF / (W * MT * NT), R = R0 < 1 ? 1 : R0 > 4 ? 4 : R0;
    static constexpr int RED = 2 * R * W * MT * NT * 64;                       // f32x4 of LDS
    static constexpr int MID = W4F ? W * CW * SC * MT * 4 * (ZERO ? 2 : 1) : 1;

    struct Words {
        u32x4_t w[NT][CW][W4F ? 1 : 4];
        unsigned s[NT][CW][SC];                        // the dword that holds the scale, as loaded
        unsigned char z[NT][CW][ZERO ? SC : 1];        // zero point
    };

    u32x4_t a[CW][MT][NA][4];
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

    // The wave's chunks c0 .. c0 + CW - 1 of panel `panel` of v, for matrix j of
    // the step.  What lies past the chunks, the groups or, with `some` false,
    // all of it, is out of the buffers' ranges: read as zero, without a fetch.
    __device__ __forceinline__ void load_w4(Words& b, int j, const W4View& v, int panel, int c0, bool some) const
    {
        const int l16 = lane & 15;
        const __amdgpu_buffer_rsrc_t rw =
            make_rsrc(v.words + (int64_t)panel * v.chunks * 64, some ? (int64_t)v.chunks * 1024 : 0);
        const int64_t per = (int64_t)panel * v.groups * 16;
        const int n = some ? v.groups * 16 : 0;
        const __amdgpu_buffer_rsrc_t rs =
            make_rsrc(static_cast<const char*>(v.scales) + per * (v.scale_f32 ? 4 : 2), n * (v.scale_f32 ? 4 : 2));
        const __amdgpu_buffer_rsrc_t rz = make_rsrc(v.zeros + (ZERO ? per : 0), n);
#pragma unroll
        for (int i = 0; i < CW; ++i) {
            b.w[j][i][0] = load16_stream(rw, (c0 + i) * 1024 + lane * 16);
#pragma unroll
            for (int q = 0; q < SC; ++q) {
                const int at = (int)((unsigned)((c0 + i) * 128 + 32 * GS * q) / (unsigned)v.group) * 16 + l16;
                b.s[j][i][q] = load4(rs, v.scale_f32 ? at * 4 : at / 2 * 4);
                if constexpr (ZERO)
                    b.z[j][i][q] = __builtin_amdgcn_raw_buffer_load_b8(rz, at, 0, 0);
            }
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
            const __amdgpu_buffer_rsrc_t r = make_rsrc(base, some ? (int64_t)rows * K * 2 : 0);
#pragma unroll
            for (int i = 0; i < CW; ++i)
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    const int k = (c0 + i) * 128 + 32 * t + 8 * (lane >> 4);
                    b.w[j][i][t] = load16_stream(r, k < K ? (l16 * K + k) * 2 : kOOB);
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

    // After the fragments are set: their constant sums.
    __device__ __forceinline__ void correct()
    {
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
                                c = mfma_bf16(a[i][m][n][t], splat4(kCentre), c);
                                if constexpr (ZERO)
                                    s = mfma_bf16(a[i][m][n][t], splat4(kOnes), s);
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

    __device__ __forceinline__ void multiply(f32x4_t (&total)[MT][NT], const Words& b) const
    {
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int j = 0; j < NT; ++j)
                total[m][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < CW; ++i) {
            if constexpr (W4F) {
                f32x4_t acc[MT][NT];
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    const int q = t / GS;
                    if (t % GS == 0) {
#pragma unroll
                        for (int m = 0; m < MT; ++m) {
                            const f32x4_t c = mid[((i * SC + q) * MT + m) * 4 + (lane >> 4)];
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
                                acc[m][j] = mfma_bf16(a[i][m][n][t], w, acc[m][j]);
                    }
                    if (t % GS == GS - 1) {
#pragma unroll
                        for (int m = 0; m < MT; ++m) {
                            f32x4_t s = {0.f, 0.f, 0.f, 0.f};
                            if constexpr (ZERO)
                                s = mid[CW * SC * MT * 4 + ((i * SC + q) * MT + m) * 4 + (lane >> 4)];
#pragma unroll
                            for (int j = 0; j < NT; ++j) {
                                const float scale = __uint_as_float((b.s[j][i][q] << up) & keep);
                                float d = 0.0f;
                                if constexpr (ZERO)
                                    d = 8.0f - (float)b.z[j][i][q];
#pragma unroll
                                for (int r = 0; r < 4; ++r)
                                    total[m][j][r] =
                                        fmaf(scale, ZERO ? fmaf(d, s[r], acc[m][j][r]) : acc[m][j][r], total[m][j][r]);
                            }
                        }
                    }
                }
            } else {
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int m = 0; m < MT; ++m)
#pragma unroll
                        for (int n = 0; n < NA; ++n)
#pragma unroll
                            for (int j = 0; j < NT; ++j)
                                total[m][j] = mfma_bf16(a[i][m][n][t], b.w[j][i][t], total[m][j]);
            }
        }
    }

    // One panel: the wave's sums to LDS.  After every R panels, and the last,
    // a barrier; then the waves share out the tiles and pass the sums over all
    // waves to done(index, m, sums).
    template <class Done>
    __device__ __forceinline__ void step(int index, int n, const Words& b, const Done& done)
    {
        f32x4_t total[MT][NT];
        multiply(total, b);
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
    // some) fills the wave's chunks, or skips them if !some; rows(block) sets
    // its fragments; done(block, index, m, sums) as in step.  The next step's
    // words are on their way across the change of blocks too.  No other branch
    // goes round a load, and nothing is computed from a loaded value before
    // its step: where two paths meet, or where a value is first used, the wait
    // for it would come before the younger loads are out.  (Scales shifted
    // into place as they were loaded: 42 us instead of 30 for 16 x 28672 x
    // 8192.)
    template <class Rows, class Load, class Done>
    __device__ __forceinline__ void run(int blocks, int n, const Rows& rows, const Load& load, const Done& done)
    {
        Words b[2];
        int block = 0, index = 0;
        load(0, 0, b[0], true);
        rows(0);
        correct();
        auto one = [&](const Words& now, Words& next) {
            const bool turns = index + 1 == n;
            const int nb = turns ? block + 1 : block, ni = turns ? 0 : index + 1;
            const bool more = nb < blocks;
            load(more ? nb : block, ni, next, more);
            step(index, n, now, [&](int i, int m, f32x4_t (&sum)[NT]) { done(block, i, m, sum); });
            if (more && turns) {
                rows(nb);
                correct();
            }
            block = nb;
            index = ni;
            return more;
        };
        while (one(b[0], b[1]) && one(b[1], b[0])) {
        }
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
