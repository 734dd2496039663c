// Argument checks shared by the entry points on 4-bit and expert weights.
#pragma once

#include <cstdint>

#include "runtime.hpp"
#include "w4.hpp"

namespace tg {

constexpr size_t kLdsBytes = 160 * 1024;       // of a workgroup on gfx950
constexpr int kCus = 256;

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// TG_OK, or the error (set) for a K x N weight of `w`'s format.
int check_weight(const tg_weight* w, int64_t K, int64_t N, const char* name);

// The i-th K x N matrix of a stack of 4-bit weights.
inline W4View view_w4(const tg_weight& w, int64_t K, int64_t N, int64_t i)
{
    W4View v{};
    const int64_t panels = ceil_div(N, 16);
    v.group = w.group;
    v.scale_f32 = w.scale_dtype == TG_F32;
    v.chunks = (int)ceil_div(K, 128);
    v.groups = (int)ceil_div(K, w.group);
    v.words = static_cast<const u32x4_t*>(w.data) + i * panels * v.chunks * 64;
    const int64_t at = i * panels * v.groups * 16;
    v.scales = static_cast<const char*>(w.scales) + at * (v.scale_f32 ? 4 : 2);
    v.zeros = w.zeros ? static_cast<const unsigned char*>(w.zeros) + at : nullptr;
    return v;
}

// Panels of `chunks` KiB that a workgroup's 32-bit offsets reach.
inline int panels_in_reach(int chunks) { return (1 << 20) / chunks; }

inline int launched(const char* what)
{
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? TG_OK : set_hip_error(e, what);
}

}  // namespace tg
