// Argument checks shared by the entry points on 4-bit and expert weights.
#pragma once

#include <cstdint>

#include "runtime.hpp"
#include "w4.hpp"

namespace tg {

constexpr size_t kLdsBytes = 160 * 1024;       // of a workgroup on gfx950

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Compute units to share the work among: of the device description in force.
inline int64_t compute_units() { return current_desc().n_cu; }

// TG_OK, or the error (set) that a call reports for weight `name`.
int check_weight(const tg_weight* w, const char* name);

// The first matrix, with K rows, of a stack of 4-bit weights.
inline W4View view_w4(const tg_weight& w, int64_t K)
{
    W4View v{};
    v.group = w.group;
    v.scale_f32 = w.scale_dtype == TG_F32;
    v.chunks = (int)ceil_div(K, 128);
    v.groups = (int)ceil_div(K, w.group);
    v.words = static_cast<const u32x4_t*>(w.data);
    v.scales = w.scales;
    v.zeros = static_cast<const unsigned char*>(w.zeros);
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
