// Argument checks shared by the entry points on 8-bit matrices.
#pragma once

#include <cstdint>

#include "w4_host.hpp"

namespace tg {

constexpr int64_t kMaxSide = (int64_t)1 << 24;

// TG_OK, or the error (set) that a call reports for matrix `name`.
inline int check_f8(const tg_f8* m, const char* name, bool rows_only)
{
    if (!m || !m->codes || !m->scales)
        return set_error(TG_E_INVAL, std::string(name) + ": codes and scales must be given");
    if (m->block != 1 && (rows_only || m->block != 128))
        return set_error(TG_E_INVAL, std::string(name) + (rows_only ? ": block must be 1" : ": block must be 1 or 128"));
    if (((uintptr_t)m->codes & 15u) || ((uintptr_t)m->scales & 3u))
        return set_error(TG_E_INVAL, std::string(name) + ": codes must be 16-byte aligned, scales 4-byte");
    return TG_OK;
}

}  // namespace tg
