// Host-side helpers shared by the paged key/value cache's translation units.
#pragma once
#include "internal.h"

namespace atc_gb300 {

// Status word value that the paged-cache kernels leave for device data out of bounds
constexpr int kDevBadPage = 7;

inline bool misaligned(const void* p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0; }

// Checks of a cache descriptor that every entry point makes.
inline int check_cache(const fmha_kv_cache* c, const char* who)
{
    const std::string w(who);
    if (!c || !c->k || !c->v) return set_error(FMHA_ERR_INVALID, w + ": NULL cache or cache pointer");
    if (c->num_pages < 1 || c->page_size < 1 || c->Hkv < 1)
        return set_error(FMHA_ERR_INVALID, w + ": cache needs num_pages, page_size and Hkv >= 1");
    if (c->D != 64 && c->D != 128) return set_error(FMHA_ERR_UNSUPPORTED, w + ": cache D must be 64 or 128");
    if (misaligned(c->k, 16) || misaligned(c->v, 16)) return set_error(FMHA_ERR_INVALID, w + ": cache pools must be 16-byte aligned");
    const int64_t st[3] = {c->page_stride, c->head_stride, c->token_stride};
    for (int64_t x : st)
        if (x < c->D || x % 8 != 0 || x >= (1LL << 38))
            return set_error(FMHA_ERR_INVALID, w + ": cache strides must be multiples of 8 elements, at least D and below 2^38");
    return FMHA_OK;
}

}  // namespace atc_gb300
