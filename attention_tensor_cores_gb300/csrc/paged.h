// Host-side helpers shared by the paged key/value cache's translation units.
#pragma once
#include <initializer_list>

#include "internal.h"

namespace atc_gb300 {

inline bool misaligned(const void* p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0; }

// Checks of a cache descriptor that every entry point makes.
inline int check_cache(const fmha_kv_cache* c, const char* who)
{
    const auto refuse = [&](int code, const char* what) { return set_error(code, std::string(who) + what); };
    if (!c || !c->k || !c->v) return refuse(FMHA_ERR_INVALID, ": NULL cache or cache pointer");
    if (c->num_pages < 1 || c->page_size < 1 || c->Hkv < 1)
        return refuse(FMHA_ERR_INVALID, ": cache needs num_pages, page_size and Hkv >= 1");
    if (static_cast<long long>(c->num_pages) * c->page_size >= (1LL << 31))
        return refuse(FMHA_ERR_UNSUPPORTED, ": cache of 2^31 tokens or more");
    if (c->D != 64 && c->D != 128) return refuse(FMHA_ERR_UNSUPPORTED, ": cache D must be 64 or 128");
    if (misaligned(c->k, 16) || misaligned(c->v, 16)) return refuse(FMHA_ERR_INVALID, ": cache pools must be 16-byte aligned");
    for (const int64_t x : {c->page_stride, c->head_stride, c->token_stride})
        if (x < c->D || x % 8 != 0 || x >= (1LL << 38))
            return refuse(FMHA_ERR_INVALID, ": cache strides must be multiples of 8 elements, at least D and below 2^38");
    return FMHA_OK;
}

}  // namespace atc_gb300
