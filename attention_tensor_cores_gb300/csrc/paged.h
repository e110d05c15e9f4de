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

// D = 128: runs of 8 keys from one page to the next
inline int64_t page_groups(const fmha_kv_cache* c) { return c->num_pages > 1 ? c->page_stride / (8 * c->token_stride) : c->page_size / 8; }

inline int make_pool_map(CUtensorMap* map, const void* pool, const fmha_kv_cache* c, int box)
{
    if (c->D == 128) {
        const uint64_t dims[5] = {64, 8, 2, static_cast<uint64_t>((c->num_pages - 1) * page_groups(c) + c->page_size / 8),
                                  static_cast<uint64_t>(c->Hkv)};
        const uint64_t strides[4] = {static_cast<uint64_t>(c->token_stride) * 2, 128, static_cast<uint64_t>(c->token_stride) * 16,
                                     static_cast<uint64_t>(c->head_stride) * 2};
        const uint32_t boxes[5] = {64, 8, 2, static_cast<uint32_t>(box / 8), 1};
        return make_tmap_bf16(map, pool, 5, dims, strides, boxes);
    }
    const uint64_t dims[4] = {static_cast<uint64_t>(c->D), static_cast<uint64_t>(c->page_size), static_cast<uint64_t>(c->Hkv),
                              static_cast<uint64_t>(c->num_pages)};
    const uint64_t strides[3] = {static_cast<uint64_t>(c->token_stride) * 2, static_cast<uint64_t>(c->head_stride) * 2,
                                 static_cast<uint64_t>(c->page_stride) * 2};
    const uint32_t boxes[4] = {64, static_cast<uint32_t>(box), 1, 1};
    return make_tmap_bf16(map, pool, 4, dims, strides, boxes);
}

// Keys of a TMA box: the largest power of two up to a tile of 128 that divides the page
inline int page_box(const fmha_kv_cache* c)
{
    int box = 128;
    while (c->page_size % box) box >>= 1;
    return box;
}

// What the tensor maps of an attention over pages need
inline int check_tiles(const fmha_kv_cache* c, const char* who)
{
    if (c->page_size % 8 != 0) return set_error(FMHA_ERR_UNSUPPORTED, std::string(who) + ": page_size must be a multiple of 8");
    if (c->D == 128 && c->num_pages > 1 &&
        (c->page_stride % (8 * c->token_stride) != 0 || page_groups(c) < c->page_size / 8 || page_groups(c) * (c->num_pages + 1LL) >= (1LL << 31)))
        return set_error(FMHA_ERR_UNSUPPORTED, std::string(who) + ": with D = 128, page_stride must be a multiple of 8 * token_stride that "
                                                                  "holds a page, and the pool less than 2^31 runs of 8 tokens");
    return FMHA_OK;
}

}  // namespace atc_gb300
