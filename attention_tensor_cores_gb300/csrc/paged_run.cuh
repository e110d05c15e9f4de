// What the launches of the paged decode kernel (decode_kernel.cuh) have in common: of the whole attention over pages (paged.cu),
// and of what is left of requests that share their first pages (prefix_kernel.cuh).
#pragma once
#include "decode_kernel.cuh"
#include "paged.h"

namespace atc_gb300 {

struct PagedArgs {
    const void* q;
    const fmha_kv_cache* c;
    const int32_t* table;
    int max_pages;
    const int32_t* seqlens;
    void* out;
    float* lse;
    int B, Hq, Sq;
    float scale;
    int out_kind, causal;
    float* o_stage;        // NVFP4: where the FP32 O goes when the caller has given a place for it
    unsigned* amax_bits;
    const float* nv_sg;
    uint8_t *nv_codes, *nv_scales;
    float* nv_ts;
};

struct Shape {
    int G, chunks, U;   // rows of a unit, units per key/value head, units
};

inline Shape paged_shape(int B, int Hq, int Sq, const fmha_kv_cache* c)
{
    const int rows = (Hq / c->Hkv) * Sq;
    Shape s{};
    s.chunks = rows > 0 ? (rows + kN - 1) / kN : 1;
    s.G = rows > 0 ? (rows + s.chunks - 1) / s.chunks : 0;
    s.U = rows > 0 ? B * c->Hkv * s.chunks : 0;
    return s;
}

namespace {

// The tensor maps of Q, K and V and the parameters that do not depend on the split
template <int D>
int paged_setup(const PagedArgs& a, const Shape& s, CUtensorMap (&m)[3], DecodeParams& p)
{
    const int rows = (a.Hq / a.c->Hkv) * a.Sq;
    {
        const uint64_t dims[3] = {static_cast<uint64_t>(D), static_cast<uint64_t>(rows), static_cast<uint64_t>(a.B) * a.c->Hkv};
        const uint64_t strides[2] = {static_cast<uint64_t>(D) * 2, static_cast<uint64_t>(rows) * D * 2};
        const uint32_t box[3] = {64, static_cast<uint32_t>(kN), 1};
        const int rc = make_tmap_bf16(&m[0], a.q, 3, dims, strides, box);
        if (rc) return rc;
    }
    const int box = page_box(a.c);
    int rc = make_pool_map(&m[1], a.c->k, a.c, box);
    if (rc) return rc;
    rc = make_pool_map(&m[2], a.c->v, a.c, box);
    if (rc) return rc;

    p = DecodeParams{};
    p.U = s.U;
    p.Hkv = a.c->Hkv * s.chunks;
    p.G = s.G;
    p.chunks = s.chunks;
    p.Gtot = rows;
    p.D = D;
    p.Sq = a.Sq;
    p.c = a.scale * kLog2e;
    p.seqlens = a.seqlens;
    p.table = a.table;
    p.max_pages = a.max_pages;
    p.num_pages = a.c->num_pages;
    p.page = a.c->page_size;
    p.by_page = FastDiv(static_cast<uint32_t>(p.page));
    p.box = box;
    while ((1 << p.box_log2) < box) ++p.box_log2;
    p.groups = static_cast<int>(page_groups(a.c));
    p.cap = a.max_pages * a.c->page_size;
    p.Skv = p.cap;
    p.out = a.out_kind == FMHA_OUT_NVFP4 ? nullptr : a.out;
    p.out_f32 = a.out_kind == FMHA_OUT_F32 ? 1 : 0;
    p.lse = a.lse;
    p.status = device_status_ptr();
    p.limit = wait_limit();
    return FMHA_OK;
}

}  // namespace
}  // namespace atc_gb300
