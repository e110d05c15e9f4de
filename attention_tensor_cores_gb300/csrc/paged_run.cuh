// Launch of the paged decode kernel (decode_kernel.cuh): for the whole attention over pages (paged.cu), and for what
// is left of requests that share their first pages (paged_rest.cu).
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

// Requests of which a part is attended to elsewhere
struct PagedRest {
    const int32_t* prefix;   // device [B + 2], from the kernel that does so: tiles before each request's own, their number and the
                             // CTAs that they are split over
    float* part_o;           // [U + SMs][16][D]
    float* part_lse;         // [U + SMs][16]
};
int launch_paged_rest(const PagedArgs& a, const PagedRest& rest, cudaStream_t st);

namespace {

struct PagedWs {
    size_t prefix_off, ctr_off, lse_off, o_off, stage_off, amax_off, total;
};

// The kernel merges split units itself, except for single-pass NVFP4, whose rows a combine kernel encodes (as in
// the dense decode), and for more SMs than it has slots for a unit's partials.  It finds the work split itself,
// except for very large batches, and where the combine kernel, which takes it from global memory, is to see it.
inline bool needs_combine(bool encode, int nsm) { return encode || nsm > kMaxFixSlots; }
inline bool needs_prefix(int B, bool encode, int nsm) { return needs_combine(encode, nsm) || B > kInlineB; }

inline PagedWs paged_ws(int B, int Hq, int Sq, const fmha_kv_cache* c, const fmha_opts* o)
{
    auto al = [](size_t x) { return (x + 255) & ~size_t(255); };
    const Shape s = paged_shape(B, Hq, Sq, c);
    if (s.U == 0) return {};   // nothing to do, nothing to do it in
    const int nsm = num_sms() > 0 ? num_sms() : 256;   // sized for the largest plausible SM count
    const bool split = o && o->num_splits != 1;
    const size_t slots = split ? static_cast<size_t>(s.U) + nsm : 0;
    PagedWs w{};
    size_t off = 0;
    w.prefix_off = off;
    off += split && needs_prefix(B, o->nvfp4_scale_in != nullptr, nsm) ? al((static_cast<size_t>(B) + 2) * 4) : 0;
    w.ctr_off = off;
    off += split ? al(static_cast<size_t>(s.U) * 8) : 0;
    w.lse_off = off;
    off += al(slots * kN * 4);
    w.o_off = off;
    off += al(slots * kN * c->D * 4);
    const bool two_pass = o && o->out_kind == FMHA_OUT_NVFP4 && !o->nvfp4_scale_in;
    w.stage_off = off;
    off += two_pass && !o->out_f32 ? al(static_cast<size_t>(B) * Hq * Sq * c->D * 4) : 0;
    w.amax_off = off;
    off += two_pass ? 256 : 0;
    w.total = off;
    return w;
}

template <int D, bool CAUSAL, bool REST>
auto kernel_for(int G) -> decltype(&decode_kernel<D, CAUSAL, 1, true, REST>)
{
    switch (decode_columns(G)) {
        case 1: return decode_kernel<D, CAUSAL, 1, true, REST>;
        case 4: return decode_kernel<D, CAUSAL, 4, true, REST>;
        case 8: return decode_kernel<D, CAUSAL, 8, true, REST>;
        default: return decode_kernel<D, CAUSAL, 16, true, REST>;
    }
}

// CTAs of the decode kernel over U units of at most cap keys each that are split over n SMs: no more than paged_ctas
// gives work to
inline int rest_grid(int U, int cap, int n)
{
    const long long tiles = static_cast<long long>(U) * ((static_cast<long long>(cap) + kTileKV - 1) / kTileKV), most = tiles / kMinPiece > U ? tiles / kMinPiece : U;
    return static_cast<int>(most < n ? most : n);
}

// rest: what is left of requests whose first keys are attended to elsewhere (REST), else NULL
template <int D, bool CAUSAL, bool REST = false>
int run_paged(const PagedArgs& a, bool split, const PagedWs& w, uint8_t* base, cudaStream_t st, const PagedRest* rest = nullptr)
{
    using C = DecodeCfg<D>;
    const int nsm = num_sms();
    if (nsm <= 0) return set_error(FMHA_ERR_CUDA, "cannot query the SM count");
    const Shape s = paged_shape(a.B, a.Hq, a.Sq, a.c);
    const int rows = (a.Hq / a.c->Hkv) * a.Sq;

    CUtensorMap qmap, kmap, vmap;
    {
        const uint64_t dims[3] = {static_cast<uint64_t>(D), static_cast<uint64_t>(rows), static_cast<uint64_t>(a.B) * a.c->Hkv};
        const uint64_t strides[2] = {static_cast<uint64_t>(D) * 2, static_cast<uint64_t>(rows) * D * 2};
        const uint32_t box[3] = {64, static_cast<uint32_t>(kN), 1};
        const int rc = make_tmap_bf16(&qmap, a.q, 3, dims, strides, box);
        if (rc) return rc;
    }
    const int box = page_box(a.c);
    int rc = make_pool_map(&kmap, a.c->k, a.c, box);
    if (rc) return rc;
    rc = make_pool_map(&vmap, a.c->v, a.c, box);
    if (rc) return rc;

    DecodeParams p{};
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
    p.split = split ? 1 : 0;
    p.fixup = split && !needs_combine(a.nv_sg != nullptr, nsm) ? 1 : 0;
    p.prefix = split && needs_prefix(a.B, a.nv_sg != nullptr, nsm) ? reinterpret_cast<const int32_t*>(base + w.prefix_off) : nullptr;
    p.out = a.out_kind == FMHA_OUT_NVFP4 ? nullptr : a.out;
    p.out_f32 = a.out_kind == FMHA_OUT_F32 ? 1 : 0;
    p.lse = a.lse;
    p.o_stage = a.o_stage;
    p.amax_bits = a.amax_bits;
    p.nv_sg = a.nv_sg;
    p.nv_codes = a.nv_codes;
    p.nv_scales = a.nv_scales;
    p.nv_ts = a.nv_ts;
    p.part_lse = split ? reinterpret_cast<float*>(base + w.lse_off) : nullptr;
    p.part_o = split ? reinterpret_cast<float*>(base + w.o_off) : nullptr;
    p.unit_ctr = split ? reinterpret_cast<unsigned long long*>(base + w.ctr_off) : nullptr;
    if constexpr (REST) {
        p.fixup = 0;
        p.prefix = rest->prefix;
        p.part_lse = rest->part_lse;
        p.part_o = rest->part_o;
        p.unit_ctr = nullptr;
    }
    p.gen = next_call_tag();
    p.status = device_status_ptr();
    p.limit = wait_limit();

    // one CTA per SM, or fewer when even full tables have fewer key tiles (whole units: fewer units)
    const long long tiles = split ? static_cast<long long>(s.U) * ((p.cap + kTileKV - 1) / kTileKV) : s.U;
    const unsigned grid = static_cast<unsigned>(REST ? rest_grid(s.U, p.cap, nsm) : tiles < nsm ? tiles : nsm);
    p.ctas = static_cast<int>(grid);
    if (p.prefix && !REST) {
        FMHA_CHECK_CUDA(launch_pdl(tile_prefix_kernel<true>, dim3(1), dim3(1024), 0, st, p, const_cast<int32_t*>(p.prefix)));
        count_launch();
    }
    const auto kernel = kernel_for<D, CAUSAL, REST>(s.G);
    const int smem = C::smem_bytes(decode_columns(s.G), true);
    FMHA_CHECK_CUDA(set_smem_limit_once(reinterpret_cast<const void*>(kernel), smem));
    if (!REST) timing_mark_begin(st);
    const cudaError_t e = launch_pdl(kernel, dim3(grid), dim3(decode_threads<true>()), static_cast<size_t>(smem),
                                     st, qmap, kmap, vmap, p);
    if (!REST) timing_mark_end(st);
    FMHA_CHECK_CUDA(e);
    count_launch();
    if (split && !p.fixup && !REST) {
        FMHA_CHECK_CUDA(launch_pdl(combine_kernel<true>, dim3(static_cast<unsigned>(s.U * s.G)), dim3(static_cast<unsigned>(D)), 0,
                                   st, p, static_cast<int>(grid)));
        count_launch();
    }
    return FMHA_OK;
}

}  // namespace
}  // namespace atc_gb300
