// Attention over a paged key/value cache (fmha_fwd_paged): the decode kernel of decode_kernel.cuh with
// its key and value tiles gathered page by page.
//
//   o = softmax(scale q K^T) V over keys j < n_b, K and V row j of request b at
//   pool[table[b][j / page]][kv-head][j % page]
//
// A 128-key tile is filled by TMA boxes of the largest power of two of keys that divides both the page
// and the tile; the tensor maps take any strides of pages, heads and keys, and offsets never pass through
// 32-bit arithmetic.  A box of 2^i >= 8 keys is a whole number of 128-byte-swizzle atoms of 8 keys x 64
// features.  At D = 128 the map has five dimensions (feature of 64, key of 8, half of the features, run of
// 8 keys over all pages, head), so that one box brings whole 256-byte keys: half the boxes.
//
// Bound: HBM (every key and value row read once) where there are keys enough, else latency: about 4 us from
// launch to the first S (lengths, split, page, K), a tile each 0.5 to 1 us, and 1 us of epilogue, 3 to 5 with a
// merge.  B64 Hq32 Hkv8 D128, up to 32768 keys in pages of 16: 611 us, 7.0 TB/s = 1.03 of the measured copy
// bandwidth (reads only); B8 Hq32 Hkv32 4096 keys: 82 us, 6.5 TB/s = 0.96 (84.7 a call live); B1 Hq32 Hkv8 500
// keys: 8.1 us.
#include <cuda_runtime.h>

#include "paged_run.cuh"

namespace atc_gb300 {
namespace {

struct PagedWs {
    size_t prefix_off, ctr_off, lse_off, o_off, stage_off, amax_off, total;
};

// The kernel merges split units itself, except for single-pass NVFP4, whose rows a combine kernel encodes (as in
// the dense decode), and for more SMs than it has slots for a unit's partials.  It finds the work split itself,
// except for very large batches, and where the combine kernel, which takes it from global memory, is to see it.
bool needs_combine(bool encode, int nsm) { return encode || nsm > kMaxFixSlots; }
bool needs_prefix(int B, bool encode, int nsm) { return needs_combine(encode, nsm) || B > kInlineB; }

PagedWs paged_ws(int B, int Hq, int Sq, const fmha_kv_cache* c, const fmha_opts* o)
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

template <int D, bool CAUSAL>
auto kernel_for(int G) -> decltype(&decode_kernel<D, CAUSAL, 1, true>)
{
    switch (decode_columns(G)) {
        case 1: return decode_kernel<D, CAUSAL, 1, true>;
        case 4: return decode_kernel<D, CAUSAL, 4, true>;
        case 8: return decode_kernel<D, CAUSAL, 8, true>;
        default: return decode_kernel<D, CAUSAL, 16, true>;
    }
}

template <int D, bool CAUSAL>
int run_paged(const PagedArgs& a, bool split, const PagedWs& w, uint8_t* base, cudaStream_t st)
{
    using C = DecodeCfg<D>;
    const int nsm = num_sms();
    if (nsm <= 0) return set_error(FMHA_ERR_CUDA, "cannot query the SM count");
    const Shape s = paged_shape(a.B, a.Hq, a.Sq, a.c);
    CUtensorMap maps[3];
    DecodeParams p;
    const int rc = paged_setup<D>(a, s, maps, p);
    if (rc) return rc;
    p.split = split ? 1 : 0;
    p.fixup = split && !needs_combine(a.nv_sg != nullptr, nsm) ? 1 : 0;
    p.prefix = split && needs_prefix(a.B, a.nv_sg != nullptr, nsm) ? reinterpret_cast<const int32_t*>(base + w.prefix_off) : nullptr;
    p.o_stage = a.o_stage;
    p.amax_bits = a.amax_bits;
    p.nv_sg = a.nv_sg;
    p.nv_codes = a.nv_codes;
    p.nv_scales = a.nv_scales;
    p.nv_ts = a.nv_ts;
    p.part_lse = split ? reinterpret_cast<float*>(base + w.lse_off) : nullptr;
    p.part_o = split ? reinterpret_cast<float*>(base + w.o_off) : nullptr;
    p.unit_ctr = split ? reinterpret_cast<unsigned long long*>(base + w.ctr_off) : nullptr;
    p.gen = next_call_tag();

    // one CTA per SM, or fewer when even full tables have fewer key tiles (whole units: fewer units)
    const long long tiles = split ? static_cast<long long>(s.U) * ((p.cap + kTileKV - 1) / kTileKV) : s.U;
    const unsigned grid = static_cast<unsigned>(tiles < nsm ? tiles : nsm);
    p.ctas = static_cast<int>(grid);
    if (p.prefix) {
        FMHA_CHECK_CUDA(launch_pdl(tile_prefix_kernel<true>, dim3(1), dim3(1024), 0, st, p, const_cast<int32_t*>(p.prefix)));
        count_launch();
    }
    const auto kernel = kernel_for<D, CAUSAL>(s.G);
    const int smem = C::smem_bytes(decode_columns(s.G), true);
    FMHA_CHECK_CUDA(set_smem_limit_once(reinterpret_cast<const void*>(kernel), smem));
    timing_mark_begin(st);
    const cudaError_t e = launch_pdl(kernel, dim3(grid), dim3(decode_threads<true>()), static_cast<size_t>(smem),
                                     st, maps[0], maps[1], maps[2], p);
    timing_mark_end(st);
    FMHA_CHECK_CUDA(e);
    count_launch();
    if (split && !p.fixup) {
        FMHA_CHECK_CUDA(launch_pdl(combine_kernel<true>, dim3(static_cast<unsigned>(s.U * s.G)), dim3(static_cast<unsigned>(D)), 0,
                                   st, p, static_cast<int>(grid)));
        count_launch();
    }
    return FMHA_OK;
}

int check_paged(const fmha_kv_cache* c, int B, int Hq, int Sq, int max_pages, const fmha_opts* o)
{
    const char* who = "fmha_fwd_paged";
    if (B < 0 || Hq <= 0 || Sq < 0 || max_pages < 1 || Hq % c->Hkv != 0)
        return set_error(FMHA_ERR_INVALID, std::string(who) + ": need B >= 0, Sq >= 0, max_pages >= 1, Hq > 0 a multiple of Hkv");
    const int rc = check_tiles(c, who);
    if (rc) return rc;
    const long long cap = static_cast<long long>(max_pages) * c->page_size;
    const long long rows = static_cast<long long>(B) * Hq * Sq;
    const long long units = static_cast<long long>(B) * c->Hkv * ((static_cast<long long>(Hq / c->Hkv) * Sq + kN - 1) / kN);
    if (cap > (1LL << 31) - 256 || rows >= (1LL << 31) || units * ((cap + kTileKV - 1) / kTileKV) >= (1LL << 31))
        return set_error(FMHA_ERR_UNSUPPORTED, std::string(who) + ": max_pages * page_size, the rows or the key tiles pass 2^31");
    if (o) {
        if (o->out_kind < FMHA_OUT_BF16 || o->out_kind > FMHA_OUT_NVFP4 || o->num_splits < 0)
            return set_error(FMHA_ERR_INVALID, std::string(who) + ": bad out_kind or num_splits");
        if (o->seqlens_k) return set_error(FMHA_ERR_INVALID, std::string(who) + ": opts.seqlens_k must be NULL (seqlens is an argument)");
    }
    return FMHA_OK;
}

}  // namespace
}  // namespace atc_gb300

using namespace atc_gb300;

extern "C" size_t fmha_paged_workspace_size(int B, int Hq, int Sq, const fmha_kv_cache* cache, const fmha_opts* opts)
{
    if (!cache || cache->Hkv < 1 || B < 0 || Hq <= 0 || Sq < 0 || Hq % cache->Hkv || (cache->D != 64 && cache->D != 128) ||
        static_cast<long long>(B) * Hq * Sq >= (1LL << 31))
        return 0;
    return paged_ws(B, Hq, Sq, cache, opts).total;
}

extern "C" int fmha_fwd_paged(const void* q, const fmha_kv_cache* cache, const int32_t* block_table, int max_pages,
                              const int32_t* seqlens, void* out, float* lse, int B, int Hq, int Sq, float scale,
                              fmha_stream_t stream, const fmha_opts* opts)
{
    int rc = check_cache(cache, "fmha_fwd_paged");
    if (rc) return rc;
    const bool empty = B == 0 || Sq == 0;
    if (!empty && (!q || !block_table || !seqlens || !out)) return set_error(FMHA_ERR_INVALID, "fmha_fwd_paged: NULL q/block_table/seqlens/out");
    if (!(scale > 0.f) || !(scale < INFINITY))
        return set_error(FMHA_ERR_INVALID, "fmha_fwd_paged: scale must be a positive finite number");
    rc = check_paged(cache, B, Hq, Sq, max_pages, opts);
    if (rc) return rc;
    if (misaligned(q, 16) || misaligned(out, 16) || misaligned(lse, 4) || misaligned(block_table, 4) || misaligned(seqlens, 4))
        return set_error(FMHA_ERR_INVALID, "fmha_fwd_paged: q/out 16-byte, lse/block_table/seqlens 4-byte aligned");
    const int out_kind = opts ? opts->out_kind : FMHA_OUT_BF16;
    const bool nvfp4 = out_kind == FMHA_OUT_NVFP4;
    if (nvfp4 && !empty) {
        if (!opts->out_scales || !opts->out_tensor_scale)
            return set_error(FMHA_ERR_INVALID, "fmha_fwd_paged: NVFP4 output needs out_scales and out_tensor_scale");
        if (misaligned(opts->out_f32, 16) || misaligned(opts->nvfp4_scale_in, 4) || misaligned(opts->out_amax, 4))
            return set_error(FMHA_ERR_INVALID, "fmha_fwd_paged: out_f32 16-byte, nvfp4_scale_in and out_amax 4-byte aligned");
    }
    void* ws = opts ? opts->workspace : nullptr;
    if (misaligned(ws, 256)) return set_error(FMHA_ERR_INVALID, "fmha_fwd_paged: workspace must be 256-byte aligned");
    if (!device_status_ptr()) return set_error(FMHA_ERR_CUDA, "no CUDA device");
    // split over every SM when there is a workspace to split in, as fmha_fwd_ex
    fmha_opts o = opts ? *opts : fmha_opts{};
    if (!ws && o.num_splits == 0) o.num_splits = 1;
    const PagedWs w = paged_ws(B, Hq, Sq, cache, &o);
    if (w.total > 0 && (!ws || o.workspace_bytes < w.total))
        return set_error(FMHA_ERR_WORKSPACE, "fmha_fwd_paged: workspace missing or smaller than fmha_paged_workspace_size()");
    const int64_t n = static_cast<int64_t>(B) * Hq * Sq * cache->D;
    if (n == 0) return FMHA_OK;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    uint8_t* base = static_cast<uint8_t*>(ws);

    PagedArgs a{};
    a.q = q;
    a.c = cache;
    a.table = block_table;
    a.max_pages = max_pages;
    a.seqlens = seqlens;
    a.out = out;
    a.lse = lse;
    a.B = B;
    a.Hq = Hq;
    a.Sq = Sq;
    a.scale = scale;
    a.out_kind = out_kind;
    const bool two_pass = nvfp4 && !o.nvfp4_scale_in;
    if (nvfp4) {
        a.o_stage = o.out_f32 ? o.out_f32 : (two_pass ? reinterpret_cast<float*>(base + w.stage_off) : nullptr);
        a.amax_bits = o.out_amax ? reinterpret_cast<unsigned*>(o.out_amax)
                                 : (two_pass ? reinterpret_cast<unsigned*>(base + w.amax_off) : nullptr);
        if (a.amax_bits) FMHA_CHECK_CUDA(cudaMemsetAsync(a.amax_bits, 0, sizeof(unsigned), st));
        if (!two_pass) {
            a.nv_sg = o.nvfp4_scale_in;
            a.nv_codes = static_cast<uint8_t*>(out);
            a.nv_scales = o.out_scales;
            a.nv_ts = o.out_tensor_scale;
        }
    }
    const bool split = o.num_splits != 1;
    const bool causal = o.causal && Sq > 1;   // one query sees every key either way
    if (cache->D == 64)
        rc = causal ? run_paged<64, true>(a, split, w, base, st) : run_paged<64, false>(a, split, w, base, st);
    else
        rc = causal ? run_paged<128, true>(a, split, w, base, st) : run_paged<128, false>(a, split, w, base, st);
    if (rc || !two_pass) return rc;
    return launch_nvfp4(a.o_stage, static_cast<uint8_t*>(out), o.out_scales, o.out_tensor_scale, a.amax_bits, n, true, st);
}
