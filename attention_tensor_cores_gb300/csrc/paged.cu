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
