// Decode attention over dense keys and values: workspace layout and launches of the kernels in
// decode_kernel.cuh, and the allocation-free entry point.
#include <cuda_runtime.h>

#include <atomic>
#include <cstdio>

#include "decode_kernel.cuh"
#include "internal.h"

namespace atc_gb300 {

// ---- host side ------------------------------------------------------------------------------------
namespace {

struct DecodeWs {
    size_t prefix_off, ctr_off, lse_off, o_off, stage_off, total;
};

DecodeWs decode_ws_layout(const AttnArgs& a, bool split, int nsm)
{
    auto al = [](size_t x) { return (x + 255) & ~size_t(255); };
    const size_t U = static_cast<size_t>(a.B) * a.Hkv;
    const size_t slots = split ? U + nsm : 0;
    DecodeWs w{};
    size_t off = 0;
    w.prefix_off = off;
    off += (split && a.seqlens) ? al((U + 1) * 4) : 0;
    w.ctr_off = off;
    off += split ? al(U * 8) : 0;   // fixup arrival counters
    w.lse_off = off;
    off += al(slots * kN * 4);
    w.o_off = off;
    off += al(slots * kN * a.D * 4);
    w.stage_off = off;
    const bool stage = (a.out_kind == FMHA_OUT_NVFP4) && !a.out_f32 && !a.nv_sg;
    off += stage ? al(static_cast<size_t>(a.B) * a.Hq * a.Sq * a.D * 4) : 0;
    w.total = off;
    return w;
}

template <int D, bool CAUSAL>
auto kernel_for(int G) -> decltype(&decode_kernel<D, CAUSAL, 1>)
{
    switch (decode_columns(G)) {
        case 1: return decode_kernel<D, CAUSAL, 1>;
        case 4: return decode_kernel<D, CAUSAL, 4>;
        case 8: return decode_kernel<D, CAUSAL, 8>;
        default: return decode_kernel<D, CAUSAL, 16>;
    }
}

template <int D, bool CAUSAL>
int run_decode(const AttnArgs& a, bool split, void* ws, cudaStream_t st)
{
    using C = DecodeCfg<D>;
    const int nsm = num_sms();
    if (nsm <= 0) return set_error(FMHA_ERR_CUDA, "cannot query the SM count");
    const int U = a.B * a.Hkv;
    const int G = (a.Hq / a.Hkv) * a.Sq;
    const DecodeWs w = decode_ws_layout(a, split, nsm);
    uint8_t* base = static_cast<uint8_t*>(ws);

    CUtensorMap qmap, kmap, vmap;
    {
        const uint64_t dims[3] = {static_cast<uint64_t>(D), static_cast<uint64_t>(G), static_cast<uint64_t>(U)};
        const uint64_t strides[2] = {static_cast<uint64_t>(D) * 2, static_cast<uint64_t>(G) * D * 2};
        const uint32_t box[3] = {64, static_cast<uint32_t>(kN), 1};
        int rc = make_tmap_bf16(&qmap, a.q, 3, dims, strides, box);
        if (rc) return rc;
    }
    {
        const uint64_t dims[3] = {static_cast<uint64_t>(D), static_cast<uint64_t>(a.Skv), static_cast<uint64_t>(U)};
        const uint64_t strides[2] = {static_cast<uint64_t>(D) * 2, static_cast<uint64_t>(a.Skv) * D * 2};
        const uint32_t box[3] = {64, static_cast<uint32_t>(kTileKV), 1};
        int rc = make_tmap_bf16(&kmap, a.k, 3, dims, strides, box);
        if (rc) return rc;
        rc = make_tmap_bf16(&vmap, a.v, 3, dims, strides, box);
        if (rc) return rc;
    }

    DecodeParams p{};
    p.U = U;
    p.Hkv = a.Hkv;
    p.G = G;
    p.Skv = a.Skv;
    p.D = D;
    p.Sq = a.Sq > 0 ? a.Sq : 1;
    p.c = a.scale * kLog2e;
    p.seqlens = a.seqlens;
    p.tiles_uniform = (a.Skv + kTileKV - 1) / kTileKV;
    p.split = split ? 1 : 0;
    p.prefix = (split && a.seqlens) ? reinterpret_cast<const int32_t*>(base + w.prefix_off) : nullptr;
    const bool nvfp4 = a.out_kind == FMHA_OUT_NVFP4;
    p.out = nvfp4 ? nullptr : a.out;
    p.out_f32 = a.out_kind == FMHA_OUT_F32 ? 1 : 0;
    p.lse = a.lse;
    p.o_stage = nvfp4 ? (a.out_f32 ? a.out_f32 : (a.nv_sg ? nullptr : reinterpret_cast<float*>(base + w.stage_off))) : nullptr;
    p.amax_bits = nvfp4 ? reinterpret_cast<unsigned*>(a.amax_slot) : nullptr;
    p.nv_sg = a.nv_sg;
    p.nv_codes = a.nv_codes;
    p.nv_scales = a.nv_scales;
    p.nv_ts = a.nv_ts;
    p.part_lse = split ? reinterpret_cast<float*>(base + w.lse_off) : nullptr;
    p.part_o = split ? reinterpret_cast<float*>(base + w.o_off) : nullptr;
    // Split units are merged in the kernel by the CTA completing them (a unit's last partial lands
    // at the end of a CTA's range, so the merge costs a few microseconds of tail instead of the
    // combine launch).  Measured slower for ragged batches, which keep the combine kernel (it also
    // writes units without keys); single-pass NVFP4 keeps it too (one block per row encodes).
    p.fixup = (split && !a.nv_sg && !a.seqlens && nsm <= kMaxFixSlots) ? 1 : 0;
    p.unit_ctr = split ? reinterpret_cast<unsigned long long*>(base + w.ctr_off) : nullptr;
    p.gen = next_call_tag();
    p.status = device_status_ptr();
    p.limit = wait_limit();

    if (p.prefix) {
        FMHA_CHECK_CUDA(launch_pdl(tile_prefix_kernel<false>, dim3(1), dim3(1024), 0, st, p,
                                   const_cast<int32_t*>(p.prefix)));
        count_launch();
    }
    // The epilogue warpgroup takes each item's epilogue off the softmax warps when a unit has several
    // query columns (publishing a 16-column partial costs several tiles' streaming time); with one
    // column the epilogue is short and the six-warp kernel, whose softmax warps run it, measured faster.
    const auto kernel = kernel_for<D, CAUSAL>(G);
    const bool epi = G > 1;
    FMHA_CHECK_CUDA(set_smem_limit_once(reinterpret_cast<const void*>(kernel), C::kSmemBytes));
    // one CTA per SM, or one per key tile when a uniform-length problem has fewer tiles than SMs (a
    // small problem then launches only the CTAs that have work)
    int grid = split ? nsm : (U < nsm ? U : nsm);
    if (split && !p.prefix) {
        const long long tiles = static_cast<long long>(U) * p.tiles_uniform;
        if (tiles < grid) {
            grid = static_cast<int>(tiles);
        } else {
            // When the units divide evenly over at least 5/6 of the SMs, each CTA streams the same
            // number of whole units: no partial to publish or merge, and that many SMs still keep
            // HBM busy (B8 H32 Skv4096: 128 CTAs of two units 87.3 us, 152 CTAs of 53.9 tiles 88.6)
            for (int g = grid; 6 * g >= 5 * nsm; --g)
                if (U % g == 0) {
                    grid = g;
                    break;
                }
        }
    }
    if (grid > 0) {
        timing_mark_begin(st);
        const cudaError_t e = launch_pdl(kernel, dim3(static_cast<unsigned>(grid)),
                                         dim3(epi ? decode_threads<true>() : decode_threads<false>()), C::kSmemBytes, st, qmap,
                                         kmap, vmap, p);
        timing_mark_end(st);
        FMHA_CHECK_CUDA(e);
        count_launch();
    }
    if (split && !p.fixup && U * G > 0) {
        FMHA_CHECK_CUDA(launch_pdl(combine_kernel<false>, dim3(static_cast<unsigned>(U * G)), dim3(static_cast<unsigned>(D)), 0,
                                   st, p, grid));
        count_launch();
    }
    return FMHA_OK;
}

}  // namespace

size_t decode_workspace_bytes(const AttnArgs& a, int num_splits)
{
    const int nsm = num_sms() > 0 ? num_sms() : 256;   // sized for the largest plausible SM count
    const bool split = num_splits != 1;
    return decode_ws_layout(a, split, nsm).total;
}

int launch_decode(const AttnArgs& a, int num_splits, void* ws, size_t ws_bytes, cudaStream_t st)
{
    const bool split = num_splits != 1 && ws != nullptr;
    const int nsm = num_sms();
    const DecodeWs w = decode_ws_layout(a, split, nsm);
    if (w.total > 0 && (!ws || ws_bytes < w.total)) return set_error(FMHA_ERR_WORKSPACE, "decode: workspace too small");
    switch (a.D) {
        case 64: return a.causal ? run_decode<64, true>(a, split, ws, st) : run_decode<64, false>(a, split, ws, st);
        case 128: return a.causal ? run_decode<128, true>(a, split, ws, st) : run_decode<128, false>(a, split, ws, st);
        default: return set_error(FMHA_ERR_UNSUPPORTED, "decode path: D must be 64 or 128");
    }
}

}  // namespace atc_gb300

// ================================================================================================
// Split-KV decode without any device allocation by the caller or the library.
//
// Some callers cannot provide the workspace that fmha_fwd_ex's split-KV path needs: plug-ins and
// foreign-language bindings that are handed only tensor pointers and have no allocator to ask,
// and latency-critical loops that must not call cudaMalloc (it can synchronise the device and
// its latency is unbounded).  For them the split partials and the tile prefix live in the fixed
// array below, which every GPU that loads this library holds until the process exits.
//
// The array is shared by every call on a device and keeps the contents of the last call.  No
// part of it needs to start at zero: each byte a call reads (tile prefix, partial O and LSE) is
// written earlier in the same call.  Calls that overlap on the GPU (different streams, or
// different host threads, without ordering between them) race on it.
// ================================================================================================
static __device__ __align__(256) unsigned char g_fmha_decode_scratch[FMHA_NOALLOC_SCRATCH_BYTES];

namespace atc_gb300 {
namespace {

constexpr int kMaxScratchDevices = 64;
std::atomic<void*> g_decode_scratch_addr[kMaxScratchDevices];

// Device address of the scratch array on the current device, looked up once per device (with
// that device current) and cached.
int decode_scratch_address(void** out)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_error(e, "cudaGetDevice");
    if (dev < 0 || dev >= kMaxScratchDevices) return set_error(FMHA_ERR_UNSUPPORTED, "device index out of range");
    void* p = g_decode_scratch_addr[dev].load();
    if (!p) {
        e = cudaGetSymbolAddress(&p, g_fmha_decode_scratch);
        if (e != cudaSuccess) return cuda_error(e, "cudaGetSymbolAddress(decode scratch)");
        g_decode_scratch_addr[dev].store(p);
    }
    *out = p;
    return FMHA_OK;
}

}  // namespace
}  // namespace atc_gb300

extern "C" int fmha_fwd_decode_noalloc(const void* q, const void* k, const void* v, void* out, float* lse, int B,
                                       int Hq, int Hkv, int Sq, int Skv, int D, float scale,
                                       const int32_t* seqlens_k, fmha_stream_t stream)
{
    using namespace atc_gb300;
    if (!q || !k || !v || !out) return set_error(FMHA_ERR_INVALID, "fmha_fwd_decode_noalloc: NULL q/k/v/out");
    if (B < 0 || Hq <= 0 || Hkv <= 0 || Sq < 0 || Skv <= 0 || Hq % Hkv != 0)
        return set_error(FMHA_ERR_INVALID, "fmha_fwd_decode_noalloc: need B >= 0, Sq >= 0, Skv >= 1, Hq % Hkv == 0");
    if (D != 64 && D != 128) return set_error(FMHA_ERR_INVALID, "fmha_fwd_decode_noalloc: D must be 64 or 128");
    if (!(scale > 0.f) || !(scale < INFINITY))
        return set_error(FMHA_ERR_INVALID, "fmha_fwd_decode_noalloc: scale must be a positive finite number");
    if (static_cast<long long>(Hq / Hkv) * Sq > 16)
        return set_error(FMHA_ERR_INVALID, "fmha_fwd_decode_noalloc: at most 16 query rows per key/value head");
    auto mis = [](const void* p, uintptr_t m) { return (reinterpret_cast<uintptr_t>(p) & m) != 0; };
    if (mis(q, 15) || mis(k, 15) || mis(v, 15) || mis(out, 15) || mis(lse, 3) || mis(seqlens_k, 3))
        return set_error(FMHA_ERR_INVALID, "fmha_fwd_decode_noalloc: q/k/v/out 16-byte, lse/seqlens 4-byte aligned");
    if (static_cast<long long>(B) * Hkv * Skv >= (1LL << 31))
        return set_error(FMHA_ERR_UNSUPPORTED, "fmha_fwd_decode_noalloc: more than 2^31 key rows");
    if (static_cast<long long>(B) * Hq * Sq == 0) return FMHA_OK;
    if (!device_status_ptr()) return set_error(FMHA_ERR_CUDA, "no CUDA device");

    AttnArgs a{};
    a.q = q;
    a.k = k;
    a.v = v;
    a.out = out;
    a.lse = lse;
    a.B = B;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.Sq = Sq;
    a.Skv = Skv;
    a.D = D;
    a.scale = scale;
    a.seqlens = seqlens_k;
    a.out_kind = FMHA_OUT_BF16;
    const size_t need = decode_workspace_bytes(a, 0);
    if (need > FMHA_NOALLOC_SCRATCH_BYTES) {
        char msg[200];
        snprintf(msg, sizeof msg,
                 "fmha_fwd_decode_noalloc: this problem needs %zu bytes of split-KV scratch, the static area holds %zu "
                 "(B*Hkv and the SM count set the size)",
                 need, static_cast<size_t>(FMHA_NOALLOC_SCRATCH_BYTES));
        return set_error(FMHA_ERR_WORKSPACE, msg);
    }
    void* scratch = nullptr;
    int rc = decode_scratch_address(&scratch);
    if (rc) return rc;
    return launch_decode(a, 0, scratch, FMHA_NOALLOC_SCRATCH_BYTES, reinterpret_cast<cudaStream_t>(stream));
}

