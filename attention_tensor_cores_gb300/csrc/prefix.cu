// Attention of requests that share their first pages (fmha_fwd_prefix): the call, its workspace, and the merge of the partials
// that prefix_kernel.cuh leaves.
#include <cuda_runtime.h>

#include "paged_run.cuh"
#include "prefix.h"
#include "prefix_split.cuh"

namespace atc_gb300 {
namespace {

struct MergeParams {
    int rows, Hkv, R, nb;
    int shares;                // warps of a row: 1, 2, 4 or 8
    int G, chunks;             // of the decode kernel's units
    int weigh;
    const int4* plan;
    const int2* own;
    const float *common_o, *common_lse;   // partials of the groups' common keys
    const float *own_o, *own_lse;         // and of the requests' own: [U + SMs][16]
    void* out;                 // BF16 or F32, or NULL
    int out_f32;
    float* lse;
    float* o_stage;            // FP32 copy for NVFP4, else NULL
    unsigned* amax_bits;
};

// Merges the partials of a row: the pieces of its group's common keys and of its own.  Bound by latency: the plan, then LSEs and
// the first eight partials together, then eight partials at a time.  Where there are few rows, up to eight warps share theirs
// (16 requests of Hq32 Hkv8 D128 behind 8192 common keys, about 30 partials a row: 26.3 us a call from a graph, 29.4 with a warp
// per row); twice the warps made 64 requests behind 2048 keys 29.4 us instead of 26.3.
template <int D>
__global__ void __launch_bounds__(256, 3) prefix_merge_kernel(const __grid_constant__ MergeParams p)
{
    constexpr int V = D / 32;   // features of a lane
    griddep_launch_dependents();
    griddep_wait();
    __shared__ float part[8][D], part_m[8], part_l[8];
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, share = warp % p.shares, row = (blockIdx.x * 8 + warp) / p.shares;
    if (row >= p.rows) return;   // the last block's, warps of whole rows
    const int unit = row / p.R, rr = row - unit * p.R, b = unit / p.Hkv, h = unit - b * p.Hkv;
    const int4 head = p.plan[0], g = p.plan[1 + b];   // g: place, tiles, requests and first one of the group
    const int2 o = p.own[b];
    // the CTAs [c, c + n) of a line have pieces of its unit of nt tiles at place s; a lane looks at a cut
    const auto find = [&](const Line& line, int s, int nt, UnitCost u, int& c, int& n) {
        const int at_s = static_cast<int>(static_cast<float>(s) * (static_cast<float>(line.P) / static_cast<float>(line.T)));
        for (int i = max(min(at_s, line.P) - 1, 0);; i += 32) {   // a cut that is not behind s, although the quotient is rounded
            const int t = tile_at(line.cut(min(i + lane, line.P)) - s, nt, u);
            const unsigned before = __ballot_sync(0xffffffffu, t <= 0), behind = __ballot_sync(0xffffffffu, t >= nt);
            if (before) c = i + 31 - __clz(before);
            if (behind) {
                n = i + __ffs(behind) - 1 - c;
                return;
            }
        }
    };
    // partial i of n1 + n2: first those of the group's common keys (of a pair of row tiles with one tile two a piece, `second` rows
    // apart), then the request's own
    int c1 = 0, n1 = 0, second = 0, c2 = 0, n2 = 0;
    long long first1 = 0, first2 = 0;
    if (g.y > 0) {
        Line line;
        line.T = head.x;
        line.P = head.y & (kByTiles - 1);
        const UnitCost u = head.y & kByTiles ? UnitCost{1, 0, Cost<D>::common(g.z > p.nb).least} : Cost<D>::common(g.z > p.nb);
        const int pairs = row_pairs(g.z, p.nb), mem = b - g.w, r = mem / (2 * p.nb), rows = min(2 * p.nb, g.z - r * 2 * p.nb) * p.R;
        find(line, g.x + (h * pairs + r) * u.of(g.y), g.y, u, c1, n1);
        second = rows > p.nb * p.R ? 0 : rows;
        n1 <<= second ? 1 : 0;
        first1 = 2 * static_cast<long long>(g.w * p.Hkv + h * g.z + r * 2 * p.nb) * p.R + (mem - r * 2 * p.nb) * p.R + rr;
    }
    if (o.y > 0) {
        Line line;
        line.T = head.z;
        line.P = head.w;
        const UnitCost u = p.weigh ? Cost<D>::own(p.R > 8) : UnitCost{};
        const int chunk = rr / p.G, i = h * p.chunks + chunk, units = p.Hkv * p.chunks;
        find(line, o.x + i * u.of(o.y), o.y, u, c2, n2);
        first2 = static_cast<long long>(b * units + i) * kN + rr - chunk * p.G;
    }
    if (p.out && n1 == 0 && n2 == 1) return;   // one piece was all of it and wrote the row (for all warps of the row)
    const auto load = [](float (&x)[V], const float* from) {
        if constexpr (V == 4) {
            const float4 y = __ldcg(reinterpret_cast<const float4*>(from));
            x[0] = y.x, x[1] = y.y, x[2] = y.z, x[3] = y.w;
        } else {
            const float2 y = __ldcg(reinterpret_cast<const float2*>(from));
            x[0] = y.x, x[1] = y.y;
        }
    };
    float m = -INFINITY, l = 0.f, acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.f;
    const int mine = (n1 + n2 - share + p.shares - 1) / p.shares;   // this warp's: every p.shares-th
    for (int i0 = 0; i0 < mine; i0 += 32) {   // a lane per partial
        const int i = (i0 + lane) * p.shares + share, n = min(mine - i0, 32);
        long long at = 0;
        const float *lse = p.common_lse, *src = p.common_o;
        if (i < n1) {
            at = first1 + static_cast<long long>(c1 + (second ? i >> 1 : i)) * (2 * kRows) + (second && (i & 1) ? second : 0);
        } else {
            at = first2 + static_cast<long long>(c2 + i - n1) * kN;
            lse = p.own_lse;
            src = p.own_o;
        }
        const float x = lane < n ? __ldcg(lse + at) : -INFINITY;
        src += at * D;
        // the first rows are on their way before it is known what they weigh
        constexpr int kAhead = 8;
        const auto row_of = [&](int k) {
            return reinterpret_cast<const float*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(src), k)) + lane * V;
        };
        float v[kAhead][V];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const float* from = row_of(k);
            if (k < n) load(v[k], from);
        }
        const float top = fmax_nan(m, redux_max_nan(x));
        if (top == -INFINITY) continue;   // no visible key so far
        const float keep = m == -INFINITY ? 0.f : __expf(m - top), w = lane < n ? __expf(x - top) : 0.f;
        m = top;
        l = l * keep + warp_sum(w);
#pragma unroll
        for (int v = 0; v < V; ++v) acc[v] *= keep;
        const auto add = [&](const float (&x)[V], float wk) {
#pragma unroll
            for (int i = 0; i < V; ++i) acc[i] = fmaf(wk, x[i], acc[i]);
        };
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const float wk = __shfl_sync(0xffffffffu, w, k);
            if (k < n) add(v[k], wk);
        }
#pragma unroll 8
        for (int k = kAhead; k < n; ++k) {
            float x[V];
            load(x, row_of(k));
            add(x, __shfl_sync(0xffffffffu, w, k));
        }
    }
    if (p.shares > 1) {
#pragma unroll
        for (int v = 0; v < V; ++v) part[warp][lane * V + v] = acc[v];
        if (lane == 0) {
            part_m[warp] = m;
            part_l[warp] = l;
        }
        named_bar_sync(1 + warp / p.shares, 32 * p.shares);   // the row's warps
        if (share) return;
        float top = m;
        for (int w = 1; w < p.shares; ++w) top = fmax_nan(top, part_m[warp + w]);
        const float keep = m == -INFINITY ? 0.f : __expf(m - top);
        l *= keep;
#pragma unroll
        for (int v = 0; v < V; ++v) acc[v] *= keep;
        for (int w = 1; w < p.shares; ++w) {
            if (part_m[warp + w] == -INFINITY) continue;   // nothing visible there
            const float x = __expf(part_m[warp + w] - top);
            l = fmaf(x, part_l[warp + w], l);
#pragma unroll
            for (int v = 0; v < V; ++v) acc[v] = fmaf(x, part[warp + w][lane * V + v], acc[v]);
        }
        m = top;
    }
    const bool none = l == 0.f;
    const float inv = none ? 0.f : 1.f / l;
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        acc[i] = none ? 0.f : acc[i] * inv;
        amax = fmaxf(amax, fabsf(acc[i]));
    }
    const size_t at = static_cast<size_t>(row) * D + lane * V;
    if (p.o_stage) {
        if constexpr (V == 4) *reinterpret_cast<float4*>(p.o_stage + at) = make_float4(acc[0], acc[1], acc[2], acc[3]);
        else *reinterpret_cast<float2*>(p.o_stage + at) = make_float2(acc[0], acc[1]);
    }
    if (p.out && p.out_f32) {
        float* dst = static_cast<float*>(p.out) + at;
        if constexpr (V == 4) *reinterpret_cast<float4*>(dst) = make_float4(acc[0], acc[1], acc[2], acc[3]);
        else *reinterpret_cast<float2*>(dst) = make_float2(acc[0], acc[1]);
    } else if (p.out) {
        uint16_t* dst = static_cast<uint16_t*>(p.out) + at;
        if constexpr (V == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(acc[0], acc[1]), pack_bf16x2(acc[2], acc[3]));
        else *reinterpret_cast<uint32_t*>(dst) = pack_bf16x2(acc[0], acc[1]);
    }
    if (lane == 0 && p.lse) p.lse[row] = none ? -INFINITY : m + __logf(l);
    if (p.amax_bits) {
        amax = warp_max(amax);
        if (lane == 0 && amax > 0.f) atomicMax(p.amax_bits, __float_as_uint(amax));
    }
}

struct PrefixWs {
    size_t plan_off, own_off, pre_off, common_lse_off, common_o_off, own_lse_off, own_o_off, stage_off, amax_off, total;
};

// With so many key tiles at most, all requests' tables full, every request is read by itself.  The plan, a cold softmax
// and the merge cost about 20 us; a tile that another request has just brought to L2 costs the paged attention 4 to 5 ns.
// Hkv8 D128, shared against one by one: 4 requests behind 8192 keys (2240 tiles) 24.3 and 20.9 us, 8 of them (4416) 25.5 and
// 28.8; 8 groups of 4 behind up to 2000 keys (4608) 28.1 and 20.7, 4 behind 4096 (4480) 32.5 and 28.2; one group of 16 behind 8192
// (8800) 26.1 and 47.4.  No number of tiles tells these apart: 6000 sends the 8 requests of 4416 tiles the slower way by 3 us, 4400
// would send the groups of 4 the slower way by 4 to 7.
// The lengths are on the device, so what counts here is the room in the table.  A wide one takes short requests the longer way:
// 4 requests of 1000 keys 19.6 us with room for 131072 tokens, 11.9 with a table of their own size; 32 of 300 keys, no
// two of a group, 16.2 and 9.6.
constexpr long long kFewTiles = 6000;
// Requests with more rows are not shared; the paged attention takes them in chunks
constexpr int kMaxSharedRows = 64;
bool shareable(int Hq, int Sq, const fmha_kv_cache* c) { return static_cast<long long>(Hq / c->Hkv) * Sq <= kMaxSharedRows; }

PrefixWs prefix_ws(int B, int Hq, int Sq, const fmha_kv_cache* c, const fmha_opts* o)
{
    const auto al = [](size_t x) { return (x + 255) & ~size_t(255); };
    PrefixWs w{};
    const size_t rows = static_cast<size_t>(B) * Hq * Sq;
    if (rows == 0) return w;
    const size_t nsm = num_sms() > 0 ? num_sms() : 256;   // sized for the largest plausible SM count
    const size_t common = 2 * rows + nsm * 2 * kRows, own = (static_cast<size_t>(paged_shape(B, Hq, Sq, c).U) + nsm) * kN;
    size_t off = 0;
    const auto take = [&](size_t& at, size_t bytes) {
        at = off;
        off += al(bytes);
    };
    take(w.plan_off, (1 + static_cast<size_t>(B)) * sizeof(int4));
    take(w.own_off, static_cast<size_t>(B) * sizeof(int2));
    take(w.pre_off, (static_cast<size_t>(B) + 1) * 4);
    take(w.common_lse_off, common * 4);
    take(w.common_o_off, common * c->D * 4);
    take(w.own_lse_off, own * 4);
    take(w.own_o_off, own * c->D * 4);
    const bool nvfp4 = o && o->out_kind == FMHA_OUT_NVFP4;
    take(w.stage_off, nvfp4 && !o->out_f32 ? rows * c->D * 4 : 0);
    take(w.amax_off, nvfp4 ? 4 : 0);
    w.total = off;
    return w;
}

int check_prefix(const fmha_kv_cache* c, int B, int Hq, int Sq, int N, int max_pages, const fmha_opts* o)
{
    const std::string who = "fmha_fwd_prefix";
    if (B < 0 || Hq <= 0 || Sq < 0 || N < (B > 0 ? 1 : 0) || max_pages < 1 || Hq % c->Hkv != 0)
        return set_error(FMHA_ERR_INVALID, who + ": need B >= 0, Sq >= 0, N >= 1, max_pages >= 1, Hq > 0 a multiple of Hkv");
    const int rc = check_tiles(c, who.c_str());
    if (rc) return rc;
    const long long cap = static_cast<long long>(max_pages) * c->page_size, rows = static_cast<long long>(B) * Hq * Sq;
    if (N > kMaxGroups) return set_error(FMHA_ERR_UNSUPPORTED, who + ": more than 8192 groups");
    if (cap > (1LL << 31) - 256 || rows >= (1LL << 29) || B > (1 << 24))
        return set_error(FMHA_ERR_UNSUPPORTED, who + ": max_pages * page_size past 2^31, 2^29 rows or 2^24 requests");
    const long long units = static_cast<long long>(B) * c->Hkv * ((static_cast<long long>(Hq / c->Hkv) * Sq + kN - 1) / kN);
    if (units * ((cap + kTileKV - 1) / kTileKV) >= (1LL << 31)) return set_error(FMHA_ERR_UNSUPPORTED, who + ": 2^31 key tiles or more");
    if (o) {
        if (o->out_kind < FMHA_OUT_BF16 || o->out_kind > FMHA_OUT_NVFP4 || o->num_splits < 0)
            return set_error(FMHA_ERR_INVALID, who + ": bad out_kind or num_splits");
        if (o->seqlens_k) return set_error(FMHA_ERR_INVALID, who + ": opts.seqlens_k must be NULL (seqlens is an argument)");
        if (o->num_splits == 1) return set_error(FMHA_ERR_UNSUPPORTED, who + ": num_splits = 1 (common keys are a part of each request's)");
    }
    return FMHA_OK;
}

template <int D>
int run_prefix(const PrefixParams& p, MergeParams& m, const PagedArgs& a, cudaStream_t st)
{
    const int rc = launch_prefix<D>(p, a, const_cast<float*>(m.own_o), const_cast<float*>(m.own_lse), st);
    if (rc) return rc;
    m.shares = 1;
    while (m.shares < 8 && static_cast<long long>(m.rows) * m.shares * 2 <= 16LL * num_sms()) m.shares *= 2;   // half of the warps that fit
    const int per = 8 / m.shares, blocks = (m.rows + per - 1) / per, each = (blocks + num_sms() - 1) / num_sms();
    // Blocks that start early would fill the SMs whose CTA ends first.  Shared memory that they do not use leaves as many on each SM
    // as make them reach over all (16 requests behind 8192 keys, calls back to back: 29.3 us without, 26.3 with).
    constexpr int kSpread = 200 * 1024;
    FMHA_CHECK_CUDA(set_smem_limit_once(reinterpret_cast<const void*>(prefix_merge_kernel<D>), kSpread));
    FMHA_CHECK_CUDA(launch_pdl(prefix_merge_kernel<D>, dim3(static_cast<unsigned>(blocks)), dim3(256), static_cast<size_t>(each < 3 ? kSpread / each : 0), st, m));
    count_launch();
    return FMHA_OK;
}

}  // namespace
}  // namespace atc_gb300

using namespace atc_gb300;

extern "C" size_t fmha_prefix_workspace_size(int B, int Hq, int Sq, const fmha_kv_cache* cache, const fmha_opts* opts)
{
    if (!cache || cache->Hkv < 1 || B < 0 || Hq <= 0 || Sq < 0 || Hq % cache->Hkv || (cache->D != 64 && cache->D != 128) ||
        static_cast<long long>(B) * Hq * Sq >= (1LL << 29))
        return 0;
    const fmha_opts o = opts ? *opts : fmha_opts{};
    const size_t paged = fmha_paged_workspace_size(B, Hq, Sq, cache, &o);
    const size_t own = shareable(Hq, Sq, cache) ? prefix_ws(B, Hq, Sq, cache, &o).total : 0;
    return own > paged ? own : paged;
}

extern "C" int fmha_fwd_prefix(const void* q, const fmha_kv_cache* cache, const int32_t* block_table, int max_pages, const int32_t* seqlens,
                               const int32_t* cu_groups, const int32_t* prefix_lens, int N, void* out, float* lse, int B, int Hq, int Sq,
                               float scale, fmha_stream_t stream, const fmha_opts* opts)
{
    int rc = check_cache(cache, "fmha_fwd_prefix");
    if (rc) return rc;
    const bool empty = B == 0 || Sq == 0;
    if (!empty && (!q || !block_table || !seqlens || !out || !cu_groups || !prefix_lens))
        return set_error(FMHA_ERR_INVALID, "fmha_fwd_prefix: NULL q/block_table/seqlens/cu_groups/prefix_lens/out");
    if (!(scale > 0.f) || !(scale < INFINITY)) return set_error(FMHA_ERR_INVALID, "fmha_fwd_prefix: scale must be a positive finite number");
    rc = check_prefix(cache, B, Hq, Sq, N, max_pages, opts);
    if (rc) return rc;
    if (misaligned(q, 16) || misaligned(out, 16) || misaligned(lse, 4) || misaligned(block_table, 4) || misaligned(seqlens, 4) ||
        misaligned(cu_groups, 4) || misaligned(prefix_lens, 4))
        return set_error(FMHA_ERR_INVALID, "fmha_fwd_prefix: q/out 16-byte, the other arrays 4-byte aligned");
    const fmha_opts o = opts ? *opts : fmha_opts{};
    const bool nvfp4 = o.out_kind == FMHA_OUT_NVFP4;
    if (nvfp4 && !empty) {
        if (!o.out_scales || !o.out_tensor_scale) return set_error(FMHA_ERR_INVALID, "fmha_fwd_prefix: NVFP4 output needs out_scales and out_tensor_scale");
        if (misaligned(o.out_f32, 16) || misaligned(o.nvfp4_scale_in, 4) || misaligned(o.out_amax, 4))
            return set_error(FMHA_ERR_INVALID, "fmha_fwd_prefix: out_f32 16-byte, nvfp4_scale_in and out_amax 4-byte aligned");
    }
    if (misaligned(o.workspace, 256)) return set_error(FMHA_ERR_INVALID, "fmha_fwd_prefix: workspace must be 256-byte aligned");
    if (!device_status_ptr()) return set_error(FMHA_ERR_CUDA, "no CUDA device");
    const size_t need = fmha_prefix_workspace_size(B, Hq, Sq, cache, &o);
    if (need > 0 && (!o.workspace || o.workspace_bytes < need))
        return set_error(FMHA_ERR_WORKSPACE, "fmha_fwd_prefix: workspace missing or smaller than fmha_prefix_workspace_size()");
    if (empty) return FMHA_OK;
    const Shape shape = paged_shape(B, Hq, Sq, cache);
    const long long most = static_cast<long long>(shape.U) * ((static_cast<long long>(max_pages) * cache->page_size + kTileKV - 1) / kTileKV);
    if (!shareable(Hq, Sq, cache) || most <= kFewTiles)
        return fmha_fwd_paged(q, cache, block_table, max_pages, seqlens, out, lse, B, Hq, Sq, scale, stream, &o);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const PrefixWs w = prefix_ws(B, Hq, Sq, cache, &o);
    uint8_t* base = static_cast<uint8_t*>(o.workspace);

    PrefixParams p{};
    p.B = B;
    p.Hkv = cache->Hkv;
    p.R = Hq / cache->Hkv * Sq;
    p.Sq = Sq;
    p.gr = Groups{cu_groups, prefix_lens, N, kRows / p.R, p.R, shape.chunks};
    p.causal = o.causal && Sq > 1;   // one query sees every key either way
    p.c = scale * kLog2e;
    p.seqlens = seqlens;
    p.table = block_table;
    p.max_pages = max_pages;
    p.num_pages = cache->num_pages;
    p.page = cache->page_size;
    p.by_page = FastDiv(static_cast<uint32_t>(p.page));
    p.box = page_box(cache);
    while ((1 << p.box_log2) < p.box) ++p.box_log2;
    p.groups = static_cast<int>(page_groups(cache));
    p.cap = max_pages * cache->page_size;
    p.part_o = reinterpret_cast<float*>(base + w.common_o_off);
    p.part_lse = reinterpret_cast<float*>(base + w.common_lse_off);
    p.plan = reinterpret_cast<int4*>(base + w.plan_off);
    p.rest_prefix = reinterpret_cast<int32_t*>(base + w.pre_off);
    p.own = reinterpret_cast<int2*>(base + w.own_off);
    p.rest_units = p.Hkv * shape.chunks;
    p.weigh = most < kMaxWeighed ? 1 : 0;
    p.status = device_status_ptr();
    p.limit = wait_limit();

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
    a.out_kind = o.out_kind;   // NVFP4: the decode kernel writes no output, only partials
    a.causal = p.causal;

    MergeParams m{};
    m.rows = B * Hq * Sq;
    m.Hkv = p.Hkv;
    m.R = p.R;
    m.nb = p.gr.nb;
    m.G = shape.G;
    m.chunks = shape.chunks;
    m.plan = p.plan;
    m.own = p.own;
    m.weigh = p.weigh;
    m.common_o = p.part_o;
    m.common_lse = p.part_lse;
    m.own_o = reinterpret_cast<float*>(base + w.own_o_off);
    m.own_lse = reinterpret_cast<float*>(base + w.own_lse_off);
    m.out = nvfp4 ? nullptr : out;
    m.out_f32 = o.out_kind == FMHA_OUT_F32 ? 1 : 0;
    m.lse = lse;
    if (nvfp4) {
        m.o_stage = o.out_f32 ? o.out_f32 : reinterpret_cast<float*>(base + w.stage_off);
        m.amax_bits = o.out_amax ? reinterpret_cast<unsigned*>(o.out_amax) : reinterpret_cast<unsigned*>(base + w.amax_off);
        FMHA_CHECK_CUDA(cudaMemsetAsync(m.amax_bits, 0, sizeof(unsigned), st));
    }
    rc = cache->D == 64 ? run_prefix<64>(p, m, a, st) : run_prefix<128>(p, m, a, st);
    if (rc || !nvfp4) return rc;
    return launch_nvfp4(m.o_stage, static_cast<uint8_t*>(out), o.out_scales, o.out_tensor_scale, m.amax_bits,
                        static_cast<int64_t>(m.rows) * cache->D, true, st, o.nvfp4_scale_in);
}
