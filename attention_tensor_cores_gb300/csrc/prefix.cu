// Attention of requests that share their first pages (fmha_fwd_prefix): each group's common keys are read
// once for all its requests.
//
//   o_b = softmax(scale q_b K_b^T) V_b as in fmha_fwd_paged.  With the keys of request b in disjoint sets C_1, C_2, ..
//   and O_i, lse_i the attention over C_i alone:   lse = log sum_i exp(lse_i),   o_b = sum_i exp(lse_i - lse) O_i
//
// so a group's common keys, in whole tiles of 128, are a problem whose rows are the queries of all its requests
// (prefix_kernel), what is left of each request is a decode problem (paged_rest.cu), and a third kernel merges a row's
// partials.  Per key/value head a request has R = (Hq / Hkv) Sq rows.
//
// prefix_kernel:
//  * Row tiles.  S = Q K^T with M = 128 query rows: floor(128 / R) requests of a group.  A row is a thread's (Tensor
//    Memory lane), so maxima and sums need no other thread.
//  * A CTA has two softmax warpgroups ("sides"), each with its own S, P and O in Tensor Memory and its own running
//    maximum and sum.  With more than 128 rows in the group they take two row tiles, over the same key tiles; else the same rows
//    over every other key tile.  While one computes exponentials the tensor core runs the other's products.
//  * P goes to the tensor core as two BF16, the rounded weight (half a step, 2^-9) and what the rounding left, both over the
//    S that they come from (16 keys' scores become 8 columns of pairs of either), in an MMA each: P is good to 2^-17
//    as in fmha_fwd_paged, and the output's rounding is the only one that shows.
//  * Work split.  The key tiles of all problems (group, kv-head, pair of row tiles) are laid end to end and cut for the CTAs (as in
//    decode_kernel.cuh); each piece's normalised partials go to the workspace.  Lengths are on the device, so every CTA sums
//    the groups itself; one more CTA sums the requests and leaves their places for the two other kernels.
//  * Roles: warps 0-3 and 4-7 the sides, 8 K, 9 Q and V, 10 MMA (a warp for each side's products measured slower: 1.58 us a
//    tile of 128 rows and keys against 1.32), 11 finds the pieces and hands them to the others through a ring in shared
//    memory.  Every wait is bounded, as in decode_kernel.cuh.
#include <cuda_runtime.h>

#include "paged_run.cuh"

namespace atc_gb300 {
namespace {

constexpr int kRows = 128;          // query rows of a tile
constexpr int kItems = 4;           // slots of the item ring
constexpr int kItemReaders = 11;    // K, V and MMA warps, eight softmax warps
constexpr int kMaxGroups = 8192;
constexpr int kPrefixThreads = 384;
// registers: two softmax warpgroups and the control warpgroup, 2 * 208 + 88 = 504 of an SM quarter's 512
constexpr uint32_t kRegsSide = 208;
static_assert(128 * (2 * kRegsSide + kRegsCtl) <= kPrefixThreads * 168, "register split exceeds the launch allocation");
struct Groups {
    const int32_t* cu = nullptr;       // [n + 1] first request of each
    const int32_t* prefix = nullptr;   // [n] tokens in the same pages
    int n = 0;
    int nb = 0;                        // requests in a row tile of prefix.cu
};

// A group's keys are shared when that spares at least so many tiles of one key/value head: its rows' partials cost
// about as much.
constexpr int kMinShared = 4;

// Tiles of keys that the requests [b0, b1) of a group read together.  n0: keys of the first one, through whose row
// they are read.
__device__ __forceinline__ int shared_tiles(const Groups& gr, int b0, int b1, int prefix, int n0)
{
    const int members = b1 - b0;
    if (members < 2) return 0;
    const int tiles = min(max(prefix, 0), n0) / kTileKV, row_tiles = (members + gr.nb - 1) / gr.nb;
    return static_cast<long long>(members - row_tiles) * tiles < kMinShared ? 0 : tiles;
}

// last g < n with start[g] <= x (start non-decreasing, start[0] <= x)
__device__ __forceinline__ int group_of(const int* start, int n, int x)
{
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (start[mid] <= x) lo = mid; else hi = mid - 1;
    }
    return lo;
}

// The groups' first requests and shared tiles into shared memory (2 n + 1 ints), by the whole block.  keys(b): request b's
// keys.  Returns whether cu is a list of groups of B requests; if not, nothing is shared.
template <typename Keys>
__device__ __forceinline__ bool load_groups(const Groups& gr, int B, int* cu, int* tiles, Keys&& keys)
{
    bool bad = false;
    for (int g = threadIdx.x; g <= gr.n; g += blockDim.x) cu[g] = gr.cu[g];
    __syncthreads();
    for (int g = threadIdx.x; g <= gr.n; g += blockDim.x)
        bad = bad || cu[g] < 0 || cu[g] > B || (g > 0 ? cu[g] < cu[g - 1] : cu[g] != 0) || (g == gr.n && cu[g] != B);
    const bool grouped = !__syncthreads_or(bad);
    for (int g = threadIdx.x; g < gr.n; g += blockDim.x)
        tiles[g] = grouped && cu[g + 1] > cu[g] ? shared_tiles(gr, cu[g], cu[g + 1], gr.prefix[g], keys(cu[g])) : 0;
    __syncthreads();
    return grouped;
}

template <int D>
struct PrefixCfg {
    static constexpr int kAtoms = D / 64;
    static constexpr int kStagesK = D == 64 ? 4 : 2, kStagesV = D == 64 ? 5 : 3;   // V waits for the softmax, K does not
    static constexpr int kQBytes = kAtoms * kRows * 128;                          // a row tile
    static constexpr int kKVBytes = kAtoms * kTileKV * 128;
    static constexpr int kOffQ = 0;
    static constexpr int kOffK = kOffQ + 2 * kQBytes;
    static constexpr int kOffV = kOffK + kStagesK * kKVBytes;
    static constexpr int kSmemBytes = kOffV + kStagesV * kKVBytes + 1024;   // + alignment slack
    // Tensor Memory columns of a side: S (and P over it), O
    static constexpr uint32_t col_s(uint32_t i) { return i * 128; }
    static constexpr uint32_t col_o(uint32_t i) { return 256 + i * 128; }
};

struct PrefixParams {
    int B;               // requests
    Groups gr;
    int Hkv, R, Sq;      // rows of a request and key/value head; row r is query r % Sq
    int causal;
    float c;             // scale * log2(e)
    const int32_t* seqlens;
    const int32_t* table;
    int max_pages, num_pages, page;
    FastDiv by_page;
    int box, box_log2, groups;   // as in DecodeParams
    int cap;             // max_pages * page: lengths are clamped to it
    float* part_o;       // [rows][D] partials of common keys
    float* part_lse;
    // for the other two kernels
    int4* plan;          // [1 + B]: (tiles, CTAs) of the line; of each request its group's place on the line, tiles, requests and first one
    int32_t* rest_prefix;   // [B + 2]: tiles before each request's own, their number and the CTAs that they are split over
    int rest_units, rest_ctas;   // units of a request and CTAs of the decode kernel
    int* status;
    long long limit;
};

// A piece of a problem
struct PrefixItem {
    int t0, t1;      // tiles of keys (none: no more pieces)
    int trow, head;  // row of the block table: the group's first request
    int b0, rows;    // first request of the first row tile, and rows of both
    int prow;        // first row of the partials
};

__device__ __forceinline__ int keys_of(const PrefixParams& p, int b) { return min(max(p.seqlens[b], 0), p.cap); }

// pairs of row tiles of a group
__host__ __device__ __forceinline__ int row_pairs(int members, int nb) { return (members + 2 * nb - 1) / (2 * nb); }

// Sum over the lanes before this one, and the lane's own
__device__ __forceinline__ int warp_scan_inc(int v)
{
    const int lane = static_cast<int>(lane_id());
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
    }
    return v;
}

// The groups on the line of tiles, by the whole CTA: first requests, tiles and places in shared memory (3 N + 1 ints).
// Returns whether cu_groups is a list of groups; line: its tiles and CTAs of n.
__device__ bool place_groups(const PrefixParams& p, int* cu, int* tiles, int* place, int2* sums, int n, Line& line)
{
    const int N = p.gr.n, tid = static_cast<int>(threadIdx.x), lane = tid & 31, warp = tid >> 5;
    const bool grouped = load_groups(p.gr, p.B, cu, tiles, [&](int b) { return keys_of(p, b); });
    // a run of groups per thread, then a scan over the threads
    const int per = (N + kPrefixThreads - 1) / kPrefixThreads, g0 = min(N, tid * per), g1 = min(N, g0 + per);
    const auto weight = [&](int g) { return p.Hkv * row_pairs(cu[g + 1] - cu[g], p.gr.nb) * tiles[g]; };
    int own = 0, units = 0;
    for (int g = g0; g < g1; ++g) {
        if (tiles[g] == 0) continue;
        own += weight(g);
        units += weight(g) / tiles[g];
    }
    const int inc = warp_scan_inc(own);
    units = static_cast<int>(__reduce_add_sync(0xffffffffu, static_cast<unsigned>(units)));
    if (lane == 31) sums[warp] = make_int2(inc, units);
    __syncthreads();
    int at = inc - own;
    units = 0;
    line.T = 0;
    for (int w = 0; w < kPrefixThreads / 32; ++w) {
        at += w < warp ? sums[w].x : 0;
        line.T += sums[w].x;
        units += sums[w].y;
    }
    line.P = paged_ctas(line.T, units, n);
    for (int g = g0; g < g1; ++g) {
        place[g] = at;
        if (tiles[g]) at += weight(g);
    }
    __syncthreads();
    return grouped;
}

// The requests' places for the decode kernel and the merge, by one CTA
__device__ void place_requests(const PrefixParams& p, const int* cu, const int* tiles, const int* place, int2* sums, bool grouped, const Line& line)
{
    const int B = p.B, tid = static_cast<int>(threadIdx.x), lane = tid & 31, warp = tid >> 5;
    const int per = (B + kPrefixThreads - 1) / kPrefixThreads, b0 = min(B, tid * per), b1 = min(B, b0 + per);
    const int first = grouped && b0 < b1 ? group_of(cu, p.gr.n, b0) : 0;
    const auto rest = [&](int b, int& g) {
        if (grouped)
            while (cu[g + 1] <= b) ++g;
        return max((keys_of(p, b) + kTileKV - 1) / kTileKV - (grouped ? tiles[g] : 0), 0);
    };
    int own = 0, with_keys = 0, g = first;
    for (int b = b0; b < b1; ++b) {
        const int t = rest(b, g);
        own += t;
        with_keys += t > 0 ? 1 : 0;
    }
    const int inc = warp_scan_inc(own);
    with_keys = static_cast<int>(__reduce_add_sync(0xffffffffu, static_cast<unsigned>(with_keys)));
    __syncthreads();
    if (lane == 31) sums[warp] = make_int2(inc, with_keys);
    __syncthreads();
    int at = inc - own, total = 0;
    with_keys = 0;
    for (int w = 0; w < kPrefixThreads / 32; ++w) {
        at += w < warp ? sums[w].x : 0;
        total += sums[w].x;
        with_keys += sums[w].y;
    }
    g = first;
    for (int b = b0; b < b1; ++b) {
        p.rest_prefix[b] = at;
        at += rest(b, g);
        p.plan[1 + b] = grouped ? make_int4(place[g], tiles[g], cu[g + 1] - cu[g], cu[g]) : make_int4(0, 0, 1, b);
    }
    if (tid == 0) {
        p.rest_prefix[B] = total;
        p.rest_prefix[B + 1] = paged_ctas(total * p.rest_units, with_keys * p.rest_units, p.rest_ctas);
        p.plan[0] = make_int4(line.T, line.P, 0, 0);
        if (!grouped) report_bad_page(p.status);
    }
}

template <int D>
__global__ void __launch_bounds__(kPrefixThreads, 1)
    prefix_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                  const __grid_constant__ PrefixParams p)
{
    using C = PrefixCfg<D>;
    using L = TileLayout<D, true>;
    constexpr int SK = C::kStagesK, SV = C::kStagesV;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));

    __shared__ uint64_t q_full, q_empty, k_full[SK], k_empty[SK], v_full[SV], v_empty[SV];
    // of each side: S is ready; P is stored over it; a piece's last PV is done; O has been read.  A QK needs no barrier for its
    // S: the MMA warp issues it behind the PV that read the P there.  So S of a side's next tile says that PV of the last one is
    // done, too.
    __shared__ uint64_t s_full[2], p_full[2], o_done[2], o_empty[2], mma_done;
    __shared__ uint64_t item_full[kItems], item_empty[kItems];
    __shared__ PrefixItem items[kItems];
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;
    __shared__ int2 sums[kPrefixThreads / 32];
    __shared__ int4 start_raw[2];
    Start* start_sh = reinterpret_cast<Start*>(start_raw);

    const int warp = threadIdx.x / 32, lane = static_cast<int>(threadIdx.x) & 31, N = p.gr.n;
    const int cta = static_cast<int>(blockIdx.x), ctas = static_cast<int>(gridDim.x) - 1;   // the last one is for the requests
    // in the memory that the key tiles will take
    int *cu = reinterpret_cast<int*>(smem), *tiles = cu + N + 1, *place = tiles + N;
    Line line;
    griddep_launch_dependents();
    if (cta == ctas) {
        griddep_wait();
        const bool grouped = place_groups(p, cu, tiles, place, sums, ctas, line);
        place_requests(p, cu, tiles, place, sums, grouped, line);
        return;
    }
    const WaitCtl wc{&abort_flag, p.status, p.limit};
    if (threadIdx.x == 0) {
        abort_flag = 0;
        mbar_init(&q_full, 1);
        mbar_init(&q_empty, 1);
        for (int i = 0; i < SK; ++i) {
            mbar_init(&k_full[i], 1);
            mbar_init(&k_empty[i], 1);
        }
        for (int i = 0; i < SV; ++i) {
            mbar_init(&v_full[i], 1);
            mbar_init(&v_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 4);    // one arrival per warp
            mbar_init(&o_done[i], 1);
            mbar_init(&o_empty[i], 4);   // one arrival per warp
        }
        for (int i = 0; i < kItems; ++i) {
            mbar_init(&item_full[i], 1);
            mbar_init(&item_empty[i], kItemReaders);
        }
        mbar_init(&mma_done, 1);
        fence_barrier_init();
    }
    if (warp == 10) {
        tmem_alloc(&tmem_slot, 512);
        tmem_relinquish();
    }
    if (threadIdx.x == 8 * 32) {
        tma_prefetch_desc(&qmap);
        tma_prefetch_desc(&kmap);
        tma_prefetch_desc(&vmap);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    griddep_wait();   // the previous kernel of the stream has completed: global memory from here on
    // A CTA's cut of the line at x, in the group of tiles [s, ..), nt to a unit
    const auto start_at = [](int x, int g, int s, int nt) {
        Start r;
        const int i = (x - s) / nt, u = s + i * nt, y = unit_cut(x, u, u + nt);
        r.g = y;
        r.b = g;
        r.i = y == u + nt ? i + 1 : i;
        r.t0 = y == u + nt ? 0 : y - u;
        return r;
    };
    // Up to 32 groups: a lane each of the warp that hands out the pieces, and the others need not wait for it
    if (N > 32) {
        const bool grouped = place_groups(p, cu, tiles, place, sums, ctas, line);
        if (threadIdx.x < 2) {   // the CTA's two cuts of the line
            Start r;
            const int c = cta + static_cast<int>(threadIdx.x);
            if (cta < line.P && line.T > 0 && grouped) {
                if (c == line.P) {
                    r.g = line.T;
                } else {
                    const int x = line.cut(c), g = group_of(place, N, x);   // the last group that begins at or before x has tiles there
                    r = start_at(x, g, place[g], tiles[g]);
                }
            }
            start_sh[threadIdx.x] = r;
        }
        fence_proxy_async_smem();   // what was written here before key tiles land in it
        __syncthreads();
    }

    if (warp >= 8) {
        setmaxnreg_dec<kRegsCtl>();
        // ------------------------------------------------ TMA producers, as the paged ones of decode_kernel.cuh
        const bool is_k = warp == 8;
        const auto first_key = [&](int t) { return t * kTileKV + lane * p.box; };   // of this lane's box of tile t
        const int boxes = kTileKV >> p.box_log2, tile_rows = p.gr.nb * p.R;
        const CUtensorMap* map = is_k ? &kmap : &vmap;
        uint64_t *full = is_k ? k_full : v_full, *empty = is_k ? k_empty : v_empty;
        uint8_t* ring = smem + (is_k ? C::kOffK : C::kOffV);
        const uint64_t pol = policy_evict_first();
        Ring ir(kItems), r(is_k ? SK : SV);
        uint32_t issued = 0;   // loads of the ring
        const auto fill = [&](const PrefixItem& it) {
            const int32_t* row = p.table + static_cast<size_t>(it.trow) * p.max_pages;
            const auto look_up = [&](int t) { return t < it.t1 && lane < boxes ? row[p.by_page.div(first_key(t))] : 0; };
            int next_page = look_up(it.t0);
            for (int t = it.t0; t < it.t1; ++t) {
                int page = next_page;
                next_page = look_up(t + 1);
                const int j = first_key(t), off = j - p.by_page.div(j) * p.page;
                const bool mine = lane < boxes;
                if (mine && (page < 0 || page >= p.num_pages)) {
                    page = p.num_pages;
                    report_bad_page(p.status);
                }
                int go = 0;
                if (lane == 0) {
                    mbar_wait(&empty[r.idx], r.phase ^ 1, wc);
                    go = aborted(wc) ? 0 : 1;
                    if (go) mbar_arrive_expect_tx(&full[r.idx], C::kKVBytes);
                }
                if (!__shfl_sync(0xffffffffu, go, 0)) continue;
                if (mine) {
                    uint8_t* dst = ring + r.idx * C::kKVBytes + lane * (p.box / 8) * L::kGroup;
                    if constexpr (L::kInter)
                        tma_load_5d_hint(dst, map, &full[r.idx], 0, 0, 0, page * p.groups + off / 8, it.head, pol);
                    else
                        tma_load_4d_hint(dst, map, &full[r.idx], 0, off, it.head, page, pol);
                }
                ++issued;
                r.advance();
            }
        };
        // nothing may still be landing in shared memory when the CTA exits
        const auto drain = [&]() {
            const uint32_t n = static_cast<uint32_t>(r.n);
            if (lane == 0)
                for (uint32_t i = 0; i < n && i < issued; ++i) drain_wait(&full[i], ((issued - 1 - i) / n) & 1, kDrainLimit);
            __syncwarp();
        };
        if (warp == 11) {
            // ------------------------------------------------ pieces, in the order of the line
            // a lane looks at a group
            int nt, b0, members;
            const auto look = [&](int g) {
                nt = b0 = members = 0;
                if (g >= N) return false;
                const int from = p.gr.cu[g], to = p.gr.cu[g + 1];
                if (from < 0 || to < from || to > p.B || (g == 0 && from != 0) || (g == N - 1 && to != p.B)) return true;   // no list of groups
                b0 = from;
                members = to - from;
                return false;
            };
            const auto count = [&](int g) {
                if (members > 0) nt = shared_tiles(p.gr, b0, b0 + members, p.gr.prefix[g], keys_of(p, b0));
            };
            Start first;
            int end = 0;
            if (N > 32) {
                first = start_sh[0];
                end = start_sh[1].g;
            } else if (!__any_sync(0xffffffffu, look(lane))) {
                count(lane);
                const int units = nt > 0 ? p.Hkv * row_pairs(members, p.gr.nb) : 0, inc = warp_scan_inc(units * nt), at = inc - units * nt;
                line.T = __shfl_sync(0xffffffffu, inc, 31);
                line.P = paged_ctas(line.T, static_cast<int>(__reduce_add_sync(0xffffffffu, static_cast<unsigned>(units))), ctas);
                if (cta < line.P && line.T > 0) {
                    // even lanes look at the CTA's first cut, odd lanes at the next CTA's
                    const int x = line.cut(cta + (lane & 1)), x0 = __shfl_sync(0xffffffffu, x, 0), x1 = __shfl_sync(0xffffffffu, x, 1);
                    const unsigned has0 = __ballot_sync(0xffffffffu, at <= x0 && x0 < inc), has1 = __ballot_sync(0xffffffffu, at <= x1 && x1 < inc);
                    const int g = max(__ffs(lane & 1 ? has1 : has0) - 1, 0);
                    const int s = __shfl_sync(0xffffffffu, at, g), t = __shfl_sync(0xffffffffu, nt, g);
                    const Start mine = start_at(x, g, s, max(t, 1));
                    first.g = __shfl_sync(0xffffffffu, mine.g, 0);
                    first.b = __shfl_sync(0xffffffffu, mine.b, 0);
                    first.i = __shfl_sync(0xffffffffu, mine.i, 0);
                    first.t0 = __shfl_sync(0xffffffffu, mine.t0, 0);
                    end = has1 ? __shfl_sync(0xffffffffu, mine.g, 1) : line.T;   // no group: the cut behind the last tile
                }
            }
            const auto emit = [&](const PrefixItem& it) {
                int ok = 1;
                if (lane == 0) {
                    ok = mbar_wait(&item_empty[ir.idx], ir.phase ^ 1, wc) ? 1 : 0;
                    if (ok) {
                        items[ir.idx] = it;
                        mbar_arrive(&item_full[ir.idx]);
                    }
                }
                ir.advance();
                return __shfl_sync(0xffffffffu, ok, 0) != 0;
            };
            int pos = first.g, i = first.i, t0 = first.t0;
            bool go = true;
            for (int g0 = N > 32 ? first.b : 0; go && pos < end && g0 < N; g0 += 32) {
                if (N > 32) {
                    look(g0 + lane);
                    count(g0 + lane);
                }
                for (int l = N > 32 ? 0 : first.b; l < 32 && go && pos < end; ++l) {
                    const int t = __shfl_sync(0xffffffffu, nt, l), fb = __shfl_sync(0xffffffffu, b0, l), m = __shfl_sync(0xffffffffu, members, l);
                    if (t > 0) {
                        const int pairs = row_pairs(m, p.gr.nb);
                        int head = i / pairs, r = i - head * pairs;
                        while (go && head < p.Hkv && pos < end) {
                            PrefixItem it;
                            it.t0 = t0;
                            it.t1 = min(t, end - pos + t0);
                            it.trow = fb;
                            it.head = head;
                            it.b0 = fb + r * 2 * p.gr.nb;
                            it.rows = min(2 * p.gr.nb, m - r * 2 * p.gr.nb) * p.R;
                            it.prow = 2 * (fb * p.Hkv + head * m + r * 2 * p.gr.nb) * p.R + cta * 2 * kRows;
                            pos += it.t1 - it.t0;
                            t0 = 0;
                            if (++r == pairs) {
                                r = 0;
                                ++head;
                            }
                            go = emit(it);
                        }
                    }
                    i = 0;
                }
            }
            if (go) emit(PrefixItem{});
        } else if (warp == 8 || warp == 9) {
            // ------------------------------------------------ K; Q and V
            uint32_t q_issued = 0, n = 0;
            for (;; ++n) {
                if (!__all_sync(0xffffffffu, mbar_wait(&item_full[ir.idx], ir.phase, wc))) break;
                const PrefixItem it = items[ir.idx];
                __syncwarp();
                if (lane == 0) mbar_arrive(&item_empty[ir.idx]);
                ir.advance();
                if (it.t1 <= it.t0) break;
                if (!is_k && lane == 0) {
                    const int two = it.rows > tile_rows ? 2 : 1;
                    mbar_wait(&q_empty, (n & 1) ^ 1, wc);
                    if (!aborted(wc)) {
                        mbar_arrive_expect_tx(&q_full, static_cast<uint32_t>(two * tile_rows * 128 * C::kAtoms));
                        for (int s = 0; s < two; ++s)
                            for (int a = 0; a < C::kAtoms; ++a)
                                tma_load_4d_hint(smem + C::kOffQ + s * C::kQBytes + a * (kRows * 128), &qmap, &q_full, a * 64, 0, it.head,
                                                 it.b0 + s * p.gr.nb, pol);
                        ++q_issued;
                    }
                }
                __syncwarp();
                fill(it);
            }
            drain();
            if (lane == 0 && q_issued) drain_wait(&q_full, (q_issued - 1) & 1, kDrainLimit);
            __syncwarp();
        } else {
            // ------------------------------------------------ MMA issuer (the whole warp, see mma_ss_warp)
            constexpr uint32_t idesc_qk = idesc_bf16_f32(kRows, kTileKV, false, false);
            constexpr uint32_t idesc_pv = idesc_bf16_f32(kRows, D, false, true);
            constexpr uint32_t lbo_v = D >= 128 ? L::kHalf : 0u;
            // descriptors of the buffers' beginnings; steps inside them add constants to the address fields
            const uint64_t q_desc = sdesc_sw128(smem_u32(smem + C::kOffQ), 16, 1024), k_desc = sdesc_sw128(smem_u32(smem + C::kOffK), 16, L::kGroup),
                           v_desc = sdesc_sw128(smem_u32(smem + C::kOffV), lbo_v, L::kGroup);
            Ring ir(kItems), kr(SK), vr(SV), qr(1);
            uint32_t n_pv[2] = {0, 0}, n_items[2] = {0, 0};   // of each side over the kernel's life
            bool ok = true;                                   // until a wait gives up
            const auto wait = [&](uint64_t* bar, uint32_t parity) { ok = __all_sync(0xffffffffu, mbar_wait(bar, parity, wc)) && ok; };
            for (;;) {
                wait(&item_full[ir.idx], ir.phase);
                if (!ok) break;
                const PrefixItem it = items[ir.idx];
                __syncwarp();
                if (lane == 0) mbar_arrive(&item_empty[ir.idx]);
                ir.advance();
                if (it.t1 <= it.t0) break;
                // Step j is side j & 1's: with two row tiles both sides take each key tile, else every other one
                const bool two = it.rows > p.gr.nb * p.R;
                const int steps = two ? 2 * (it.t1 - it.t0) : it.t1 - it.t0;
                wait(&q_full, qr.phase);
                // QK of step j + 2 goes behind PV of step j, whose P lies over its S
                for (int j0 = -2; j0 < steps; j0 += 2) {
#pragma unroll
                    for (int side = 0; side < 2; ++side) {
                        const int j = j0 + side;
                        if (j >= 0 && j < steps) {
                            if (!two || side == 0) wait(&v_full[vr.idx], vr.phase);
                            if (j < 2) wait(&o_empty[side], (n_items[side]++ & 1) ^ 1);   // O of the side's item before has been read
                            wait(&p_full[side], n_pv[side]++ & 1);
                            tc_fence_after();
                            if (ok) {
                                const uint64_t dv = v_desc + vr.idx * (C::kKVBytes >> 4);
                                const uint32_t aP = tmem + C::col_s(side), dO = tmem + C::col_o(side);
#pragma unroll
                                for (int ks = 0; ks < kTileKV / 16; ++ks)   // 16 keys: the weights, and what their rounding left
#pragma unroll
                                    for (int half = 0; half < 2; ++half)
                                        mma_ts_warp(dO, aP + ks * 16 + half * 8, dv + ((ks * 2 * L::kGroup) >> 4), idesc_pv, ks + half > 0 || j >= 2 ? 1u : 0u);
                                if (!two || side) mma_commit_warp(&v_empty[vr.idx]);
                                if (j + 2 >= steps) mma_commit_warp(&o_done[side]);
                            }
                            if (!two || side) vr.advance();
                        }
                        if (j + 2 < steps) {
                            if (!two || side == 0) wait(&k_full[kr.idx], kr.phase);
                            tc_fence_after();
                            if (ok) {
                                const uint64_t dq = q_desc + (two && side ? C::kQBytes >> 4 : 0), dk = k_desc + kr.idx * (C::kKVBytes >> 4);
#pragma unroll
                                for (int kk = 0; kk < D / 16; ++kk)
                                    mma_ss_warp(tmem + C::col_s(side), dq + (((kk >> 2) * (kRows * 128) + (kk & 3) * 32) >> 4),
                                                dk + (((kk >> 2) * L::kHalf + (kk & 3) * 32) >> 4), idesc_qk, kk > 0 ? 1u : 0u);
                                mma_commit_warp(&s_full[side]);   // K and Q are given back by who sees it: a commit costs 150 cycles
                            }
                            if (!two || side) kr.advance();
                        }
                    }
                }
                qr.advance();
            }
            mma_commit_warp(&mma_done);
            drain_wait(&mma_done, 0, kDrainLimit);
            __syncwarp();
        }
    } else {
        setmaxnreg_inc<kRegsSide>();
        // ------------------------------------------------ a side: softmax and the piece's partials, a row per thread
        const int side = warp >> 2, tid = threadIdx.x & 127;
        const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t s_cols = tmem + lane_base + C::col_s(side), tO = tmem + lane_base + C::col_o(side);
        const int member = tid / p.R, query = (tid - member * p.R) % p.Sq, tile_rows = p.gr.nb * p.R;
        Ring ir(kItems);
        uint32_t n = 0, k_pos = 0, pieces = 0;   // this side's key tiles, all key tiles and this side's pieces over the kernel's life
        // Ahead of the first piece the code below runs once on what happens to be in O's columns, so that it is in the
        // instruction cache by the time the first scores are: cold, a tile takes 5600 cycles instead of 1700
        for (bool cold = true;; cold = false) {
            PrefixItem it{0, 0, 0, 0, 0, 2 * kRows, 0};
            if (!cold) {
                if (!__all_sync(0xffffffffu, mbar_wait(&item_full[ir.idx], ir.phase, wc))) break;
                it = items[ir.idx];
                __syncwarp();
                if (lane == 0) mbar_arrive(&item_empty[ir.idx]);
                ir.advance();
                if (it.t1 <= it.t0) break;
            }
            const bool two = it.rows > tile_rows;
            const int rows = two && side ? it.rows - tile_rows : min(it.rows, tile_rows), step = two ? 1 : 2;
            const bool busy = (warp & 3) * 32 < rows;   // of the other warps nothing is wanted
            int lim = 1 << 30;                          // keys that this row sees (rows that are none: whatever is there)
            if (tid < rows && !cold) {
                lim = keys_of(p, it.b0 + (two && side ? p.gr.nb : 0) + member);
                if (p.causal) lim += 1 - p.Sq + query;
            }
            float m = -INFINITY, l = 0.f;
            const int first = it.t0 + (two ? 0 : side);
            for (int t = cold ? -1 : first; t < it.t1; t += step) {
                const uint32_t tS = cold ? tO : s_cols;
                if (!cold) mbar_wait(&s_full[side], n & 1, wc);
                tc_fence_after();
                // the MMA warp's last product with this key tile (and with Q): two row tiles take turns, side 1 last
                if ((warp & 3) == 3 && lane == 0 && (!two || side) && !cold) {
                    mbar_arrive(&k_empty[(k_pos + (t - it.t0)) % SK]);
                    if (t + 1 == it.t1) mbar_arrive(&q_empty);
                }
                if (busy) {
                    __syncwarp();
                    float s[kTileKV];
                    uint32_t* su = reinterpret_cast<uint32_t*>(s);
#pragma unroll
                    for (int c4 = 0; c4 < kTileKV / 32; ++c4) tmem_ld32p(tS + c4 * 32, su + c4 * 32);
                    tmem_ld_wait();
                    const int see = lim - t * kTileKV;
                    if (see < kTileKV) {
#pragma unroll
                        for (int i = 0; i < kTileKV; ++i)
                            if (i >= see) s[i] = -INFINITY;
                    }
                    float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
                    for (int i = 4; i < kTileKV; i += 8) {
                        mx[0] = fmax3(mx[0], s[i], s[i + 1]);
                        mx[1] = fmax3(mx[1], s[i + 2], s[i + 3]);
                        if (i + 4 < kTileKV) {
                            mx[2] = fmax3(mx[2], s[i + 4], s[i + 5]);
                            mx[3] = fmax3(mx[3], s[i + 6], s[i + 7]);
                        }
                    }
                    // the reference moves only when a score exceeds it by more than 2^8, so P <= 256; O / l and m + log2 l
                    // are exact for any reference
                    const float mt = fmax3(fmaxf(mx[0], mx[1]), mx[2], mx[3]) * p.c;
                    const bool up = mt > m + kRescaleD && (tid < rows || t == first);
                    const float alpha = up ? ex2_approx(m - mt) : 1.f;
                    if (up) m = mt;
                    if (t > first && __any_sync(0xffffffffu, up)) {   // tcgen05.ld/st are warp-collective
                        __syncwarp();
#pragma unroll 1
                        for (int c = 0; c < D; c += 16) {
                            uint32_t o[16];
                            tmem_ld16(tO + c, o);
                            tmem_ld_wait();
#pragma unroll
                            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
                            tmem_st16(tO + c, o);
                        }
                    }
                    const uint64_t cc = f32x2(p.c, p.c);
                    const float mu = m == -INFINITY ? 0.f : -m;   // no visible key yet: -inf - 0
                    const uint64_t nm = f32x2(mu, mu);
                    uint64_t ls[4] = {0ull, 0ull, 0ull, 0ull};
                    __syncwarp();
#pragma unroll
                    for (int c = 0; c < kTileKV; c += 16) {
                        uint32_t w[16];
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            float x0, x1;
                            f32x2_split(ffma2(f32x2(s[c + 2 * i], s[c + 2 * i + 1]), cc, nm), x0, x1);
                            const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
                            ls[i & 3] = fadd2(ls[i & 3], f32x2(p0, p1));
                            w[i] = pack_bf16x2(p0, p1);
                            w[8 + i] = pack_bf16x2(p0 - __uint_as_float(w[i] << 16), p1 - __uint_as_float(w[i] & 0xffff0000u));
                        }
                        tmem_st16(tS + c, w);
                    }
                    float la, lb;
                    f32x2_split(fadd2(fadd2(ls[0], ls[1]), fadd2(ls[2], ls[3])), la, lb);
                    l = fmaf(l, alpha, la + lb);
                    tmem_st_wait();
                }
                tc_fence_before();
                __syncwarp();
                if (cold) break;
                if (lane == 0) mbar_arrive(&p_full[side]);
                ++n;
            }
            if (cold) continue;
            // the piece's partials: O / l and the LSE
            const bool any = first < it.t1;
            if (any) {
                mbar_wait(&o_done[side], pieces++ & 1, wc);
                tc_fence_after();
                __syncwarp();
            }
            if (busy) {
                const bool none = l == 0.f;   // no visible key; a NaN score makes the sum, the row and its LSE NaN
                const float inv = none ? 0.f : 1.f / l;
                const bool store = tid < rows && !aborted(wc);
                const size_t row = static_cast<size_t>(it.prow) + (side ? (two ? tile_rows : it.rows) : 0) + tid;
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                    uint32_t o[32];
                    if (any) {
                        tmem_ld32(tO + c, o);
                        tmem_ld_wait(o);
                    }
                    float x[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) x[i] = none || !any ? 0.f : __uint_as_float(o[i]) * inv;
                    if (store)
#pragma unroll
                        for (int i = 0; i < 4; ++i) st_global_v8(p.part_o + row * D + c + 8 * i, x + 8 * i);
                }
                if (store) p.part_lse[row] = none ? -INFINITY : (m + __log2f(l)) * kLn2;
            }
            if (any) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&o_empty[side]);
            }
            k_pos += it.t1 - it.t0;
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 10) tmem_dealloc(tmem, 512);
}

struct MergeParams {
    int rows, Hkv, R, nb;
    int shares;                // warps of a row: 1, 2, 4 or 8
    int G, chunks;             // of the decode kernel's units
    const int4* plan;
    const int32_t* rest_prefix;
    const float *common_o, *common_lse;   // partials of the groups' common keys
    const float *own_o, *own_lse;         // and of the requests' own: [U + SMs][16]
    void* out;                 // BF16 or F32, or NULL
    int out_f32;
    float* lse;
    float* o_stage;            // FP32 copy for NVFP4, else NULL
    unsigned* amax_bits;
};

// Merges the partials of a row: the pieces of its group's common keys and of its own.  A warp per row takes three dependent
// round trips to L2 and one for each four partials more; where there are few rows, up to eight warps share theirs (128 rows
// of 40 partials: 12 us with one, 6 with eight).
template <int D>
__global__ void __launch_bounds__(256, 5) prefix_merge_kernel(const __grid_constant__ MergeParams p)
{
    constexpr int V = D / 32;   // features of a lane
    griddep_launch_dependents();
    griddep_wait();
    __shared__ float part[8][D], part_m[8], part_l[8];
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, share = warp % p.shares, row = (blockIdx.x * 8 + warp) / p.shares;
    if (row >= p.rows) return;   // the last block's, warps of whole rows
    const int unit = row / p.R, rr = row - unit * p.R, b = unit / p.Hkv, h = unit - b * p.Hkv, B = p.rows / (p.R * p.Hkv);
    const int4 head = p.plan[0], g = p.plan[1 + b];   // g: place, tiles, requests and first one of the group
    const int before = p.rest_prefix[b], nt = p.rest_prefix[b + 1] - before;
    Line own_line;
    own_line.T = p.rest_prefix[B] * p.Hkv * p.chunks;
    own_line.P = p.rest_prefix[B + 1];

    // the CTAs [c, c + n) of a line have pieces of its unit of tiles [s, e)
    const auto find = [](const Line& line, int s, int e, int& c, int& n) {
        const float per = static_cast<float>(line.P) / static_cast<float>(line.T);
        const auto at = [&](int i) { return unit_cut(line.cut(i), s, e); };
        c = max(min(static_cast<int>(static_cast<float>(s) * per), line.P - 1), 0);
        while (c > 0 && at(c) > s) --c;
        while (at(c + 1) <= s) ++c;
        int d = max(min(static_cast<int>(static_cast<float>(e) * per), line.P), c + 1);
        while (d < line.P && at(d) < e) ++d;
        while (d > c + 1 && at(d - 1) >= e) --d;
        n = d - c;
    };
    // partial i of n1 + n2: first those of the group's common keys (of a pair of row tiles with one tile two a piece, `second` rows
    // apart), then the request's own
    int c1 = 0, n1 = 0, second = 0, c2 = 0, n2 = 0;
    long long first1 = 0, first2 = 0;
    if (g.y > 0) {
        Line line;
        line.T = head.x;
        line.P = head.y;
        const int pairs = row_pairs(g.z, p.nb), mem = b - g.w, r = mem / (2 * p.nb), s = g.x + (h * pairs + r) * g.y;
        const int rows = min(2 * p.nb, g.z - r * 2 * p.nb) * p.R;
        find(line, s, s + g.y, c1, n1);
        second = rows > p.nb * p.R ? 0 : rows;
        n1 <<= second ? 1 : 0;
        first1 = 2 * static_cast<long long>(g.w * p.Hkv + h * g.z + r * 2 * p.nb) * p.R + (mem - r * 2 * p.nb) * p.R + rr;
    }
    if (nt > 0) {
        const int chunk = rr / p.G, i = h * p.chunks + chunk, units = p.Hkv * p.chunks, s = before * units + i * nt;
        find(own_line, s, s + nt, c2, n2);
        first2 = static_cast<long long>(b * units + i) * kN + rr - chunk * p.G;
    }
    if (p.out && n1 == 0 && n2 == 1) return;   // one piece was all of it and wrote the row (for all warps of the row)
    float m = -INFINITY, l = 0.f, acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.f;
    const int mine = (n1 + n2 - share + p.shares - 1) / p.shares;   // this warp's: every p.shares-th
    for (int i0 = 0; i0 < mine; i0 += 32) {   // a lane per partial
        const int i = (i0 + lane) * p.shares + share, n = min(mine - i0, 32);
        long long at = 0;
        const float *lse = p.common_lse, *o = p.common_o;
        if (i < n1) {
            at = first1 + static_cast<long long>(c1 + (second ? i >> 1 : i)) * (2 * kRows) + (second && (i & 1) ? second : 0);
        } else {
            at = first2 + static_cast<long long>(c2 + i - n1) * kN;
            lse = p.own_lse;
            o = p.own_o;
        }
        const float x = lane < n ? __ldcg(lse + at) : -INFINITY;
        o += at * D;
        const float top = fmax_nan(m, redux_max_nan(x));
        if (top == -INFINITY) continue;   // no visible key so far
        const float keep = m == -INFINITY ? 0.f : __expf(m - top), w = lane < n ? __expf(x - top) : 0.f;
        m = top;
        l = l * keep + warp_sum(w);
#pragma unroll
        for (int v = 0; v < V; ++v) acc[v] *= keep;
#pragma unroll 4
        for (int k = 0; k < n; ++k) {
            const float* src = reinterpret_cast<const float*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(o), k)) + lane * V;
            const float wk = __shfl_sync(0xffffffffu, w, k);
            if constexpr (V == 4) {
                const float4 v = __ldcg(reinterpret_cast<const float4*>(src));
                acc[0] = fmaf(wk, v.x, acc[0]);
                acc[1] = fmaf(wk, v.y, acc[1]);
                acc[2] = fmaf(wk, v.z, acc[2]);
                acc[3] = fmaf(wk, v.w, acc[3]);
            } else {
                const float2 v = __ldcg(reinterpret_cast<const float2*>(src));
                acc[0] = fmaf(wk, v.x, acc[0]);
                acc[1] = fmaf(wk, v.y, acc[1]);
            }
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
    size_t plan_off, pre_off, common_lse_off, common_o_off, own_lse_off, own_o_off, stage_off, amax_off, total;
};

// With so many key tiles at most, all requests' tables full, every request is read by itself.  Three launches and the merge cost
// about 20 us; a tile that another request has just brought to L2 costs the paged attention 4 to 5 ns.
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
    take(w.pre_off, (static_cast<size_t>(B) + 2) * 4);
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
int run_prefix(PrefixParams& p, MergeParams& m, const PagedArgs& a, const PagedRest& rest, cudaStream_t st)
{
    using C = PrefixCfg<D>;
    CUtensorMap qmap, kmap, vmap;
    const uint64_t dims[4] = {static_cast<uint64_t>(D), static_cast<uint64_t>(p.R), static_cast<uint64_t>(p.Hkv), static_cast<uint64_t>(p.B)};
    const uint64_t strides[3] = {static_cast<uint64_t>(D) * 2, static_cast<uint64_t>(p.R) * D * 2, static_cast<uint64_t>(p.Hkv) * p.R * D * 2};
    const uint32_t box[4] = {64, static_cast<uint32_t>(p.R), 1, static_cast<uint32_t>(p.gr.nb)};
    int rc = make_tmap_bf16(&qmap, a.q, 4, dims, strides, box);
    if (!rc) rc = make_pool_map(&kmap, a.c->k, a.c, p.box);
    if (!rc) rc = make_pool_map(&vmap, a.c->v, a.c, p.box);
    if (rc) return rc;
    const int nsm = num_sms();
    if (nsm <= 0) return set_error(FMHA_ERR_CUDA, "cannot query the SM count");
    const long long cap_tiles = (static_cast<long long>(p.cap) + kTileKV - 1) / kTileKV;
    p.rest_ctas = rest_grid(a.B * p.rest_units, p.cap, nsm);
    // one CTA per SM, one of which places the requests; fewer when even full tables have no work for so many (half the
    // requests' tiles at most are common ones, see paged_ctas)
    const long long units = static_cast<long long>(p.B) * p.Hkv / 2 + 1, tiles = units * cap_tiles;
    const long long most = tiles / kMinPiece > units ? tiles / kMinPiece : units;
    const unsigned grid = static_cast<unsigned>(most < nsm - 1 ? most : nsm - 1) + 1;
    FMHA_CHECK_CUDA(set_smem_limit_once(reinterpret_cast<const void*>(prefix_kernel<D>), C::kSmemBytes));
    timing_mark_begin(st);
    const cudaError_t e = launch_pdl(prefix_kernel<D>, dim3(grid), dim3(kPrefixThreads), static_cast<size_t>(C::kSmemBytes), st, qmap, kmap, vmap, p);
    timing_mark_end(st);
    FMHA_CHECK_CUDA(e);
    count_launch();
    rc = launch_paged_rest(a, rest, st);
    if (rc) return rc;
    m.shares = 1;
    while (m.shares < 8 && static_cast<long long>(m.rows) * m.shares * 2 <= 16LL * nsm) m.shares *= 2;   // half of the warps that fit
    const int per = 8 / m.shares;
    FMHA_CHECK_CUDA(launch_pdl(prefix_merge_kernel<D>, dim3(static_cast<unsigned>((m.rows + per - 1) / per)), dim3(256), 0, st, m));
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
    p.gr = Groups{cu_groups, prefix_lens, N, kRows / p.R};
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
    p.rest_units = p.Hkv * shape.chunks;
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
    const PagedRest rest{p.rest_prefix, reinterpret_cast<float*>(base + w.own_o_off), reinterpret_cast<float*>(base + w.own_lse_off)};

    MergeParams m{};
    m.rows = B * Hq * Sq;
    m.Hkv = p.Hkv;
    m.R = p.R;
    m.nb = p.gr.nb;
    m.G = shape.G;
    m.chunks = shape.chunks;
    m.plan = p.plan;
    m.rest_prefix = p.rest_prefix;
    m.common_o = p.part_o;
    m.common_lse = p.part_lse;
    m.own_o = rest.part_o;
    m.own_lse = rest.part_lse;
    m.out = nvfp4 ? nullptr : out;
    m.out_f32 = o.out_kind == FMHA_OUT_F32 ? 1 : 0;
    m.lse = lse;
    if (nvfp4) {
        m.o_stage = o.out_f32 ? o.out_f32 : reinterpret_cast<float*>(base + w.stage_off);
        m.amax_bits = o.out_amax ? reinterpret_cast<unsigned*>(o.out_amax) : reinterpret_cast<unsigned*>(base + w.amax_off);
        FMHA_CHECK_CUDA(cudaMemsetAsync(m.amax_bits, 0, sizeof(unsigned), st));
    }
    rc = cache->D == 64 ? run_prefix<64>(p, m, a, rest, st) : run_prefix<128>(p, m, a, rest, st);
    if (rc || !nvfp4) return rc;
    return launch_nvfp4(m.o_stage, static_cast<uint8_t*>(out), o.out_scales, o.out_tensor_scale, m.amax_bits,
                        static_cast<int64_t>(m.rows) * cache->D, true, st, o.nvfp4_scale_in);
}
