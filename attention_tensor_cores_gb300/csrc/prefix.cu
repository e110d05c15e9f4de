// Attention of requests that share their first pages (fmha_fwd_prefix): each group's common keys are read
// once for all its requests.
//
//   o_b = softmax(scale q_b K_b^T) V_b as in fmha_fwd_paged.  With the keys of request b in disjoint sets
//   C_1, C_2, .., O_i and lse_i the attention over C_i alone:  lse = log sum_i exp(lse_i),  o_b = sum_i exp(lse_i - lse) O_i
//
// so a group's common keys, in whole tiles of 128, are one problem whose rows are the queries of all its requests,
// and what is left of each request is a problem of its own.  Per key/value head a request has R = (Hq / Hkv) Sq rows.
//
//  * Row tiles.  S = Q K^T with up to 128 query rows as the MMA's M: floor(128 / R) requests of a group for its common
//    keys, one request for its own.  A row is a thread's (Tensor Memory lane), so maxima and sums need no other
//    thread.  An MMA of 128 rows costs the same for any number of them, 1.5 k cycles a tile at D = 128 against 2.8 k that
//    HBM takes to bring the tile to one SM of 152: idle rows are free as long as the keys come from memory.
//  * P goes to the tensor core as two BF16, the rounded weight (half a step, 2^-9) and what the rounding left, both over
//    the S that they come from, in an MMA each: P is good to 2^-17 as in fmha_fwd_paged, and the output's rounding is
//    the only one that shows.
//  * Work split.  The key tiles of all problems, first the groups' then the requests', are laid end to end and cut
//    for P CTAs (as in decode_kernel.cuh); a piece of a problem is an item.  Lengths are on the device, so every CTA sums the
//    entries itself.  An item that is a request's whole attention writes its rows; every other one writes normalised
//    partials, which a second kernel merges, a warp per row.
//  * Roles: warps 0-3 softmax, 4-7 epilogue, 8 K, 9 V and Q, 10 MMA, 11 finds the items and hands them to the others
//    through a ring in shared memory.  S (and P) and O alternate between two buffers each in Tensor Memory.
//  * Every wait is bounded, as in decode_kernel.cuh.
#include <cuda_runtime.h>

#include "decode_kernel.cuh"
#include "paged.h"

namespace atc_gb300 {
namespace {

constexpr int kRows = 128;          // query rows of a tile
constexpr int kItems = 8;           // slots of the item ring
constexpr int kItemReaders = 11;    // K, V and MMA warps, four softmax and four epilogue warps
constexpr int kMaxGroups = 8192;
// A group's keys are shared when that spares at least so many tiles of one key/value head: its rows' partials and one
// more item for each request cost about as much.
constexpr int kMinShared = 4;

template <int D>
struct PrefixCfg {
    static constexpr int kAtoms = D / 64;
    static constexpr int kStages = D == 64 ? 6 : 3;
    static constexpr int kQBytes = kAtoms * kRows * 128;
    static constexpr int kKVBytes = kAtoms * kTileKV * 128;
    static constexpr int kOffQ = 0;
    static constexpr int kOffK = kOffQ + kQBytes;
    static constexpr int kOffV = kOffK + kStages * kKVBytes;
    static constexpr int kSmemBytes = kOffV + kStages * kKVBytes + 1024;   // + alignment slack
    // Tensor Memory columns: S[2] x 128 (P's two halves over them), O[2] x D
    static constexpr uint32_t col_s(uint32_t i) { return i * 128; }
    static constexpr uint32_t col_o(uint32_t i) { return 256 + i * D; }
};

struct PrefixParams {
    int B, N;            // requests, groups
    int Hkv, R, Sq;      // rows of a request and key/value head; column r is query r % Sq
    int Rt, ch;          // rows of a request in a tile (up to 128), tiles of a request
    int nb;              // requests of a group in a tile (below 2: nothing is shared)
    int causal;
    float c;             // scale * log2(e)
    const int32_t* cu;
    const int32_t* prefix;
    const int32_t* seqlens;
    const int32_t* table;
    int max_pages, num_pages, page;
    FastDiv by_page;
    int box, box_log2, groups;   // as in DecodeParams
    int cap;             // max_pages * page: lengths are clamped to it
    void* out;           // BF16 or F32 rows, or NULL: every row goes through the merge
    int out_f32;
    float* lse;
    float* o_stage;      // the merge's FP32 copy for NVFP4, else NULL
    unsigned* amax_bits;
    float* part_o;       // [rows][D]: common keys' partials, from own_rows on the requests' own
    float* part_lse;
    long long own_rows;
    int4* plan;          // [1 + 2 B]: (T, P), and of each request its place on the line
    int* status;
    long long limit;
};

// A piece of a problem
struct PrefixItem {
    int t0, t1;      // tiles of keys
    int keys, trow;  // tokens and row of the block table
    int b0, head;    // (first) request
    int rows, rr0;   // rows of the tile, and the first one's place in its request
    int prow;        // first row of the partial
    int kind;        // kMany, kWhole, kEnd
};
enum : int { kMany = 1, kWhole = 2, kEnd = 4 };

__device__ __forceinline__ int keys_of(const PrefixParams& p, int b) { return min(max(p.seqlens[b], 0), p.cap); }

// Tiles of keys that the requests [b0, b1) of a group read together, and their row tiles.  n0: keys of the
// first one, through whose row they are read.
__device__ __forceinline__ int shared_tiles(const PrefixParams& p, int b0, int b1, int prefix, int n0, int& row_tiles)
{
    const int members = b1 - b0;
    row_tiles = 0;
    if (members < 2 || p.nb < 2) return 0;
    row_tiles = (members + p.nb - 1) / p.nb;
    const int tiles = min(max(prefix, 0), n0) / kTileKV;
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

template <int D>
__global__ void __launch_bounds__(384, 1)
    prefix_kernel(const __grid_constant__ CUtensorMap qmany, const __grid_constant__ CUtensorMap qone, const __grid_constant__ CUtensorMap kmap,
                  const __grid_constant__ CUtensorMap vmap, const __grid_constant__ PrefixParams p)
{
    using C = PrefixCfg<D>;
    using L = TileLayout<D, true>;
    constexpr int S = C::kStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));

    __shared__ uint64_t q_full[2], q_empty[2], k_full[S], k_empty[S], v_full[S], v_empty[S];
    // S(k) is ready; P(k) is stored over it; PV(k) is done; an item's last PV is done; O has been read.  QK(k) needs no
    // barrier of its own for S's buffer: the MMA warp issues it behind PV(k - 2), which read P(k - 2) there.
    __shared__ uint64_t s_full[2], p_full[2], o_done, o_last[2], o_empty[2], ml_full, ml_empty, mma_done;
    __shared__ uint64_t item_full[kItems], item_empty[kItems];
    __shared__ PrefixItem items[kItems];
    __shared__ float2 ml[kRows];       // softmax -> epilogue: a row's reference maximum and sum
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;
    __shared__ int4 sums[12];
    __shared__ int4 start_raw[2];
    Start* start_sh = reinterpret_cast<Start*>(start_raw);

    const int warp = threadIdx.x / 32, lane = static_cast<int>(threadIdx.x) & 31;
    griddep_launch_dependents();
    const WaitCtl wc{&abort_flag, p.status, p.limit};
    if (threadIdx.x == 0) {
        abort_flag = 0;
        for (int i = 0; i < 2; ++i) {
            mbar_init(&q_full[i], 1);
            mbar_init(&q_empty[i], 1);
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 4);    // one arrival per warp
            mbar_init(&o_last[i], 1);
            mbar_init(&o_empty[i], 4);   // one arrival per warp
        }
        for (int i = 0; i < S; ++i) {
            mbar_init(&k_full[i], 1);
            mbar_init(&k_empty[i], 1);
            mbar_init(&v_full[i], 1);
            mbar_init(&v_empty[i], 1);
        }
        for (int i = 0; i < kItems; ++i) {
            mbar_init(&item_full[i], 1);
            mbar_init(&item_empty[i], kItemReaders);
        }
        mbar_init(&o_done, 1);
        mbar_init(&ml_full, 4);
        mbar_init(&ml_empty, 4);
        mbar_init(&mma_done, 1);
        fence_barrier_init();
    }
    if (warp == 10) {
        tmem_alloc(&tmem_slot, 512);
        tmem_relinquish();
    }
    if (threadIdx.x == 8 * 32) {
        tma_prefetch_desc(&qmany);
        tma_prefetch_desc(&qone);
        tma_prefetch_desc(&kmap);
        tma_prefetch_desc(&vmap);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    griddep_wait();   // the previous kernel of the stream has completed: global memory from here on

    // ---- the line of tiles: groups' common keys, then requests' own; entry e < N is a group, N + b a request
    const int B = p.B, N = p.N, cta = static_cast<int>(blockIdx.x);
    bool grouped;
    {
        // in the memory that the key tiles will take: groups' first requests, tiles and places on the line
        int* cu = reinterpret_cast<int*>(smem);
        int* tiles = cu + N + 1;
        int* place = tiles + N;
        bool bad = false, odd = false;
        for (int g = threadIdx.x; g <= N; g += blockDim.x) cu[g] = p.cu[g];
        __syncthreads();
        for (int g = threadIdx.x; g <= N; g += blockDim.x) bad = bad || cu[g] < 0 || cu[g] > B || (g > 0 ? cu[g] < cu[g - 1] : cu[g] != 0) || (g == N && cu[g] != B);
        grouped = !__syncthreads_or(bad);   // groups that are none: every request by itself
        // a run of groups and a run of requests per thread, then a scan over the threads
        const int per_g = (N + blockDim.x - 1) / blockDim.x, per_b = (B + blockDim.x - 1) / blockDim.x;
        const int g0 = min(N, static_cast<int>(threadIdx.x) * per_g), g1 = min(N, g0 + per_g);
        const int b0 = min(B, static_cast<int>(threadIdx.x) * per_b), b1 = min(B, b0 + per_b);
        int wg = 0, wb = 0, units = 0;
        for (int g = g0; g < g1; ++g) {
            int rt = 0, t = 0;
            if (grouped && cu[g + 1] > cu[g]) t = shared_tiles(p, cu[g], cu[g + 1], p.prefix[g], keys_of(p, cu[g]), rt);
            tiles[g] = t;
            wg += p.Hkv * rt * t;
            units += t ? p.Hkv * rt : 0;
        }
        __syncthreads();
        int g = grouped && b0 < b1 ? group_of(cu, N, b0) : 0;
        const int first_g = g;
        const auto own_tiles = [&](int b, int& g) {
            const int n = p.seqlens[b];
            odd = odd || n < 0 || n > p.cap;
            if (grouped)
                while (cu[g + 1] <= b) ++g;
            return max((min(max(n, 0), p.cap) + kTileKV - 1) / kTileKV - (grouped ? tiles[g] : 0), 0);
        };
        for (int b = b0; b < b1; ++b) {
            const int t = own_tiles(b, g);
            wb += p.Hkv * p.ch * t;
            units += t ? p.Hkv * p.ch : 0;
        }
        int ig = wg, ib = wb;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, ig, o), y = __shfl_up_sync(0xffffffffu, ib, o);
            if (lane >= o) {
                ig += x;
                ib += y;
            }
        }
        units = static_cast<int>(__reduce_add_sync(0xffffffffu, static_cast<unsigned>(units)));
        if (lane == 31) sums[warp] = make_int4(ig, ib, units, 0);
        __syncthreads();
        int tg = 0, tb = 0, before_g = 0, before_b = 0;
        units = 0;
        for (int w = 0; w < 12; ++w) {
            const int4 v = sums[w];
            before_g += w < warp ? v.x : 0;
            before_b += w < warp ? v.y : 0;
            tg += v.x;
            tb += v.y;
            units += v.z;
        }
        Line line;
        line.T = tg + tb;
        line.P = paged_ctas(line.T, units, static_cast<int>(gridDim.x));
        const int cut[2] = {line.cut(cta), line.cut(cta + 1)};
        // whoever has the entry that one of the CTA's two cuts falls in says so
        const auto owns = [&](int e, int s0, int nt, int n_units) {
#pragma unroll
            for (int k = 0; k < 2; ++k)
                if (cta < line.P && nt > 0 && s0 <= cut[k] && cut[k] < s0 + nt * n_units) {
                    const int i = (cut[k] - s0) / nt, s = s0 + i * nt, x = unit_cut(cut[k], s, s + nt);
                    Start r;
                    r.g = x;
                    r.b = e;
                    r.i = x == s + nt ? i + 1 : i;
                    r.t0 = x == s + nt ? 0 : x - s;
                    start_sh[k] = r;
                }
        };
        int at = before_g + ig - wg;
        for (int x = g0; x < g1; ++x) {
            const int rt = (cu[x + 1] - cu[x] + p.nb - 1) / max(p.nb, 1);
            place[x] = at;
            if (tiles[x]) {
                owns(x, at, tiles[x], p.Hkv * rt);
                at += p.Hkv * rt * tiles[x];
            }
        }
        __syncthreads();
        at = tg + before_b + ib - wb;
        g = first_g;
        for (int b = b0; b < b1; ++b) {
            const int t = own_tiles(b, g);
            owns(N + b, at, t, p.Hkv * p.ch);
            if (b % static_cast<int>(gridDim.x) == cta) {   // for the merge
                const int members = grouped ? cu[g + 1] - cu[g] : 1;
                p.plan[1 + 2 * b] = make_int4(grouped ? place[g] : 0, grouped ? tiles[g] : 0, (members + p.nb - 1) / max(p.nb, 1), members);
                p.plan[2 + 2 * b] = make_int4(at, t, grouped ? cu[g] : b, 0);
            }
            at += p.Hkv * p.ch * t;
        }
        if (threadIdx.x == 0) {
            if (cta == 0) p.plan[0] = make_int4(line.T, line.P, 0, 0);
            if (cta >= line.P || line.T == 0)
                start_sh[0] = start_sh[1] = Start{};
            else if (cta + 1 == line.P)
                start_sh[1].g = line.T;   // the cut behind the last tile
        }
        if (cta == 0 && (odd || !grouped)) report_bad_page(p.status);
        fence_proxy_async_smem();   // what was written here before key tiles land in it
        __syncthreads();
    }

    if (warp >= 8) {
        setmaxnreg_dec<kRegsCtl>();
        if (warp == 11) {
            // ------------------------------------------------ items, in the order of the line
            const Start first = start_sh[0];
            const int end = start_sh[1].g;
            Ring ir(kItems);
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
            for (int e = first.b; go && pos < end && e < N + B; e += 32) {
                // a lane looks at an entry
                const int x = e + lane;
                int nt = 0, b0 = 0, members = 1, rt = p.ch, n = 0, off = 0;
                if (x < N && grouped) {
                    b0 = p.cu[x];
                    members = p.cu[x + 1] - b0;
                    if (members > 0) {
                        n = keys_of(p, b0);
                        nt = shared_tiles(p, b0, b0 + members, p.prefix[x], n, rt);
                    }
                } else if (x >= N && x < N + B) {
                    b0 = x - N;
                    n = keys_of(p, b0);
                    if (grouped) {
                        const int g = group_of(p.cu, N, b0), f = p.cu[g];
                        int unused;
                        off = shared_tiles(p, f, p.cu[g + 1], p.prefix[g], keys_of(p, f), unused);
                    }
                    nt = max((n + kTileKV - 1) / kTileKV - off, 0);
                }
                for (int l = 0; l < 32 && go && pos < end; ++l) {
                    const int tiles = __shfl_sync(0xffffffffu, nt, l), row_tiles = __shfl_sync(0xffffffffu, rt, l);
                    const int fb = __shfl_sync(0xffffffffu, b0, l), m = __shfl_sync(0xffffffffu, members, l);
                    const int keys = __shfl_sync(0xffffffffu, n, l), skip = __shfl_sync(0xffffffffu, off, l);
                    const bool many = e + l < N;
                    if (tiles > 0) {
                        int head = i / row_tiles, r = i - head * row_tiles;
                        while (go && head < p.Hkv && pos < end) {
                            PrefixItem it;
                            it.t0 = skip + t0;
                            it.t1 = skip + min(tiles, end - pos + t0);
                            it.keys = keys;
                            it.trow = fb;
                            it.head = head;
                            if (many) {
                                it.b0 = fb + r * p.nb;
                                it.rows = min(p.nb, m - r * p.nb) * p.R;
                                it.rr0 = 0;
                                it.prow = (fb * p.Hkv + head * m + r * p.nb) * p.R + cta * kRows;
                                it.kind = kMany;
                            } else {
                                it.b0 = fb;
                                it.rr0 = r * kRows;
                                it.rows = min(p.Rt, p.R - it.rr0);
                                it.prow = (fb * p.Hkv + head) * p.R + it.rr0 + cta * p.Rt;
                                it.kind = p.out && skip == 0 && it.t1 - it.t0 == tiles ? kWhole : 0;
                            }
                            pos += it.t1 - it.t0;
                            t0 = 0;
                            if (++r == row_tiles) {
                                r = 0;
                                ++head;
                            }
                            go = emit(it);
                        }
                    }
                    i = 0;
                }
            }
            if (go) {
                PrefixItem it{};
                it.kind = kEnd;
                emit(it);
            }
        } else if (warp == 8 || warp == 9) {
            // ------------------------------------------------ TMA producers, as the paged ones of decode_kernel.cuh
            const int boxes = kTileKV >> p.box_log2;
            const bool is_k = warp == 8;
            const CUtensorMap* map = is_k ? &kmap : &vmap;
            uint64_t *full = is_k ? k_full : v_full, *empty = is_k ? k_empty : v_empty;
            uint8_t* ring = smem + (is_k ? C::kOffK : C::kOffV);
            const uint64_t pol = policy_evict_first();
            Ring ir(kItems), r(S);
            uint32_t cnt[S], qcnt[2] = {0, 0};
            for (int n = 0; n < S; ++n) cnt[n] = 0;
            uint32_t quse[2] = {0, 0}, qslot = 0;
            for (;;) {
                if (!__all_sync(0xffffffffu, mbar_wait(&item_full[ir.idx], ir.phase, wc))) break;
                const PrefixItem it = items[ir.idx];
                __syncwarp();
                if (lane == 0) mbar_arrive(&item_empty[ir.idx]);
                ir.advance();
                if (it.kind & kEnd) break;
                const bool many = it.kind & kMany;
                if (!is_k && lane == 0) {
                    // tiles of up to 64 rows take a half of the Q buffer in turns, larger ones both
                    const int rows = many ? p.nb * p.R : p.Rt;
                    const bool both = rows > 64;
                    const uint32_t s = both ? 0 : qslot;
                    mbar_wait(&q_empty[s], (quse[s] & 1) ^ 1, wc);
                    if (both) mbar_wait(&q_empty[1], (quse[1] & 1) ^ 1, wc);
                    if (!aborted(wc)) {
                        mbar_arrive_expect_tx(&q_full[s], static_cast<uint32_t>(rows * 128 * C::kAtoms));
                        for (int a = 0; a < C::kAtoms; ++a) {
                            uint8_t* dst = smem + C::kOffQ + a * (kRows * 128) + s * (64 * 128);
                            if (many)
                                tma_load_4d_hint(dst, &qmany, &q_full[s], a * 64, 0, it.head, it.b0, policy_evict_first());
                            else
                                tma_load_4d_hint(dst, &qone, &q_full[s], a * 64, it.rr0, it.head, it.b0, policy_evict_first());
                        }
                        ++qcnt[s];
                        if (both) {
                            mbar_arrive(&q_full[1]);
                            ++qcnt[1];
                        }
                    }
                    ++quse[s];
                    if (both) ++quse[1];
                    qslot = both ? 0 : s ^ 1;
                }
                __syncwarp();
                const int32_t* row = p.table + static_cast<size_t>(it.trow) * p.max_pages;
                // this lane's box of tile t starts at key first_key(t)
                const auto first_key = [&](int t) { return t * kTileKV + lane * p.box; };
                const auto look_up = [&](int t) {
                    const int j = first_key(t);
                    return t < it.t1 && lane < boxes && j < it.keys ? row[p.by_page.div(j)] : 0;
                };
                int next_page = look_up(it.t0);
                for (int t = it.t0; t < it.t1; ++t) {
                    int page = next_page;
                    next_page = look_up(t + 1);
                    const int j = first_key(t), off = j - p.by_page.div(j) * p.page;
                    const bool mine = lane < boxes && j < it.keys;
                    if (mine && (page < 0 || page >= p.num_pages)) {
                        page = p.num_pages;
                        report_bad_page(p.status);
                    }
                    const int used = (min(it.keys - t * kTileKV, kTileKV) + p.box - 1) >> p.box_log2;
                    int go = 0;
                    if (lane == 0) {
                        mbar_wait(&empty[r.idx], r.phase ^ 1, wc);
                        go = aborted(wc) ? 0 : 1;
                        if (go) mbar_arrive_expect_tx(&full[r.idx], static_cast<uint32_t>((used << p.box_log2) * 128 * C::kAtoms));
                    }
                    if (__shfl_sync(0xffffffffu, go, 0)) {
                        if (mine) {
                            uint8_t* dst = ring + r.idx * C::kKVBytes + lane * (p.box / 8) * L::kGroup;
                            if constexpr (L::kInter)
                                tma_load_5d_hint(dst, map, &full[r.idx], 0, 0, 0, page * p.groups + off / 8, it.head, pol);
                            else
                                tma_load_4d_hint(dst, map, &full[r.idx], 0, off, it.head, page, pol);
                        }
                        ++cnt[r.idx];
                    }
                    r.advance();
                }
            }
            // nothing may still be landing in shared memory when the CTA exits
            if (lane == 0) {
                for (int n = 0; n < S; ++n)
                    if (cnt[n]) drain_wait(&full[n], (cnt[n] - 1) & 1, kDrainLimit);
                for (int n = 0; n < 2; ++n)
                    if (qcnt[n]) drain_wait(&q_full[n], (qcnt[n] - 1) & 1, kDrainLimit);
            }
            __syncwarp();
        } else if (lane == 0) {
            // ------------------------------------------------ MMA issuer
            constexpr uint32_t idesc_qk = idesc_bf16_f32(kRows, kTileKV, false, false);
            constexpr uint32_t idesc_pv = idesc_bf16_f32(kRows, D, false, true);
            constexpr uint32_t lbo_v = D >= 128 ? L::kHalf : 0u;
            Ring ir(kItems), kr(S), vr(S), sr(2), pr(2), ob(2);
            uint32_t quse[2] = {0, 0}, qslot = 0;
            // the tile whose PV is still to be issued: QK of a tile goes ahead of PV of the one before, across items too
            bool behind = false, b_first = false, b_last = false;
            const auto pv = [&]() {
                mbar_wait(&p_full[pr.idx], pr.phase, wc);
                mbar_wait(&v_full[vr.idx], vr.phase, wc);
                if (b_first) mbar_wait(&o_empty[ob.idx], ob.phase ^ 1, wc);
                tc_fence_after();
                if (!aborted(wc)) {
                    const uint32_t sV = smem_u32(smem + C::kOffV + vr.idx * C::kKVBytes);
                    const uint32_t aP = tmem + C::col_s(pr.idx), dO = tmem + C::col_o(ob.idx);
#pragma unroll
                    for (int half = 0; half < 2; ++half)
#pragma unroll
                        for (int ks = 0; ks < kTileKV / 16; ++ks)
                            mma_ts(dO, aP + half * 64 + ks * 8, sdesc_sw128(sV + ks * 2 * L::kGroup, lbo_v, L::kGroup), idesc_pv,
                                   half > 0 || ks > 0 || !b_first ? 1u : 0u);
                    mma_commit(&v_empty[vr.idx]);
                    mma_commit(&o_done);
                    if (b_last) mma_commit(&o_last[ob.idx]);
                }
                pr.advance();
                vr.advance();
                if (b_last) ob.advance();
            };
            for (;;) {
                if (!mbar_wait(&item_full[ir.idx], ir.phase, wc)) break;
                const PrefixItem it = items[ir.idx];
                mbar_arrive(&item_empty[ir.idx]);
                ir.advance();
                if (it.kind & kEnd) break;
                const bool both = ((it.kind & kMany) ? p.nb * p.R : p.Rt) > 64;
                const uint32_t s = both ? 0 : qslot;
                mbar_wait(&q_full[s], quse[s] & 1, wc);
                if (both) mbar_wait(&q_full[1], quse[1] & 1, wc);
                const uint32_t sQ = smem_u32(smem + C::kOffQ + s * (64 * 128));
                for (int t = it.t0; t < it.t1; ++t) {
                    mbar_wait(&k_full[kr.idx], kr.phase, wc);
                    tc_fence_after();
                    if (!aborted(wc)) {
                        const uint32_t sK = smem_u32(smem + C::kOffK + kr.idx * C::kKVBytes);
                        const uint32_t dS = tmem + C::col_s(sr.idx);
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk)
                            mma_ss(dS, sdesc_sw128(sQ + (kk >> 2) * (kRows * 128) + (kk & 3) * 32, 16, 1024),
                                   sdesc_sw128(sK + (kk >> 2) * L::kHalf + (kk & 3) * 32, 16, L::kGroup), idesc_qk, kk > 0 ? 1u : 0u);
                        mma_commit(&s_full[sr.idx]);
                        mma_commit(&k_empty[kr.idx]);
                        if (t + 1 == it.t1) {
                            mma_commit(&q_empty[s]);
                            if (both) mma_commit(&q_empty[1]);
                        }
                    }
                    kr.advance();
                    sr.advance();
                    if (behind) pv();
                    behind = true;
                    b_first = t == it.t0;
                    b_last = t + 1 == it.t1;
                }
                ++quse[s];
                if (both) ++quse[1];
                qslot = both ? 0 : s ^ 1;
            }
            if (behind) pv();
            mma_commit(&mma_done);
            drain_wait(&mma_done, 0, kDrainLimit);
        }
    } else if (warp < 4) {
        setmaxnreg_inc<kRegsSm>();
        // ------------------------------------------------ softmax, a row per thread
        const int tid = threadIdx.x;
        const uint32_t lane_base = static_cast<uint32_t>(warp * 32) << 16;
        const int member = p.ch == 1 ? tid / p.R : 0, member_row = tid - member * p.R;   // of a tile of several requests
        Ring ir(kItems), sr(2), vr(S), ob(2), hr(1);
        uint32_t tiles_done = 0;
        for (;;) {
            if (!__all_sync(0xffffffffu, mbar_wait(&item_full[ir.idx], ir.phase, wc))) break;
            const PrefixItem it = items[ir.idx];
            __syncwarp();
            if (lane == 0) mbar_arrive(&item_empty[ir.idx]);
            ir.advance();
            if (it.kind & kEnd) break;
            const bool busy = warp * 32 < it.rows;   // of the other warps nothing is wanted
            int lim = 0;                             // keys that this row sees
            if (tid < it.rows) {
                const bool many = it.kind & kMany;
                const int rr = many ? member_row : it.rr0 + tid;
                lim = many ? keys_of(p, it.b0 + member) : it.keys;
                if (p.causal) lim += 1 - p.Sq + rr % p.Sq;
            }
            float m = -INFINITY, l = 0.f;
            for (int t = it.t0; t < it.t1; ++t, ++tiles_done) {
                mbar_wait(&s_full[sr.idx], sr.phase, wc);
                tc_fence_after();
                if (busy) {
                    const uint32_t tS = tmem + lane_base + C::col_s(sr.idx);
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
                    const bool up = mt > m + kRescaleD;
                    const float alpha = up ? ex2_approx(m - mt) : 1.f;
                    if (up) m = mt;
                    if (t > it.t0 && __any_sync(0xffffffffu, up)) {   // tcgen05.ld/st are warp-collective
                        mbar_wait(&o_done, (tiles_done - 1) & 1, wc);   // PV of the tile before
                        tc_fence_after();
                        __syncwarp();
                        const uint32_t tO = tmem + lane_base + C::col_o(ob.idx);
#pragma unroll 1
                        for (int c4 = 0; c4 < D / 16; ++c4) {
                            uint32_t o[16];
                            tmem_ld16(tO + c4 * 16, o);
                            tmem_ld_wait();
#pragma unroll
                            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
                            tmem_st16(tO + c4 * 16, o);
                        }
                    }
                    const uint64_t cc = f32x2(p.c, p.c);
                    const float mu = m == -INFINITY ? 0.f : -m;   // no visible key yet: -inf - 0
                    const uint64_t nm = f32x2(mu, mu);
                    uint64_t ls[4] = {0ull, 0ull, 0ull, 0ull};
                    __syncwarp();
#pragma unroll
                    for (int c = 0; c < kTileKV / 32; ++c) {
                        uint32_t hi[16], lo[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            float x0, x1;
                            f32x2_split(ffma2(f32x2(s[c * 32 + 2 * i], s[c * 32 + 2 * i + 1]), cc, nm), x0, x1);
                            const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
                            ls[i & 3] = fadd2(ls[i & 3], f32x2(p0, p1));
                            hi[i] = pack_bf16x2(p0, p1);
                            lo[i] = pack_bf16x2(p0 - __uint_as_float(hi[i] << 16), p1 - __uint_as_float(hi[i] & 0xffff0000u));
                        }
                        tmem_st16(tS + c * 16, hi);
                        tmem_st16(tS + 64 + c * 16, lo);
                    }
                    float la, lb;
                    f32x2_split(fadd2(fadd2(ls[0], ls[1]), fadd2(ls[2], ls[3])), la, lb);
                    l = fmaf(l, alpha, la + lb);
                }
                // Rows of V behind the last key may hold anything, and P = 0 does not cancel NaN in the MMA: zero them
                if ((t + 1) * kTileKV > it.keys) {
                    mbar_wait(&v_full[vr.idx], vr.phase, wc);
                    if (t * kTileKV + tid >= it.keys) {
                        uint8_t* rowp = smem + C::kOffV + vr.idx * C::kKVBytes + L::row(tid);
#pragma unroll
                        for (int a = 0; a < C::kAtoms; ++a)
#pragma unroll
                            for (int i = 0; i < 8; ++i) reinterpret_cast<uint4*>(rowp + a * L::kHalf)[i ^ (tid & 7)] = make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async_smem();
                }
                __syncwarp();
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[sr.idx]);
                sr.advance();
                vr.advance();
            }
            mbar_wait(&ml_empty, hr.phase ^ 1, wc);
            ml[tid] = make_float2(m, l);
            __syncwarp();
            if (lane == 0) mbar_arrive(&ml_full);
            hr.advance();
            ob.advance();
        }
    } else {
        setmaxnreg_inc<kRegsEpi>();
        // ------------------------------------------------ epilogue, a row per thread
        const int tid = threadIdx.x - 128;
        const uint32_t lane_base = static_cast<uint32_t>((warp - 4) * 32) << 16;
        Ring ir(kItems), ob(2), hr(1);
        for (;;) {
            if (!__all_sync(0xffffffffu, mbar_wait(&item_full[ir.idx], ir.phase, wc))) break;
            const PrefixItem it = items[ir.idx];
            __syncwarp();
            if (lane == 0) mbar_arrive(&item_empty[ir.idx]);
            ir.advance();
            if (it.kind & kEnd) break;
            mbar_wait(&ml_full, hr.phase, wc);
            const float2 v = ml[tid];
            __syncwarp();
            if (lane == 0) mbar_arrive(&ml_empty);
            hr.advance();
            mbar_wait(&o_last[ob.idx], ob.phase, wc);
            tc_fence_after();
            __syncwarp();
            if ((warp - 4) * 32 < it.rows) {
                const bool none = v.y == 0.f;   // no visible key; a NaN score makes the sum, the row and its LSE NaN
                const float inv = none ? 0.f : 1.f / v.y, lse = none ? -INFINITY : (v.x + __log2f(v.y)) * kLn2;
                const bool store = tid < it.rows && !aborted(wc);
                const size_t orow = (static_cast<size_t>(it.b0) * p.Hkv + it.head) * p.R + it.rr0 + tid;
                const size_t prow = static_cast<size_t>((it.kind & kMany) ? 0 : p.own_rows) + it.prow + tid;
                const bool whole = it.kind & kWhole;
#pragma unroll
                for (int c4 = 0; c4 < D / 32; ++c4) {
                    uint32_t o[32];
                    tmem_ld32p(tmem + lane_base + C::col_o(ob.idx) + c4 * 32, o);
                    tmem_ld_wait();
                    float x[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) x[i] = none ? 0.f : __uint_as_float(o[i]) * inv;
                    if (store && whole && !p.out_f32) {
                        uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + orow * D + c4 * 32);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            dst[i] = make_uint4(pack_bf16x2(x[8 * i], x[8 * i + 1]), pack_bf16x2(x[8 * i + 2], x[8 * i + 3]),
                                                pack_bf16x2(x[8 * i + 4], x[8 * i + 5]), pack_bf16x2(x[8 * i + 6], x[8 * i + 7]));
                    } else if (store && whole) {
                        float4* dst = reinterpret_cast<float4*>(static_cast<float*>(p.out) + orow * D + c4 * 32);
#pragma unroll
                        for (int i = 0; i < 8; ++i) dst[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
                    } else if (store) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) st_global_v8(p.part_o + prow * D + c4 * 32 + 8 * i, x + 8 * i);
                    }
                }
                if (store && !whole) p.part_lse[prow] = lse;
                if (store && whole && p.lse) p.lse[orow] = lse;
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&o_empty[ob.idx]);
            ob.advance();
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 10) tmem_dealloc(tmem, 512);
}

// Merges the partials of a row, a warp each: the pieces of its group's common keys and of its own.
template <int D>
__global__ void __launch_bounds__(256) prefix_merge_kernel(const __grid_constant__ PrefixParams p, int rows)
{
    constexpr int V = D / 32;   // features of a lane
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31, row = blockIdx.x * 8 + threadIdx.x / 32;
    if (row >= rows) return;
    const int unit = row / p.R, rr = row - unit * p.R, b = unit / p.Hkv, h = unit - b * p.Hkv;
    const int4 head = p.plan[0], g = p.plan[1 + 2 * b], o = p.plan[2 + 2 * b];
    Line line;
    line.T = head.x;
    line.P = head.y;

    float m = -INFINITY, l = 0.f, acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.f;
    int pieces = 0;
    // the pieces of the unit of tiles [s, e); that of CTA c has this row at first + c * step
    const auto merge = [&](int s, int e, long long first, int step) {
        int c0 = max(min(static_cast<int>(static_cast<float>(s) * (static_cast<float>(line.P) / static_cast<float>(line.T))), line.P - 1), 0);
        while (c0 > 0 && line.cut(c0) > s) --c0;
        while (c0 + 1 < line.P && line.cut(c0 + 1) <= s) ++c0;
        c0 = max(c0 - 1, 0);   // a cut behind s may have moved back to it
        for (; c0 < line.P && unit_cut(line.cut(c0), s, e) < e; c0 += 32) {
            const int c = c0 + lane;
            const bool has = c < line.P && unit_cut(line.cut(c), s, e) < unit_cut(line.cut(c + 1), s, e);
            const unsigned which = __ballot_sync(0xffffffffu, has);
            if (!which) continue;
            pieces += __popc(which);
            const float x = has ? __ldcg(p.part_lse + first + static_cast<long long>(c) * step) : -INFINITY;
            const float top = fmax_nan(m, redux_max_nan(x));
            if (top == -INFINITY) continue;   // no visible key so far
            const float keep = m == -INFINITY ? 0.f : __expf(m - top), w = has ? __expf(x - top) : 0.f;
            m = top;
            l = l * keep + warp_sum(w);
#pragma unroll
            for (int i = 0; i < V; ++i) acc[i] *= keep;
            const int k0 = __ffs(which) - 1, n = __popc(which);   // pieces of neighbouring CTAs
#pragma unroll 4
            for (int k = k0; k < k0 + n; ++k) {
                const float* src = p.part_o + (first + static_cast<long long>(c0 + k) * step) * D + lane * V;
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
    };
    if (g.y > 0) {   // (place, tiles, row tiles, requests) of the group; R <= 64
        const int mem = b - o.z, r = mem / p.nb, s = g.x + (h * g.z + r) * g.y;
        merge(s, s + g.y, static_cast<long long>(o.z * p.Hkv + h * g.w + mem) * p.R + rr, kRows);
    }
    if (o.y > 0) {
        const int chunk = rr / kRows, s = o.x + (h * p.ch + chunk) * o.y;
        merge(s, s + o.y, p.own_rows + row, p.Rt);
    }
    if (p.out && g.y == 0 && pieces == 1) return;   // one item was all of it and wrote the row
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
    size_t plan_off, lse_off, o_off, stage_off, amax_off, total;
    long long own_rows;
};

PrefixWs prefix_ws(int B, int Hq, int Sq, const fmha_kv_cache* c, const fmha_opts* o)
{
    const auto al = [](size_t x) { return (x + 255) & ~size_t(255); };
    PrefixWs w{};
    const size_t rows = static_cast<size_t>(B) * Hq * Sq;
    if (rows == 0) return w;
    const size_t nsm = num_sms() > 0 ? num_sms() : 256;   // sized for the largest plausible SM count
    const size_t R = static_cast<size_t>(Hq / c->Hkv) * Sq;
    w.own_rows = R <= kRows / 2 ? static_cast<long long>(rows + nsm * kRows) : 0;
    const size_t parts = static_cast<size_t>(w.own_rows) + rows + nsm * (R < kRows ? R : kRows);
    w.plan_off = 0;
    w.lse_off = al((1 + 2 * static_cast<size_t>(B)) * sizeof(int4));
    w.o_off = w.lse_off + al(parts * 4);
    w.stage_off = w.o_off + al(parts * c->D * 4);
    const bool nvfp4 = o && o->out_kind == FMHA_OUT_NVFP4;
    w.amax_off = w.stage_off + (nvfp4 && !o->out_f32 ? al(rows * c->D * 4) : 0);
    w.total = w.amax_off + (nvfp4 ? 256 : 0);
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
    if (cap > (1LL << 31) - 256 || rows >= (1LL << 30) || B > (1 << 24))
        return set_error(FMHA_ERR_UNSUPPORTED, who + ": max_pages * page_size past 2^31, 2^30 rows or 2^24 requests");
    const long long units = static_cast<long long>(B) * c->Hkv * ((static_cast<long long>(Hq / c->Hkv) * Sq + kRows - 1) / kRows);
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
int run_prefix(PrefixParams& p, const void* q, const fmha_kv_cache* c, int rows, cudaStream_t st)
{
    using C = PrefixCfg<D>;
    CUtensorMap qmany, qone, kmap, vmap;
    const uint64_t dims[4] = {static_cast<uint64_t>(D), static_cast<uint64_t>(p.R), static_cast<uint64_t>(p.Hkv), static_cast<uint64_t>(p.B)};
    const uint64_t strides[3] = {static_cast<uint64_t>(D) * 2, static_cast<uint64_t>(p.R) * D * 2, static_cast<uint64_t>(p.Hkv) * p.R * D * 2};
    const uint32_t many[4] = {64, static_cast<uint32_t>(p.Rt), 1, static_cast<uint32_t>(p.nb > 1 ? p.nb : 1)}, one[4] = {64, static_cast<uint32_t>(p.Rt), 1, 1};
    int rc = make_tmap_bf16(&qmany, q, 4, dims, strides, many);
    if (!rc) rc = make_tmap_bf16(&qone, q, 4, dims, strides, one);
    if (!rc) rc = make_pool_map(&kmap, c->k, c, p.box);
    if (!rc) rc = make_pool_map(&vmap, c->v, c, p.box);
    if (rc) return rc;
    const int nsm = num_sms();
    if (nsm <= 0) return set_error(FMHA_ERR_CUDA, "cannot query the SM count");
    const long long tiles = static_cast<long long>(p.B) * p.Hkv * p.ch * ((static_cast<long long>(p.cap) + kTileKV - 1) / kTileKV);
    const unsigned grid = static_cast<unsigned>(tiles < nsm ? tiles : nsm);
    FMHA_CHECK_CUDA(set_smem_limit_once(reinterpret_cast<const void*>(prefix_kernel<D>), C::kSmemBytes));
    timing_mark_begin(st);
    const cudaError_t e = launch_pdl(prefix_kernel<D>, dim3(grid), dim3(384), static_cast<size_t>(C::kSmemBytes), st, qmany, qone, kmap, vmap, p);
    timing_mark_end(st);
    FMHA_CHECK_CUDA(e);
    count_launch();
    FMHA_CHECK_CUDA(launch_pdl(prefix_merge_kernel<D>, dim3(static_cast<unsigned>((rows + 7) / 8)), dim3(256), 0, st, p, rows));
    count_launch();
    return FMHA_OK;
}

}  // namespace
}  // namespace atc_gb300

using namespace atc_gb300;

extern "C" size_t fmha_prefix_workspace_size(int B, int Hq, int Sq, const fmha_kv_cache* cache, const fmha_opts* opts)
{
    if (!cache || cache->Hkv < 1 || B < 0 || Hq <= 0 || Sq < 0 || Hq % cache->Hkv || (cache->D != 64 && cache->D != 128) ||
        static_cast<long long>(B) * Hq * Sq >= (1LL << 30))
        return 0;
    return prefix_ws(B, Hq, Sq, cache, opts).total;
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
    const PrefixWs w = prefix_ws(B, Hq, Sq, cache, &o);
    if (w.total > 0 && (!o.workspace || o.workspace_bytes < w.total))
        return set_error(FMHA_ERR_WORKSPACE, "fmha_fwd_prefix: workspace missing or smaller than fmha_prefix_workspace_size()");
    if (empty) return FMHA_OK;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    uint8_t* base = static_cast<uint8_t*>(o.workspace);
    const int rows = B * Hq * Sq;

    PrefixParams p{};
    p.B = B;
    p.N = N;
    p.Hkv = cache->Hkv;
    p.R = Hq / cache->Hkv * Sq;
    p.Sq = Sq;
    p.Rt = p.R < kRows ? p.R : kRows;
    p.ch = (p.R + kRows - 1) / kRows;
    p.nb = kRows / p.Rt;
    p.causal = o.causal && Sq > 1;   // one query sees every key either way
    p.c = scale * kLog2e;
    p.cu = cu_groups;
    p.prefix = prefix_lens;
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
    p.out = nvfp4 ? nullptr : out;
    p.out_f32 = o.out_kind == FMHA_OUT_F32 ? 1 : 0;
    p.lse = lse;
    p.plan = reinterpret_cast<int4*>(base + w.plan_off);
    p.part_lse = reinterpret_cast<float*>(base + w.lse_off);
    p.part_o = reinterpret_cast<float*>(base + w.o_off);
    p.own_rows = w.own_rows;
    p.status = device_status_ptr();
    p.limit = wait_limit();
    if (nvfp4) {
        p.o_stage = o.out_f32 ? o.out_f32 : reinterpret_cast<float*>(base + w.stage_off);
        p.amax_bits = o.out_amax ? reinterpret_cast<unsigned*>(o.out_amax) : reinterpret_cast<unsigned*>(base + w.amax_off);
        FMHA_CHECK_CUDA(cudaMemsetAsync(p.amax_bits, 0, sizeof(unsigned), st));
    }
    rc = cache->D == 64 ? run_prefix<64>(p, q, cache, rows, st) : run_prefix<128>(p, q, cache, rows, st);
    if (rc || !nvfp4) return rc;
    return launch_nvfp4(p.o_stage, static_cast<uint8_t*>(out), o.out_scales, o.out_tensor_scale, p.amax_bits,
                        static_cast<int64_t>(rows) * cache->D, true, st, o.nvfp4_scale_in);
}
