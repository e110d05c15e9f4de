// Attention of requests that share their first pages (fmha_fwd_prefix): each group's common keys are read
// once for all its requests.
//
//   o_b = softmax(scale q_b K_b^T) V_b as in fmha_fwd_paged.  With the keys of request b in disjoint sets C_1, C_2, ..
//   and O_i, lse_i the attention over C_i alone:   lse = log sum_i exp(lse_i),   o_b = sum_i exp(lse_i - lse) O_i
//
// so a group's common keys, in whole tiles of 128, are a problem whose rows are the queries of all its requests
// (prefix_body), what is left of each request is a decode problem (decode_body), and a second kernel merges a row's partials
// (prefix.cu).  Per key/value head a request has R = (Hq / Hkv) Sq rows.
//
//  * One launch for both kinds of keys, a CTA per SM: the first CTAs take common keys, which the tensor cores and the softmax
//    bound, the others own keys, which memory bounds, as many of either as their work's share.  Lengths are on the device, so
//    every CTA sums the groups and the requests itself (make_plan).
//  * Work split.  The key tiles of all problems of a kind (group, kv-head and pair of row tiles; request and kv-head) are laid end to end
//    and cut for the CTAs (as in decode_kernel.cuh), by what they cost (prefix_split.cuh); what is not a request's whole attention goes to the workspace as
//    normalised partials.
//
// Common keys:
//  * Row tiles.  S = Q K^T with M = 128 query rows: floor(128 / R) requests of a group.  A row is a thread's (Tensor
//    Memory lane), so maxima and sums need no other thread.
//  * A CTA has two softmax warpgroups ("sides"), each with its own S, P and O in Tensor Memory and its own running
//    maximum and sum.  With more than 128 rows in the group they take two row tiles, over the same key tiles; else the same rows
//    over every other key tile.  While one computes exponentials the tensor core runs the other's products.
//  * P goes to the tensor core as two BF16, the rounded weight (half a step, 2^-9) and what the rounding left, both over the
//    S that they come from (16 keys' scores become 8 columns of pairs of either), in an MMA each: P is good to 2^-17
//    as in fmha_fwd_paged, and the output's rounding is the only one that shows.
//  * Long pieces.  The tensor core cuts off what its sums have no bits for: C products added up (an MMA each, 16 a tile) may lose
//    C 2^-23 of sum p |v|, always towards zero (values of 1, 1024 tiles: 4e-4).  So a side's accumulator takes at most kChain
//    tiles, 2^-13 of it, and what follows of a piece is merged with its partials by the threads that stored them (a part more
//    costs 3 to 7 us: 4 groups of 64 behind 32768 keys, in pieces of 85 tiles, 275 us a call for 268).
//  * Roles: warps 0-3 and 4-7 the sides, 8 K, 9 Q and V, 10 MMA (a warp for each side's products measured slower: 1.58 us a
//    tile of 128 rows and keys against 1.32), 11 finds the pieces and hands them to the others through a ring in shared
//    memory.  Every wait is bounded, as in decode_kernel.cuh.
#pragma once
#include <cuda_runtime.h>

#include "paged_run.cuh"
#include "prefix.h"
#include "prefix_split.cuh"

namespace atc_gb300 {
namespace {

constexpr int kItems = 4;           // slots of the item ring
constexpr int kItemReaders = 11;    // K, V and MMA warps, eight softmax warps
constexpr int kPrefixThreads = 384;
constexpr int kChain = 64;          // key tiles that an accumulator takes: 1024 MMAs
static_assert(kPrefixThreads == decode_threads<true>(), "common and own keys in one launch");
// registers: two softmax warpgroups and the control warpgroup, 2 * 208 + 88 = 504 of an SM quarter's 512
constexpr uint32_t kRegsSide = 208;
static_assert(128 * (2 * kRegsSide + kRegsCtl) <= kPrefixThreads * 168, "register split exceeds the launch allocation");

// Tiles of keys that the requests [b0, b1) of a group read together.  n0: keys of the first one, through whose row
// they are read.  None, unless what each request would take for them is more than what they take together and in the merge.
template <int D>
__device__ __forceinline__ int shared_tiles(const Groups& gr, int b0, int b1, int prefix, int n0)
{
    using K = Cost<D>;
    const int members = b1 - b0;
    if (members < 2) return 0;
    const int tiles = min(max(prefix, 0), n0) / kTileKV;
    const long long alone = static_cast<long long>(members) * gr.chunks * tiles * K::kAgain,
                    together = static_cast<long long>(row_pairs(members, gr.nb)) * K::common(members > gr.nb).of(tiles) + static_cast<long long>(members) * gr.R * K::kMerge;
    return alone > together ? tiles : 0;
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
template <int D, typename Keys>
__device__ __forceinline__ bool load_groups(const Groups& gr, int B, int* cu, int* tiles, Keys&& keys)
{
    bool bad = false;
    for (int g = threadIdx.x; g <= gr.n; g += blockDim.x) cu[g] = gr.cu[g];
    __syncthreads();
    for (int g = threadIdx.x; g <= gr.n; g += blockDim.x)
        bad = bad || cu[g] < 0 || cu[g] > B || (g > 0 ? cu[g] < cu[g - 1] : cu[g] != 0) || (g == gr.n && cu[g] != B);
    const bool grouped = !__syncthreads_or(bad);
    for (int g = threadIdx.x; g < gr.n; g += blockDim.x)
        tiles[g] = grouped && cu[g + 1] > cu[g] ? shared_tiles<D>(gr, cu[g], cu[g + 1], gr.prefix[g], keys(cu[g])) : 0;
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

// Dynamic shared memory of a launch: of common keys, or of own keys with what the decode kernel has beside its tiles
template <int D, int NC>
constexpr int prefix_smem()
{
    const int own = ((DecodeCfg<D>::smem_bytes(NC, true) + 15) & ~15) + static_cast<int>(sizeof(DecodeShared<D, true>));
    return PrefixCfg<D>::kSmemBytes > own ? PrefixCfg<D>::kSmemBytes : own;
}

__device__ __forceinline__ int keys_of(const PrefixParams& p, int b) { return min(max(p.seqlens[b], 0), p.cap); }

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

// A piece of a problem, or a part of a long one
struct PrefixItem {
    int t0, t1;      // tiles of keys (none: no more pieces)
    int trow, head;  // row of the block table: the group's first request
    int b0, rows;    // first request of the first row tile, and rows of both
    int prow;        // first row of the partials
    bool again;      // which hold the piece's earlier tiles
};

template <int D>
struct PrefixShared {
    static constexpr int SK = PrefixCfg<D>::kStagesK, SV = PrefixCfg<D>::kStagesV;
    uint64_t q_full, q_empty, k_full[SK], k_empty[SK], v_full[SV], v_empty[SV];
    // of each side: S is ready; P is stored over it; a piece's last PV is done; O has been read.  A QK needs no barrier for its
    // S: the MMA warp issues it behind the PV that read the P there.  So S of a side's next tile says that PV of the last one is
    // done, too.
    uint64_t s_full[2], p_full[2], o_done[2], o_empty[2], mma_done;
    uint64_t item_full[kItems], item_empty[kItems];
    PrefixItem items[kItems];
    int abort_flag;
};

// Common keys: CTA `cta`'s part of the line, from `first` up to tile `end`
template <int D>
__device__ __forceinline__ void prefix_body(const CUtensorMap& qmap, const CUtensorMap& kmap, const CUtensorMap& vmap, const PrefixParams& p,
                                            PrefixShared<D>& sh, uint8_t* smem, int cta, const Start& first, int end, uint32_t tmem)
{
    using C = PrefixCfg<D>;
    using L = TileLayout<D, true>;
    constexpr int SK = C::kStagesK, SV = C::kStagesV;
    auto &k_full = sh.k_full, &k_empty = sh.k_empty;
    auto &v_full = sh.v_full, &v_empty = sh.v_empty;
    auto &s_full = sh.s_full, &p_full = sh.p_full, &o_done = sh.o_done, &o_empty = sh.o_empty;
    auto &item_full = sh.item_full, &item_empty = sh.item_empty;
    auto& items = sh.items;
    uint64_t &q_full = sh.q_full, &q_empty = sh.q_empty, &mma_done = sh.mma_done;
    int& abort_flag = sh.abort_flag;
    const int warp = threadIdx.x / 32, lane = static_cast<int>(threadIdx.x) & 31, N = p.gr.n;
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
    if (threadIdx.x == 8 * 32) {
        tma_prefetch_desc(&qmap);
        tma_prefetch_desc(&kmap);
        tma_prefetch_desc(&vmap);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
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
            for (int g0 = first.b; go && pos < end && g0 < N; g0 += 32) {
                const int g = g0 + lane;   // a lane looks at a group
                int nt = 0, b0 = 0, members = 0;
                if (g < N) {
                    b0 = p.gr.cu[g];
                    members = p.gr.cu[g + 1] - b0;
                    if (members > 0) nt = shared_tiles<D>(p.gr, b0, b0 + members, p.gr.prefix[g], keys_of(p, b0));
                }
                for (int l = 0; l < 32 && go && pos < end; ++l) {
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
                            it.again = false;
                            pos += it.t1 - it.t0;
                            t0 = 0;
                            if (++r == pairs) {
                                r = 0;
                                ++head;
                            }
                            // in parts of one length, if it is long (of one row tile the sides take every other key tile)
                            const int last = it.t1, n = last - it.t0, most = it.rows > tile_rows ? kChain : 2 * kChain, parts = (n + most - 1) / most;
                            const int each = (n + parts - 1) / parts;
                            do {
                                it.t1 = min(last, it.t0 + each);
                                go = emit(it);
                                it.t0 = it.t1;
                                it.again = true;
                            } while (go && it.t0 < last);
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
            PrefixItem it{0, 0, 0, 0, 0, 2 * kRows, 0, false};
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
                    tmem_ld_wait<kTileKV>(su);
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
                            tmem_ld_wait(o);
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
                float inv = none ? 0.f : 1.f / l, lse = none ? -INFINITY : (m + __log2f(l)) * kLn2;
                const bool store = tid < rows && !aborted(wc);
                const size_t row = static_cast<size_t>(it.prow) + (side ? (two ? tile_rows : it.rows) : 0) + tid;
                const bool merge = it.again && store;
                float keep = 0.f;   // the weight of the partials that are there
                if (merge) {
                    const float before = ld_global(p.part_lse + row), top = fmax_nan(before, lse);
                    if (top != -INFINITY) {
                        const float wb = __expf(before - top), w = __expf(lse - top), sum = wb + w;
                        keep = wb / sum;
                        inv *= w / sum;
                        lse = top + __logf(sum);
                    }
                }
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                    uint32_t o[32];
                    __syncwarp();   // tcgen05.ld is warp-collective, and rows that are none have left others to their partials
                    if (any) {
                        tmem_ld32(tO + c, o);
                        tmem_ld_wait(o);
                    }
                    float x[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) x[i] = none || !any ? 0.f : __uint_as_float(o[i]) * inv;
                    if (merge)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            float y[8];
                            ld_global_v8(y, p.part_o + row * D + c + 8 * i);
#pragma unroll
                            for (int k = 0; k < 8; ++k) x[8 * i + k] = fmaf(keep, y[k], x[8 * i + k]);
                        }
                    if (store)
#pragma unroll
                        for (int i = 0; i < 4; ++i) st_global_v8(p.part_o + row * D + c + 8 * i, x + 8 * i);
                }
                if (store) p.part_lse[row] = lse;
            }
            if (any) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&o_empty[side]);
            }
            k_pos += it.t1 - it.t0;
        }
    }

}


// ---- the work split ----------------------------------------------------------------------------------------
// What the launch's CTAs find out, each by itself, from the lengths: the common keys' line of tiles and its CTAs, the first of
// the launch; the own keys' line and its CTAs, the others.  first and end count tiles.
struct Plan {
    Line common, own;   // of costs (UnitCost)
    int border;    // CTAs below take common keys
    Start first;   // of this CTA's part of its line
    int end;
};

// x of n CTAs such that common / x + d = own / (n - x): both kinds end at the same time
__device__ __forceinline__ float common_share(float n, float common, float own, float d)
{
    const float h = d * n - common - own;
    return __fdividef(h + __fsqrt_rn(h * h + 4.f * d * common * n), 2.f * d);
}

// By the whole CTA.  scratch: 3 N + 1 ints; pre, keys: B + 1 and B ints of shared memory, or NULL (then the prefix is global)
template <int D>
__device__ __forceinline__ void make_plan(const PrefixParams& p, int* scratch, int* pre, int* keys, int4* sums, int4* sums2, Start* start_sh, Plan& out)
{
    const int B = p.B, N = p.gr.n, tid = static_cast<int>(threadIdx.x), lane = tid & 31, warp = tid >> 5;
    const int cta = static_cast<int>(blockIdx.x), ctas = static_cast<int>(gridDim.x);
    int *cu = scratch, *tiles = cu + N + 1, *place = tiles + N;
    // a run of groups and a run of requests per thread, then a scan over the threads; the lengths come in while the groups do
    const int per_g = (N + kPrefixThreads - 1) / kPrefixThreads, g0 = min(N, tid * per_g), g1 = min(N, g0 + per_g);
    const int per_b = (B + kPrefixThreads - 1) / kPrefixThreads, b0 = min(B, tid * per_b), b1 = min(B, b0 + per_b);
    const int len0 = b0 < b1 ? p.seqlens[b0] : 0;
    const bool grouped = load_groups<D>(p.gr, B, cu, tiles, [&](int b) { return keys_of(p, b); });
    const UnitCost own = p.weigh ? Cost<D>::own(p.R > 8) : UnitCost{};
    UnitCost one = Cost<D>::common(false), two = Cost<D>::common(true);
    if (!p.weigh) {
        one.tile = two.tile = 1;
        one.start = two.start = 0;
    }
    const auto units_of = [&](int g) { return p.Hkv * row_pairs(cu[g + 1] - cu[g], p.gr.nb); };
    const auto cost_of_kind = [&](int kind) { return kind & 1 ? two : one; };
    const auto cost_of = [&](int g) { return cost_of_kind(cu[g + 1] - cu[g] > p.gr.nb ? 1 : 0); };
    const int g_first = grouped && b0 < b1 ? group_of(cu, N, b0) : 0;
    const auto length = [&](int b) { return b == b0 ? len0 : p.seqlens[b]; };
    const auto own_tiles = [&](int b, int& g) {   // and g becomes b's group
        if (grouped)
            while (cu[g + 1] <= b) ++g;
        return max((min(max(length(b), 0), p.cap) + kTileKV - 1) / kTileKV - (grouped ? tiles[g] : 0), 0);
    };
    // each thread's sums: tiles, costs and units of common keys, tiles and requests of own ones
    int wg = 0, cg = 0, units = 0, wb = 0, with_keys = 0, g = g_first, most = 0, least = INT32_MAX;
    bool odd = !grouped;
    for (int x = g0; x < g1; ++x) {
        if (tiles[x] == 0) continue;
        units += units_of(x);
        const int kind = 2 * tiles[x] + (cu[x + 1] - cu[x] > p.gr.nb ? 1 : 0);
        most = max(most, kind);
        least = min(least, kind);
        wg += units_of(x) * tiles[x];
        cg += units_of(x) * cost_of(x).of(tiles[x]);
    }
    for (int b = b0; b < b1; ++b) {
        const int n = length(b), t = own_tiles(b, g);
        odd = odd || n < 0 || n > p.cap;
        if (keys) keys[b] = min(max(n, 0), p.cap);
        wb += t;
        with_keys += t > 0 ? 1 : 0;
    }
    const int ig = warp_scan_inc(wg), ic = warp_scan_inc(cg), ib = warp_scan_inc(wb), ik = warp_scan_inc(with_keys);
    units = static_cast<int>(__reduce_add_sync(0xffffffffu, static_cast<unsigned>(units)));
    most = __reduce_max_sync(0xffffffffu, most);
    least = __reduce_min_sync(0xffffffffu, least);
    if (lane == 31) {
        sums[warp] = make_int4(ig, ic, ib, ik);
        sums2[warp] = make_int4(units, most, least, 0);
    }
    if (tid == 0) start_sh[0] = start_sh[1] = Start{};
    __syncthreads();
    // a lane per warp
    const bool is_warp = lane < kPrefixThreads / 32, is_before = lane < warp;
    const int4 v = is_warp ? sums[lane] : make_int4(0, 0, 0, 0), u = is_warp ? sums2[lane] : make_int4(0, 0, INT32_MAX, 0);
    const auto sum = [](int x) { return static_cast<int>(__reduce_add_sync(0xffffffffu, static_cast<unsigned>(x))); };
    const int shared = sum(v.x), total = sum(v.z);
    int at_g = ig - wg + sum(is_before ? v.x : 0), at_c = ic - cg + sum(is_before ? v.y : 0), at_b = ib - wb + sum(is_before ? v.z : 0),
        at_k = ik - with_keys + sum(is_before ? v.w : 0);
    out.common.T = sum(v.y);
    with_keys = sum(v.w);
    units = sum(u.x);
    most = __reduce_max_sync(0xffffffffu, u.y);
    least = __reduce_min_sync(0xffffffffu, u.z);
    out.own.T = p.rest_units * (own.start * with_keys + own.tile * total);
    // the CTAs of common keys, in pairs (see prefix_kernel)
    out.border = out.common.P = 0;
    bool even = false;
    if (shared > 0) {
        using K = Cost<D>;
        const int room = total > 0 ? (ctas & ~1) - 2 : ctas;
        const float n = static_cast<float>(ctas), scale = p.weigh ? 1.f : static_cast<float>(K::own(p.R > 8).tile),
                    C = scale * static_cast<float>(out.common.T), O = scale * static_cast<float>(out.own.T);
        float x = n;
        if (total > 0) {
            // both kinds end at the same time, and common keys not before memory has given all
            x = common_share(n, C, O, K::start(most & 1));
            x = fminf(x, __fdividef(C, fmaxf(K::kRead * (static_cast<float>(shared) + static_cast<float>(total) * static_cast<float>(p.rest_units)) - K::kFirst, 1.f)));
        }
        const int fewest = cost_of_kind(most).least;   // tiles that a CTA may have
        x = fminf(x, static_cast<float>(max(shared / fewest, units)));
        int P = min(max(2 * static_cast<int>(x * 0.5f + 0.5f), 2), room);
        // units that are all the same: as many CTAs for each, if what that moves x by costs less than units cut across
        if (most == least && p.weigh) {
            const int k = min(min(static_cast<int>(__fdividef(x, static_cast<float>(units)) + 0.5f), room / units), max((most >> 1) / fewest, 1));
            const float off = fabsf(static_cast<float>(k * units) - x), y = fmaxf(n - x, 1.f);
            even = k > 0 && off * fmaxf(__fdividef(C, x * x), __fdividef(O, y * y)) < static_cast<float>(cost_of_kind(most).start);
            if (even) P = k * units;
        }
        out.common.P = P;
        out.border = (P + 1) & ~1;
        if (even) {
            one.tile = two.tile = 1;
            one.start = two.start = 0;
            out.common.T = shared;
            at_c = at_g;
        }
    }
    out.own.P = paged_ctas(total * p.rest_units, with_keys * p.rest_units, max(ctas - out.border, 1));
    // whoever has the entry that one of the CTA's two cuts falls in says so
    const bool common = cta < out.border;
    const Line& line = common ? out.common : out.own;
    const int c = common ? cta : cta - out.border;
    const bool works = c < line.P && line.T > 0;
    const int cut[2] = {works ? line.cut(c) : 0, works ? line.cut(c + 1) : 0};
    const auto owns = [&](int e, int at, int tile0, UnitCost u, int nt, int n) {   // entry e: n units of nt tiles from tile0 on, at `at` of the line
        const int of = u.of(nt);
        const bool has[2] = {works && at <= cut[0] && cut[0] < at + of * n, works && at <= cut[1] && cut[1] < at + of * n};
        if (!has[0] && !has[1]) return;
        int i[2], x[2];   // of both, so that the divisions run beside one another
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const unsigned off = has[k] ? static_cast<unsigned>(cut[k] - at) : 0u;
            i[k] = static_cast<int>(off / static_cast<unsigned>(of));
            x[k] = tile_at(static_cast<int>(off) - i[k] * of, nt, u);
        }
#pragma unroll
        for (int k = 0; k < 2; ++k)
            if (has[k]) {
                Start r;
                r.g = tile0 + i[k] * nt + x[k];
                r.b = e;
                r.i = x[k] == nt ? i[k] + 1 : i[k];
                r.t0 = x[k] == nt ? 0 : x[k];
                start_sh[k] = r;
            }
    };
    for (int x = g0; x < g1; ++x) {
        place[x] = at_c;
        if (tiles[x] == 0) continue;
        if (common) owns(x, at_c, at_g, cost_of(x), tiles[x], units_of(x));
        at_g += units_of(x) * tiles[x];
        at_c += units_of(x) * cost_of(x).of(tiles[x]);
    }
    // f(b, place of request b on the line, its tiles and those before it, its group)
    const auto requests = [&](auto&& f) {
        int g = g_first, tile = at_b, unit = at_k;
        for (int b = b0; b < b1; ++b) {
            const int t = own_tiles(b, g);
            f(b, p.rest_units * (own.start * unit + own.tile * tile), t, tile, g);
            tile += t;
            unit += t > 0 ? 1 : 0;
        }
    };
    if (!common || !pre)
        requests([&](int b, int at, int t, int tile, int) {
            if (!common && t > 0) owns(b, at, tile * p.rest_units, own, t, p.rest_units);
            (pre ? pre : p.rest_prefix)[b] = tile;   // without shared memory every CTA writes it, the same, and reads its own
        });
    if (tid == 0) {
        (pre ? pre : p.rest_prefix)[B] = total;
        if (works && c + 1 == line.P) start_sh[1].g = common ? shared : total * p.rest_units;   // the cut behind the last tile
    }
    __syncthreads();
    out.first = start_sh[0];
    out.end = works ? start_sh[1].g : 0;
    // for the merge
    if (tid == 0 && cta == 0) p.plan[0] = make_int4(out.common.T, out.common.P | (even || !p.weigh ? kByTiles : 0), out.own.T, out.own.P);
    requests([&](int b, int at, int t, int, int g) {
        if (b % ctas != cta) return;
        p.plan[1 + b] = grouped ? make_int4(place[g], tiles[g], cu[g + 1] - cu[g], cu[g]) : make_int4(0, 0, 1, b);
        p.own[b] = make_int2(at, t);
    });
    if (cta == 0 && odd) report_bad_page(p.status);
    fence_proxy_async_smem();   // what was written here before key tiles land in it, behind the body's first barrier
}

// Common keys by the first CTAs, own keys by the others.  Clusters of two CTAs, for nothing but their places: the two SMs of a
// cluster share an instruction cache, and a CTA takes half as long again when its neighbour runs the other kind's code
// (four groups of 64 requests behind 32768 keys, calls back to back: 410 us where CTAs come to lie as SMs get free, 262 in pairs).
template <int D, bool CAUSAL, int NC>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPrefixThreads, 1)
    prefix_kernel(const __grid_constant__ CUtensorMap qtiles, const __grid_constant__ CUtensorMap qunits, const __grid_constant__ CUtensorMap kmap,
                  const __grid_constant__ CUtensorMap vmap, const __grid_constant__ PrefixParams p, const __grid_constant__ DecodeParams dp)
{
    using Own = DecodeShared<D, true>;
    constexpr int kOffOwn = (DecodeCfg<D>::smem_bytes(NC, true) - 1024 + 15) & ~15;   // behind the decode kernel's tiles
    static_assert(kOffOwn + sizeof(Own) <= prefix_smem<D, NC>() - 1024, "shared memory");
    static_assert((3 * kMaxGroups + 1) * 4 <= kOffOwn, "the groups do not reach the own keys' shared memory");
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ PrefixShared<D> sh;
    __shared__ int4 sums[kPrefixThreads / 32], sums2[kPrefixThreads / 32], start_raw[2];
    __shared__ uint32_t tmem_slot;
    Own& own = *reinterpret_cast<Own*>(smem + kOffOwn);
    griddep_launch_dependents();
    if (threadIdx.x / 32 == 10) {
        tmem_alloc(&tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    griddep_wait();   // the previous kernel of the stream has completed: global memory from here on
    const bool fits = p.B <= kInlineB;
    Plan plan;
    make_plan<D>(p, reinterpret_cast<int*>(smem), fits ? own.pre_sh : nullptr, fits ? own.keys_sh : nullptr, sums, sums2, reinterpret_cast<Start*>(start_raw), plan);
    const int cta = static_cast<int>(blockIdx.x);
    if (cta < plan.border) {
        prefix_body<D>(qtiles, kmap, vmap, p, sh, smem, cta, plan.first, plan.end, tmem_slot);
    } else {
        const RestPlan rest{fits ? own.pre_sh : p.rest_prefix, fits ? own.keys_sh : nullptr, plan.first, plan.end, tmem_slot};
        decode_body<D, CAUSAL, NC, true, true>(qunits, kmap, vmap, dp, own, smem, cta - plan.border, static_cast<int>(gridDim.x) - plan.border, rest);
    }
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x / 32 == 10) tmem_dealloc(tmem_slot, 512);
}

template <int D, bool CAUSAL>
auto prefix_kernel_for(int G) -> decltype(&prefix_kernel<D, CAUSAL, 1>)
{
    switch (decode_columns(G)) {
        case 1: return prefix_kernel<D, CAUSAL, 1>;
        case 4: return prefix_kernel<D, CAUSAL, 4>;
        case 8: return prefix_kernel<D, CAUSAL, 8>;
        default: return prefix_kernel<D, CAUSAL, 16>;
    }
}

}  // namespace

template <int D>
int launch_prefix(PrefixParams p, const PagedArgs& a, float* own_o, float* own_lse, cudaStream_t st)
{
    const int nsm = num_sms();
    if (nsm < 4) return set_error(FMHA_ERR_CUDA, "cannot query the SM count");
    const Shape s = paged_shape(a.B, a.Hq, a.Sq, a.c);
    CUtensorMap maps[3], qtiles;
    DecodeParams dp;
    int rc = paged_setup<D>(a, s, maps, dp);
    if (rc) return rc;
    const uint64_t dims[4] = {static_cast<uint64_t>(D), static_cast<uint64_t>(p.R), static_cast<uint64_t>(p.Hkv), static_cast<uint64_t>(p.B)};
    const uint64_t strides[3] = {static_cast<uint64_t>(D) * 2, static_cast<uint64_t>(p.R) * D * 2, static_cast<uint64_t>(p.Hkv) * p.R * D * 2};
    const uint32_t box[4] = {64, static_cast<uint32_t>(p.R), 1, static_cast<uint32_t>(p.gr.nb)};
    rc = make_tmap_bf16(&qtiles, a.q, 4, dims, strides, box);
    if (rc) return rc;
    dp.split = 1;
    dp.part_o = own_o;
    dp.part_lse = own_lse;
    // one CTA per SM; fewer when even full tables have no work for so many (see paged_ctas): half as many common units, at most, as requests,
    // and own keys
    const long long cap_tiles = (static_cast<long long>(p.cap) + kTileKV - 1) / kTileKV;
    const auto most = [&](long long units) { return units * cap_tiles / kMinPiece > units ? units * cap_tiles / kMinPiece : units; };
    const long long want = most(static_cast<long long>(p.B) * p.Hkv / 2 + 1) + most(s.U);
    const unsigned grid = static_cast<unsigned>(want < 4 ? 4 : want < nsm ? want + 1 : nsm) & ~1u;   // two pairs at least, one of each kind
    const auto kernel = a.causal ? prefix_kernel_for<D, true>(s.G) : prefix_kernel_for<D, false>(s.G);
    const int nc = decode_columns(s.G), smem = nc == 1 ? prefix_smem<D, 1>() : nc == 4 ? prefix_smem<D, 4>() : nc == 8 ? prefix_smem<D, 8>() : prefix_smem<D, 16>();
    FMHA_CHECK_CUDA(set_smem_limit_once(reinterpret_cast<const void*>(kernel), smem));
    timing_mark_begin(st);
    const cudaError_t e = launch_pdl(kernel, dim3(grid), dim3(kPrefixThreads), static_cast<size_t>(smem), st, qtiles, maps[0], maps[1], maps[2], p, dp);
    timing_mark_end(st);
    FMHA_CHECK_CUDA(e);
    count_launch();
    return FMHA_OK;
}

}  // namespace atc_gb300
