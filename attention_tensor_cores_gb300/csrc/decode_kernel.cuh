// Decode attention (few query rows per key/value head): split-KV over a persistent grid, plus
// the combine of the partial results.
//
// Follows the kernel plan of "NVFP4-1.1_RAW_CUDA_CPP_APPROACH.md" (nvfp4-megamoe-kernel): TMA
// loads of Q/K/V, the QK product on tcgen05 with the accumulator in Tensor Memory, softmax warps
// reading S back with tcgen05.ld, the running max / sum with O rescale over several KV tiles
// ("in-kernel softmax with O rescale", "multi-KV-tile support"), then the PV product.  The
// GB300 design around it is this file's own:
//
//  * Swap-AB.  With G <= 16 query rows per key/value head (G = (Hq/Hkv) * Sq), the products are
//    taken transposed so that the 128 keys of a tile fill the MMA's M dimension:
//      S^T[kv][q] = K[kv][:] . Q[q][:]      (A = K tile, K-major; B = Q rows, K-major; N = 16)
//      O^T[d][q]  = V^T[d][kv] . P^T[kv][q]  (A = V tile and B = P^T, both read MN-major; N = 16)
//    Thread t of the softmax warpgroup owns TMEM lane t: key t of the tile for S, feature d = t
//    for O.  Reductions over keys are warp shuffles plus a 4-warp shared-memory step.  The softmax
//    computes NC = 1, 4, 8 or 16 of the 16 columns, the smallest that holds a unit's rows.
//  * The per-tile PV product goes to a fresh TMEM buffer (no accumulate) and the softmax threads
//    fold it into register accumulators with the rescale factor: acc = alpha * acc + O_tile.
//    O is never read-modify-written in TMEM, so there is no ordering hazard between the rescale
//    and the next MMA.
//  * Work split ("stream-K" over keys): the key tiles of all units (b, kv-head) are laid end to
//    end and CTA c of P takes tiles [c*T/P, (c+1)*T/P).  Each maximal run inside one unit is a
//    work item; an item that covers a whole unit writes the final O and LSE, otherwise it writes
//    a normalised partial (O_i, lse_i) to slot u + c of the workspace, and the CTA that completes
//    the unit (or the combine kernel) merges them: lse = log sum_i exp(lse_i),
//    O = sum_i exp(lse_i - lse) O_i.  Ragged batches balance by construction.  With
//    num_splits == 1 each CTA takes whole units instead.
//  * Paged keys and values (PAGED): the producer gathers a tile page by page (see the producer), and
//    the work split comes from the requests' lengths inside the kernel (see Line).
//  * REST: the first tiles of some requests' keys are attended to by other CTAs of the launch (prefix_kernel.cuh), which finds the
//    work split.  What is not a request's whole attention goes to the workspace as partials that a second kernel merges.
//  * Roles (decode_kernel<D, CAUSAL, NC, PAGED>): warps 0-3 softmax.  EPI (see
//    has_epilogue_warps): warps 4-7 epilogue, warp 8 TMA producer, warp 9 MMA issuer, warp 10 the second
//    producer of paged tiles, the rest only completes its warpgroup; at the end of a work item the
//    softmax warps hand its accumulators to the epilogue warps (Tensor Memory, two buffers; see DEFER)
//    and go on with the next item while the epilogue
//    normalises, stores and merges.  !EPI: warp 4 producer, warp 5 MMA, and the softmax
//    warps run each item's short epilogue themselves.  Every wait is bounded; a timeout flips the
//    CTA into a drain mode (no new TMA/MMA, loops run out) and sets the device status word.
#pragma once
#include <cuda_runtime.h>

#include <type_traits>

#include "fastdiv.cuh"
#include "internal.h"
#include "nvfp4_dev.cuh"
#include "paged.h"
#include "ptx.cuh"

namespace atc_gb300 {
namespace {

constexpr int kTileKV = 128;    // keys per tile = MMA M

// A K or V tile in shared memory is made of 1024-byte swizzle atoms, 8 keys of 64 features each.  Dense:
// the 16 atoms of the first 64 features, then those of the next.  Paged at D = 128: the two atoms of 8 keys
// side by side, so that a TMA box can bring whole keys.
template <int D, bool PAGED>
struct TileLayout {
    static constexpr bool kInter = PAGED && D == 128;
    static constexpr int kGroup = kInter ? 2048 : 1024;            // bytes from 8 keys to the next 8
    static constexpr int kHalf = kInter ? 1024 : kTileKV * 128;    // bytes from 64 features to the next 64
    __device__ static constexpr int row(int k) { return (k >> 3) * kGroup + (k & 7) * 128; }
};
constexpr int kN = 16;          // query rows per unit, padded (MMA N)
// EPI: softmax, epilogue and control warpgroups (warps 0-3, 4-7, 8-11: producer 8, MMA 9); else the
// softmax warps run each item's epilogue themselves and warps 4 and 5 are the producer and the MMA.
template <bool EPI>
constexpr int decode_threads() { return EPI ? 384 : 192; }
// Several columns: publishing a partial costs several tiles' streaming time, which the extra warps take off the
// softmax.  One dense column: it is short, and the handoff measured 1 % slower.  One paged column keeps them, as
// lengths differ and most CTAs publish: B8 Hkv16 0..2000 keys D64 21.3 -> 20.4 us, B32 Hkv8 0..500 18.6 -> 17.3,
// B8 Hkv32 4096 keys (HBM-bound) 83.3 both ways.
template <int NC, bool PAGED>
constexpr bool has_epilogue_warps() { return NC > 1 || PAGED; }
template <bool EPI>
constexpr int tma_warp() { return EPI ? 8 : 4; }
template <bool EPI>
constexpr int mma_warp() { return EPI ? 9 : 5; }
// setmaxnreg split of the launch's 168 registers a thread: on each SM quarter one warp of each
// warpgroup, 232 + 184 + 88 = 504 of its 512, and 128 * 504 = 384 * 168 in all
constexpr uint32_t kRegsSm = 232, kRegsEpi = 184, kRegsCtl = 88;
static_assert(128 * (kRegsSm + kRegsEpi + kRegsCtl) <= decode_threads<true>() * 168, "register split exceeds the launch allocation");
static_assert(kRegsSm + kRegsEpi + kRegsCtl <= 512, "register split exceeds an SM quarter");
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescaleD = 8.0f;   // log2 units: a column's reference max moves only when exceeded by more

template <int D>
struct DecodeCfg {
    static constexpr int kAtoms = D / 64;                  // 64-column swizzle atoms per row
    static constexpr int kStages = (D == 64) ? 4 : 3;      // K and V ring depth
    static constexpr int kQBytes = kAtoms * kN * 128;      // one Q buffer
    static constexpr int kKVBytes = kAtoms * kTileKV * 128;
    static constexpr int kPBytes = 2 * kN * 128;           // P^T: 128 keys x 16 columns
    static constexpr int kOffQ = 0;
    static constexpr int kOffK = kOffQ + 2 * kQBytes;
    static constexpr int kOffV = kOffK + kStages * kKVBytes;
    static constexpr int kOffP = kOffV + kStages * kKVBytes;
    static constexpr int kSmemBytes = kOffP + 2 * kPBytes + 1024;   // + alignment slack
    // paged, 16 columns: two more P buffers behind the first two (see store_p)
    static constexpr int smem_bytes(int nc, bool paged) { return kSmemBytes + (paged && nc == 16 ? 2 * kPBytes : 0); }
    // Tensor Memory columns: S[2] x 16, O[2] x 16, handoff[2] x 32; paged, 16 columns: O[2] x 32 behind them
    static constexpr uint32_t tmem_cols(int nc, bool paged) { return paged && nc == 16 ? 256 : 128; }
    static constexpr uint32_t o_col(int nc, bool paged, uint32_t buffer) { return paged && nc == 16 ? 128 + buffer * 32 : 32 + buffer * 16; }
};

struct DecodeParams {
    int U;              // units = B * Hkv (paged: B * Hkv * chunks)
    int Hkv;            // units per batch entry
    int G;              // real query rows per unit
    int Skv;
    int D;
    int Sq;             // query rows per head (column q of a unit is query q % Sq)
    float c;            // scale * log2(e)
    const int32_t* seqlens;
    const int32_t* prefix;   // tile prefix of units (dense) or batch entries (paged), else NULL
    int tiles_uniform;       // tiles per unit when prefix == NULL
    int split;               // 1 = stream-K partition, 0 = whole units per CTA
    // outputs
    void* out;               // BF16 or F32 [U*G][D] (NULL when writing FP32 staging only)
    int out_f32;             // 1: `out` is FP32
    float* lse;              // [U*G] or NULL
    float* o_stage;          // FP32 [U*G][D] copy for NVFP4, else NULL
    unsigned* amax_bits;     // NVFP4: running max |O| (FP32 bits), else NULL
    const float* nv_sg;      // single-pass NVFP4: given s_g; codes/scales written here, else NULL
    uint8_t* nv_codes;
    uint8_t* nv_scales;
    float* nv_ts;
    float* part_o;           // [slots][16][D]
    float* part_lse;         // [slots][16]
    int fixup;               // split mode: the CTA completing a unit merges its partials (no combine kernel)
    unsigned long long gen;  // this call's tag for the arrival counters (48 bits)
    unsigned long long* unit_ctr;   // [U] arrival counters: (gen << 16) | arrivals
    int* status;
    long long limit;
    // paged keys and values (PAGED kernels only)
    const int32_t* table;    // [B][max_pages] page of each run of `page` keys
    int max_pages, num_pages;
    int page;                // keys per page, a multiple of 8
    FastDiv by_page;
    int box;                 // keys per TMA box: the largest power of two up to 128 dividing `page`
    int box_log2;
    int groups;              // D = 128: runs of 8 keys from one page to the next in the tensor map
    int cap;                 // max_pages * page: lengths are clamped to it
    int chunks;              // units per key/value head: its Gtot query rows in chunks of G
    int Gtot;
    int ctas;                // of the grid
};

// Keys of batch entry b
template <bool PAGED>
__device__ __forceinline__ int batch_keys(const DecodeParams& p, int b)
{
    if constexpr (PAGED) return min(max(p.seqlens[b], 0), p.cap);
    return p.seqlens[b];
}

// ---- work items ----------------------------------------------------------------------------------
struct Item {
    int u, t0, t1;   // unit and its tile range [t0, t1)
    int n;           // valid keys of the unit
    bool whole;      // covers every tile of the unit
    int slot;        // partial slot (u + cta)
    int b, head, chunk;   // paged: batch entry, key/value head and chunk of its rows
    bool after;      // REST: the unit has keys that are attended to elsewhere
};

// Paged work split.  The line of T tiles (below 2^31) is cut for P CTAs at c T / P, P as many as leave each
// kMinPiece tiles or as there are units with keys; a cut less than kMinPiece tiles from an end of its unit moves
// there.  A piece of a unit costs its publication and a share of the merge, several tiles' time, so short units
// stay whole.  With 2, 4 and 6 tiles at least (Hq32 Hkv8 D128): B1 500 keys 10.1, 8.1 and 8.1 us, B1 2000 13.6,
// 12.6 and 16.4, B8 0..1000 11.7, 11.5 and 13.4, B1 8000 19.6, 18.4 and 17.3, B16 Hkv1 0..4000 17.5, 15.1 and 16.3.
constexpr int kMinPiece = 4;

struct Line {
    int T = 0, P = 1;

    // floor(c T / P) of c <= P, P at most the number of SMs (below 512)
    __device__ int cut(int c) const
    {
        if (T < (1 << 23)) return static_cast<int>(static_cast<unsigned>(c) * static_cast<unsigned>(T) / static_cast<unsigned>(P));
        return static_cast<int>(static_cast<long long>(c) * T / P);
    }
};

__device__ __forceinline__ int paged_ctas(int T, int units, int n) { return max(1, min(n, max(T / kMinPiece, units))); }

// Where a CTA's range of tiles begins: tile g, the first of item (b, i, t0)
struct Start {
    int g = 0, b = 0, i = 0, t0 = 0;
};

// the cut at x as the unit of tiles [s, e) sees it (s or e when it is not inside)
__device__ __forceinline__ int unit_cut(int x, int s, int e)
{
    if (x <= s) return s;
    if (x >= e) return e;
    return x - s <= e - x ? (x - s < kMinPiece ? s : x) : (e - x < kMinPiece ? e : x);
}

// Rows of a unit.  Dense: unit u = (b, kv-head) owns rows u * G .. u * G + G - 1.  Paged: a key/value
// head with more than 16 query rows is cut into `chunks` units of at most G rows each.
template <bool PAGED>
__device__ __forceinline__ int unit_cols(const DecodeParams& p, const Item& it)
{
    if constexpr (PAGED) return min(p.G, p.Gtot - it.chunk * p.G);
    return p.G;
}
template <bool PAGED>
__device__ __forceinline__ size_t unit_row0(const DecodeParams& p, const Item& it)
{
    if constexpr (PAGED) return (static_cast<size_t>(it.b) * (p.Hkv / p.chunks) + it.head) * p.Gtot + it.chunk * p.G;
    return static_cast<size_t>(it.u) * p.G;
}
// The unit's place in its batch entry
__device__ __forceinline__ void place_unit(const DecodeParams& p, Item& it, int b, int i)
{
    it.b = b;
    it.head = p.chunks == 1 ? i : i / p.chunks;
    it.chunk = p.chunks == 1 ? 0 : i - it.head * p.chunks;
}

template <bool PAGED, bool REST = false>
struct Sched {
    const DecodeParams* p;
    const int* pre;     // paged split mode: exclusive prefix of the batch entries' tiles
    const int* keys;    // and their keys, if in shared memory
    using Pos = std::conditional_t<PAGED, int, long long>;
    Pos g, g1;          // split mode: current / end global tile
    int u;              // whole-unit mode: next unit
    int cta, nctas;
    int b, i, t0;       // paged split mode: batch entry, unit of it and tile of that which tile g is

    __device__ int unit_tiles(int u) const
    {
        if (p->prefix) return p->prefix[u + 1] - p->prefix[u];
        if (p->seqlens) return (batch_keys<PAGED>(*p, u / p->Hkv) + kTileKV - 1) / kTileKV;
        return p->tiles_uniform;
    }
    __device__ long long unit_start(int u) const
    {
        return p->prefix ? static_cast<long long>(p->prefix[u]) : static_cast<long long>(u) * p->tiles_uniform;
    }
    __device__ int unit_keys(int u) const { return p->seqlens ? batch_keys<PAGED>(*p, u / p->Hkv) : p->Skv; }

    __device__ void init(const DecodeParams* pp, int c, int n, const int* prefix, const int* lengths, const Start& start, int end)
    {
        p = pp;
        pre = prefix;
        keys = lengths;
        cta = c;
        nctas = n;
        if (p->split) {
            if constexpr (PAGED) {
                b = start.b;
                i = start.i;
                t0 = start.t0;
                g = start.g;
                g1 = end;
                return;
            }
            const long long T = p->prefix ? p->prefix[p->U] : static_cast<long long>(p->U) * p->tiles_uniform;
            g = (static_cast<long long>(c) * T) / n;
            g1 = (static_cast<long long>(c + 1) * T) / n;
        } else {
            u = c;
        }
    }

    __device__ bool next(Item& it)
    {
        if (p->split) {
            if (g >= g1) return false;
            if constexpr (PAGED) {
                // on to the batch entry that holds tile g (entries may have no tiles)
                while (pre[b + 1] * p->Hkv <= g) {
                    ++b;
                    i = 0;
                }
                const int nt = pre[b + 1] - pre[b];
                it.t0 = t0;   // only a first item may start inside its unit
                t0 = 0;
                it.u = b * p->Hkv + i;
                it.t1 = min(nt, g1 - g + it.t0);
                it.n = keys ? keys[b] : batch_keys<true>(*p, b);
                it.whole = (it.t0 == 0 && it.t1 == nt);
                it.slot = it.u + cta;
                place_unit(*p, it, b, i);
                if constexpr (REST) {   // the line has the request's last nt tiles
                    const int off = (it.n + kTileKV - 1) / kTileKV - nt;
                    it.t0 += off;
                    it.t1 += off;
                    it.after = off > 0;
                }
                g += it.t1 - it.t0;
                ++i;
                return true;
            }
            int uu;
            if (p->prefix) {   // last unit whose start <= g (prefix is non-decreasing)
                int lo = 0, hi = p->U - 1;
                while (lo < hi) {
                    const int mid = (lo + hi + 1) >> 1;
                    if (p->prefix[mid] <= g) lo = mid; else hi = mid - 1;
                }
                uu = lo;
                while (uu + 1 < p->U && p->prefix[uu + 1] <= g) ++uu;   // skip empty units
            } else {
                uu = static_cast<int>(g / p->tiles_uniform);
            }
            const long long s = unit_start(uu);
            const int nt = unit_tiles(uu);
            it.u = uu;
            it.t0 = static_cast<int>(g - s);
            it.t1 = static_cast<int>(min(static_cast<long long>(nt), static_cast<long long>(g1) - s));
            it.n = unit_keys(uu);
            it.whole = (it.t0 == 0 && it.t1 == nt);
            it.slot = uu + cta;
            g = s + it.t1;
            return true;
        }
        if (u >= p->U) return false;
        it.u = u;
        it.t0 = 0;
        it.t1 = unit_tiles(u);
        it.n = unit_keys(u);
        it.whole = true;
        it.slot = 0;
        if constexpr (PAGED) place_unit(*p, it, u / p->Hkv, u % p->Hkv);
        u += nctas;
        return true;
    }
};

__device__ __forceinline__ void tma_load_5d_hint(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int y, int z, int w, int v,
                                                 uint64_t policy)
{
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%3, %4, %5, %6, %7}], [%2], %8;" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(v), "l"(policy)
        : "memory");
}

__device__ __forceinline__ void tma_load_4d_hint(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int y, int z, int w,
                                                 uint64_t policy)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%3, %4, %5, %6}], [%2], %7;" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "r"(w), "l"(policy)
        : "memory");
}

// P^T of a tile is an MN-major operand with the 32-byte swizzle: 16 columns of a key in a row of 32 bytes, so
// that the thread with the key stores them with at most two 16-byte stores (K-major rows of keys took one
// 2-byte store per column); rows 4..7 of each 8 have their 16-byte halves exchanged.  Atoms of 8 keys are 256
// bytes apart (SBO), the next 16 columns, if any, `lbo_bytes`.
__device__ __forceinline__ uint64_t sdesc_sw32(uint32_t saddr, uint32_t lbo_bytes, uint32_t sbo_bytes)
{
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr & 0x3FFFF) >> 4);
    d |= static_cast<uint64_t>((lbo_bytes >> 4) & 0x3FFF) << 16;
    d |= static_cast<uint64_t>((sbo_bytes >> 4) & 0x3FFF) << 32;
    d |= static_cast<uint64_t>(1) << 46;
    d |= static_cast<uint64_t>(6) << 61;
    return d;
}

// Row `key` of P^T, rounded to BF16 (the operand type of the MMA; half a step, 2^-9 to 2^-8 of a weight).  TWO
// (paged): what the rounding leaves goes along as a second BF16, so that P is good to 2^-17 and the output's
// own rounding is the only one that shows (rms error of BF16 outputs 1.7e-3 of them instead of 2.3e-3).  Up to eight
// columns it takes the other eight of the 16 (columns 8 ..), with 16 a second buffer, `low`, and an MMA of 32
// columns over both.  Neither costs time that shows: an MMA of up to 64 columns takes the same 50 cycles (a second
// MMA of 16 columns instead cost B17 Hq16 Hkv4 Sq4 D64 1.2 of 20 us).
template <int NC, bool TWO>
__device__ __forceinline__ void store_p(uint8_t* sP, uint8_t* low, int key, const float (&pv)[NC])
{
    const int first = key * 32 + ((key >> 2) & 1) * 16, second = first ^ 16;   // columns 0..7 and 8..15
    if constexpr (NC == 1) {
        const uint16_t w = float_to_bf16_bits(pv[0]);
        *reinterpret_cast<uint16_t*>(sP + first) = w;
        if constexpr (TWO)
            *reinterpret_cast<uint16_t*>(sP + second) = float_to_bf16_bits(pv[0] - __uint_as_float(static_cast<uint32_t>(w) << 16));
    } else {
        uint32_t w[NC / 2], x[NC / 2];
#pragma unroll
        for (int i = 0; i < NC / 2; ++i) {
            w[i] = pack_bf16x2(pv[2 * i], pv[2 * i + 1]);
            if constexpr (TWO)
                x[i] = pack_bf16x2(pv[2 * i] - __uint_as_float(w[i] << 16), pv[2 * i + 1] - __uint_as_float(w[i] & 0xffff0000u));
        }
        if constexpr (NC == 4) {
            *reinterpret_cast<uint2*>(sP + first) = make_uint2(w[0], w[1]);
            if constexpr (TWO) *reinterpret_cast<uint2*>(sP + second) = make_uint2(x[0], x[1]);
        } else {
            *reinterpret_cast<uint4*>(sP + first) = make_uint4(w[0], w[1], w[2], w[3]);
            if constexpr (NC == 8 && TWO) *reinterpret_cast<uint4*>(sP + second) = make_uint4(x[0], x[1], x[2], x[3]);
            if constexpr (NC == 16) {
                *reinterpret_cast<uint4*>(sP + second) = make_uint4(w[4], w[5], w[6], w[7]);
                if constexpr (TWO) {
                    *reinterpret_cast<uint4*>(low + first) = make_uint4(x[0], x[1], x[2], x[3]);
                    *reinterpret_cast<uint4*>(low + second) = make_uint4(x[4], x[5], x[6], x[7]);
                }
            }
        }
    }
}

// Tensor Memory loads and stores of N consecutive columns of this warp's 32 lanes
template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[N])
{
    static_assert(N == 1 || N == 2 || N == 4 || N == 8 || N == 16 || N == 32, "column counts in use");
    if constexpr (N == 1)
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r[0]) : "r"(taddr));
    else if constexpr (N == 2)
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x2.b32 {%0, %1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(taddr));
    else if constexpr (N == 4)
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(taddr));
    else if constexpr (N == 8)
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                     : "r"(taddr));
    else if constexpr (N == 16)
        tmem_ld16(taddr, r);
    else
        tmem_ld32(taddr, r);
}

template <int N>
__device__ __forceinline__ void tmem_st(uint32_t taddr, const uint32_t (&r)[N])
{
    static_assert(N == 1 || N == 4 || N == 8 || N == 16, "column counts in use");
    if constexpr (N == 1)
        asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(taddr), "r"(r[0]) : "memory");
    else if constexpr (N == 4)
        asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3])
                     : "memory");
    else if constexpr (N == 8)
        asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]),
                     "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                     : "memory");
    else
        tmem_st16(taddr, r);
}

// Barrier over the first 128 threads' warps that also returns whether any of them passes true
__device__ __forceinline__ bool bar_any128(int id, bool v)
{
    int r;
    asm volatile(
        "{\n"
        ".reg .pred a, b;\n"
        "setp.ne.u32 a, %1, 0;\n"
        "barrier.cta.red.or.pred b, %2, 128, a;\n"
        "selp.u32 %0, 1, 0, b;\n"
        "}\n"
        : "=r"(r)
        : "r"(v ? 1 : 0), "r"(id)
        : "memory");
    return r != 0;
}

// Largest value of the warp's 32 lanes (NaN loses against any number)
__device__ __forceinline__ float redux_max(float v)
{
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}

// Bounded wait that ignores the abort flag: used at teardown so nothing is still in flight.
__device__ __forceinline__ void drain_wait(uint64_t* bar, uint32_t parity, long long limit)
{
    const uint32_t a = smem_u32(bar);
    const long long t0 = clock64();
    while (!mbar_try_wait(a, parity)) {
        if (clock64() - t0 > limit) return;
    }
}

struct Ring {
    uint32_t idx = 0, phase = 0;
    int n;
    __device__ explicit Ring(int stages) : n(stages) {}
    __device__ void advance()
    {
        if (++idx == static_cast<uint32_t>(n)) {
            idx = 0;
            phase ^= 1;
        }
    }
};

// The same for merges, where a NaN is to be seen
__device__ __forceinline__ float redux_max_nan(float v)
{
    float r;
    asm volatile("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}

__device__ __forceinline__ float fmax_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ float warp_max(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Stream-K: the CTAs holding partials of unit u are c0..c1 of P, skipping CTAs whose tile range is
// empty (possible when there are fewer tiles than CTAs).  Fills slots[] (partial slots u + c, at
// most cap) and returns how many there are; 0 for a unit without tiles.
__device__ int unit_partial_slots(const DecodeParams& p, int u, int P, int* slots, int cap)
{
    int tiles;
    long long Tu, T;
    if (p.prefix) {
        tiles = p.prefix[u + 1] - p.prefix[u];
        Tu = p.prefix[u];
        T = p.prefix[p.U];
    } else {
        tiles = p.tiles_uniform;
        Tu = static_cast<long long>(u) * tiles;
        T = static_cast<long long>(p.U) * tiles;
    }
    if (tiles <= 0) return 0;
    const int c0 = static_cast<int>(min((((Tu + 1) * P) - 1) / T, static_cast<long long>(P - 1)));
    const int c1 = static_cast<int>(min((((Tu + tiles) * P) - 1) / T, static_cast<long long>(P - 1)));
    int n = 0;
    for (int c = c0; c <= c1 && n < cap; ++c)
        if ((static_cast<long long>(c) * T) / P != (static_cast<long long>(c + 1) * T) / P) slots[n++] = u + c;
    return n;
}

// Same for the paged split: the CTAs with a piece of unit i of batch entry b.
__device__ int paged_partial_slots(const DecodeParams& p, const int* pre, const Line& line, int b, int i, int* slots, int cap)
{
    const int tiles = pre[b + 1] - pre[b];
    if (tiles <= 0) return 0;
    const int s = pre[b] * p.Hkv + i * tiles, e = s + tiles;
    // the CTA whose cut is the last at or before s, and one before it, as a cut behind s may have moved back
    int c = min(static_cast<int>(static_cast<float>(s) * (static_cast<float>(line.P) / static_cast<float>(line.T))), line.P - 1);
    while (c > 0 && line.cut(c) > s) --c;
    while (c + 1 < line.P && line.cut(c + 1) <= s) ++c;
    c = max(c - 1, 0);
    int n = 0, lo = unit_cut(line.cut(c), s, e);
    for (; c < line.P && lo < e && n < cap; ++c) {
        const int hi = unit_cut(line.cut(c + 1), s, e);
        if (lo < hi) slots[n++] = b * p.Hkv + i + c;
        lo = hi;
    }
    return n;
}

constexpr int kMaxFixSlots = 160;   // at most one partial of a unit per SM
constexpr int kFixChunk = 32;   // partials whose weights are in shared memory at once

// Paged split mode finds the work split itself when it has up to this many batch entries: every CTA sums
// the entries' tiles into its shared memory, which costs less than a launch that leaves them in global
// memory.  Twice as many would not fit beside 16 columns' P at D = 128.
constexpr int kInlineB = 512;

// O = 0 and LSE = -inf for batch entry b without keys, by the whole CTA
__device__ __forceinline__ void write_empty_entry(const DecodeParams& p, int b)
{
    const size_t rows = static_cast<size_t>(p.Hkv / p.chunks) * p.Gtot, r0 = b * rows, n = rows * p.D;
    for (size_t i = threadIdx.x; i < n; i += blockDim.x) {
        if (p.o_stage) p.o_stage[r0 * p.D + i] = 0.f;
        if (p.out) {
            if (p.out_f32)
                static_cast<float*>(p.out)[r0 * p.D + i] = 0.f;
            else
                static_cast<uint16_t*>(p.out)[r0 * p.D + i] = 0;
        }
    }
    if (p.lse)
        for (size_t i = threadIdx.x; i < rows; i += blockDim.x) p.lse[r0 + i] = -INFINITY;
}

// Columns the softmax computes for units of G rows (the MMA's N stays kN): 1, 4, 8 or 16.
inline int decode_columns(int G) { return G <= 1 ? 1 : G <= 4 ? 4 : G <= 8 ? 8 : 16; }

// A CTA's shared memory beside the tiles
template <int D, bool PAGED>
struct DecodeShared {
    static constexpr int S = DecodeCfg<D>::kStages;
    uint64_t q_full[2], q_empty[2], k_full[S], k_empty[S], v_full[S], v_empty[S];
    // S, P and O of a tile alternate between two buffers without barriers for "empty": the MMA warp issues
    // QK(k), PV(k - 1), QK(k + 1), .. and PV(k) waits for P(k), by when the softmax has read S(k) and O(k - 2);
    // it stores P(k) after it has read O(k - 2), by when PV(k - 2) has read P(k - 2).
    uint64_t s_full[2], p_full[2], o_full[2], mma_done;
    uint64_t ep_full[2], ep_empty[2];   // softmax -> epilogue handoff
    float ep_m[2][kN];                  // the columns' reference maxima
    uint32_t tmem_slot;
    int abort_flag;
    float red_max[4][kN];
    float red_sum[4][kN];
    float col_inv[kN], col_lse[kN];   // per query column: 1 / L and the LSE of this range
    int ep_abort, fx_last;          // softmax warps: abort snapshot, "this CTA merges"
    int fx_n;
    int fx_slot[kMaxFixSlots];
    float fx_w[kN][kFixChunk], fx_lse[kN];   // merge: per column, the partials' weights and the merged LSE
    int pre_sh[PAGED ? kInlineB + 1 : 1], keys_sh[PAGED ? kInlineB : 1];
    int2 sums_sh[PAGED ? 12 : 1];
    int4 start_raw[2];
};

// REST: what the launch has found out, and what it has set up
struct RestPlan {
    const int *pre, *keys;   // prefix of the batch entries' tiles, and their keys (or NULL)
    Start first;
    int end;
    uint32_t tmem;
};

// The kernel's body for CTA `cta` of `ctas`; smem: the tiles' shared memory, 1024-byte aligned
template <int D, bool CAUSAL, int NC, bool PAGED, bool REST>
__device__ __forceinline__ void decode_body(const CUtensorMap& qmap, const CUtensorMap& kmap, const CUtensorMap& vmap, const DecodeParams& p,
                                            DecodeShared<D, PAGED>& sh, uint8_t* smem, int cta, int ctas, const RestPlan& plan)
{
    using C = DecodeCfg<D>;
    constexpr int S = C::kStages;
    constexpr bool EPI = has_epilogue_warps<NC, PAGED>();
    auto &q_full = sh.q_full, &q_empty = sh.q_empty, &s_full = sh.s_full, &p_full = sh.p_full, &o_full = sh.o_full, &ep_full = sh.ep_full, &ep_empty = sh.ep_empty;
    auto &k_full = sh.k_full, &k_empty = sh.k_empty, &v_full = sh.v_full, &v_empty = sh.v_empty;
    auto &ep_m = sh.ep_m;
    auto &red_max = sh.red_max, &red_sum = sh.red_sum;
    auto &col_inv = sh.col_inv, &col_lse = sh.col_lse, &fx_lse = sh.fx_lse;
    auto &fx_slot = sh.fx_slot;
    auto &fx_w = sh.fx_w;
    auto &pre_sh = sh.pre_sh;
    auto &keys_sh = sh.keys_sh;
    auto &sums_sh = sh.sums_sh;
    uint64_t& mma_done = sh.mma_done;
    uint32_t& tmem_slot = sh.tmem_slot;
    int &abort_flag = sh.abort_flag, &ep_abort = sh.ep_abort, &fx_last = sh.fx_last, &fx_n = sh.fx_n;
    Start* start_sh = reinterpret_cast<Start*>(sh.start_raw);

    const int warp = threadIdx.x / 32;
    if constexpr (!REST) griddep_launch_dependents();
    const WaitCtl wc{&abort_flag, p.status, p.limit};

    if (threadIdx.x == 0) {
        abort_flag = 0;
        for (int i = 0; i < 2; ++i) {
            mbar_init(&q_full[i], 1);
            mbar_init(&q_empty[i], 1);
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 4);   // one arrival per warp
            mbar_init(&o_full[i], 1);
            mbar_init(&ep_full[i], 4);   // one arrival per warp
            mbar_init(&ep_empty[i], 4);   // one arrival per warp
        }
        for (int i = 0; i < S; ++i) {
            mbar_init(&k_full[i], 1);
            mbar_init(&k_empty[i], 1);
            mbar_init(&v_full[i], 1);
            mbar_init(&v_empty[i], 1);
        }
        mbar_init(&mma_done, 1);
        fence_barrier_init();
    }
    if constexpr (!REST) {
        if (warp == mma_warp<EPI>()) {
            tmem_alloc(&tmem_slot, C::tmem_cols(NC, PAGED));
            tmem_relinquish();
        }
    }
    if constexpr (PAGED) {
        if (threadIdx.x == tma_warp<EPI>() * 32) {
            tma_prefetch_desc(&qmap);
            tma_prefetch_desc(&kmap);
            tma_prefetch_desc(&vmap);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = REST ? plan.tmem : tmem_slot;   // S buffers at columns 0/16, handoff at 64/96, O buffers at o_col()
    if constexpr (!REST) griddep_wait();   // the previous kernel of the stream has completed: global memory from here on
    if (!REST && cta == 0 && threadIdx.x == 0 && p.nv_ts) *p.nv_ts = *p.nv_sg;   // single-pass NVFP4: report s_g

    const int *pre = p.prefix, *keys = nullptr;
    Start first;        // paged split mode: the CTA's range of tiles
    int end = 0;
    Line line;
    if constexpr (REST) {
        pre = plan.pre;
        keys = plan.keys;
        first = plan.first;
        end = plan.end;
    } else if constexpr (PAGED) {
        const int B = p.U / p.Hkv, c = cta, lane = static_cast<int>(threadIdx.x) & 31;
        // the CTA's cut at x, in batch entry b of nt tiles a unit whose first tile is s0
        auto start_at = [&](int x, int b, int s0, int nt) {
            Start r;
            const int i = static_cast<int>(static_cast<unsigned>(x - s0) / static_cast<unsigned>(nt)), s = s0 + i * nt;
            r.g = unit_cut(x, s, s + nt);
            r.b = b;
            r.i = r.g == s + nt ? i + 1 : i;
            r.t0 = r.g == s + nt ? 0 : r.g - s;
            return r;
        };
        // whoever has the entry that one of the CTA's two cuts falls in says so
        auto owns = [&](int b, int start, int nt, const int (&cut)[2]) {
            const int s0 = start * p.Hkv;
#pragma unroll
            for (int k = 0; k < 2; ++k)
                if (s0 <= cut[k] && cut[k] < s0 + nt * p.Hkv) start_sh[k] = start_at(cut[k], b, s0, nt);
        };
        if (p.split && !p.prefix && B <= 32) {
            // a lane per entry, the same in every warp: no barrier (all write the same to shared memory)
            const int n = lane < B ? batch_keys<true>(p, lane) : 0, nt = (n + kTileKV - 1) / kTileKV;
            int inc = nt;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += v;
            }
            const int start = inc - nt;
            line.T = __shfl_sync(0xffffffffu, inc, 31) * p.Hkv;
            line.P = paged_ctas(line.T, __popc(__ballot_sync(0xffffffffu, n > 0)) * p.Hkv, ctas);
            keys_sh[lane] = n;
            pre_sh[lane] = start;
            if (lane == 31) pre_sh[32] = inc;
            __syncwarp();
            pre = pre_sh;
            keys = keys_sh;
            if (c < line.P && line.T > 0) {
                // even lanes look at the CTA's first cut, odd lanes at the next CTA's
                const int cut = line.cut(c + (lane & 1)), cut0 = __shfl_sync(0xffffffffu, cut, 0), cut1 = __shfl_sync(0xffffffffu, cut, 1);
                const unsigned has0 = __ballot_sync(0xffffffffu, start * p.Hkv <= cut0 && cut0 < inc * p.Hkv);
                const unsigned has1 = __ballot_sync(0xffffffffu, start * p.Hkv <= cut1 && cut1 < inc * p.Hkv);
                const int b = max(__ffs(lane & 1 ? has1 : has0) - 1, 0);
                const int s0 = __shfl_sync(0xffffffffu, start, b) * p.Hkv, tiles = __shfl_sync(0xffffffffu, nt, b);
                const Start mine = start_at(cut, b, s0, max(tiles, 1));
                first.g = __shfl_sync(0xffffffffu, mine.g, 0);
                first.b = __shfl_sync(0xffffffffu, mine.b, 0);
                first.i = __shfl_sync(0xffffffffu, mine.i, 0);
                first.t0 = __shfl_sync(0xffffffffu, mine.t0, 0);
                end = __shfl_sync(0xffffffffu, mine.g, 1);
                if (!has1) end = line.T;   // the cut behind the last tile
            }
        } else if (p.split && !p.prefix) {
            // a run of entries per thread, then a scan over the threads
            const int per = (B + blockDim.x - 1) / blockDim.x;
            const int b0 = min(B, static_cast<int>(threadIdx.x) * per), b1 = min(B, b0 + per);
            int own = 0, with_keys = 0;
            for (int b = b0; b < b1; ++b) {
                const int n = batch_keys<true>(p, b);
                keys_sh[b] = n;
                own += (n + kTileKV - 1) / kTileKV;
                with_keys += n > 0 ? 1 : 0;
            }
            int inc = own;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += v;
            }
            with_keys = static_cast<int>(__reduce_add_sync(0xffffffffu, static_cast<unsigned>(with_keys)));
            if (lane == 31) sums_sh[warp] = make_int2(inc, with_keys);
            __syncthreads();
            int before = 0, total = 0;
            with_keys = 0;
#pragma unroll
            for (int w = 0; w < decode_threads<EPI>() / 32; ++w) {
                const int2 v = sums_sh[w];
                before += w < warp ? v.x : 0;
                total += v.x;
                with_keys += v.y;
            }
            line.T = total * p.Hkv;
            line.P = paged_ctas(line.T, with_keys * p.Hkv, ctas);
            const int cut[2] = {line.cut(c), line.cut(c + 1)};
            int run = before + inc - own;
            for (int b = b0; b < b1; ++b) {
                const int nt = (keys_sh[b] + kTileKV - 1) / kTileKV;
                pre_sh[b] = run;
                if (c < line.P) owns(b, run, nt, cut);
                run += nt;
            }
            if (threadIdx.x == 0) pre_sh[B] = total;
            pre = pre_sh;
            keys = keys_sh;
        } else if (p.split) {
            line.T = pre[B] * p.Hkv;
            line.P = pre[B + 1];
            const int cut[2] = {line.cut(c), line.cut(c + 1)};
            if (c < line.P)
                for (int b = threadIdx.x; b < B; b += blockDim.x) owns(b, pre[b], pre[b + 1] - pre[b], cut);
        }
        if (p.split && (p.prefix || B > 32)) {
            if (threadIdx.x == 0) {   // cuts that no entry has
                if (c >= line.P || line.T == 0)
                    start_sh[0] = start_sh[1] = Start{};
                else if (c + 1 == line.P)
                    start_sh[1].g = line.T;
            }
            __syncthreads();
            first = start_sh[0];
            end = start_sh[1].g;
        }
    }

    Sched<PAGED, REST> sched;
    sched.init(&p, cta, ctas, pre, keys, first, end);
    Item it;

    // fills fx_slot with the slots of the unit's partials
    auto partial_slots = [&](const Item& it) {
        if constexpr (PAGED) return paged_partial_slots(p, pre, line, it.b, it.head * p.chunks + it.chunk, fx_slot, kMaxFixSlots);
        return unit_partial_slots(p, it.u, ctas, fx_slot, kMaxFixSlots);
    };

    // The epilogue of one item, run by 128 threads: the epilogue warpgroup (named barrier 2) or, without
    // one, the softmax warps themselves (barrier 1).  tid: O^T row (Tensor Memory lane) and output
    // column, ew: warp within the group.
    // slots_ready: fx_n / fx_slot already hold this item's partial slots (the epilogue warpgroup finds
    // them while it waits for the item)
    auto run_epilogue = [&](const Item& it, bool empty, const float (&m)[NC], const float (&l)[NC],
                            const float (&acc)[NC], int tid, int ew, int bar, bool slots_ready) {
        const int lane = static_cast<int>(lane_id());
        const int G = unit_cols<PAGED>(p, it);
        const float nv_sg = p.nv_sg ? *p.nv_sg : 0.f;
        const size_t row0 = unit_row0<PAGED>(p, it);
        // final output of the unit's rows at column d < D; returns the |O| max when it is wanted.  The
        // choices are made once, not per row: the rows' stores then go out back to back.
        auto write_rows = [&](const float (&o)[NC], int d) {
            float am = 0.f;
            if (p.o_stage) {
                float* dst = p.o_stage + row0 * D + d;
#pragma unroll
                for (int q = 0; q < NC; ++q)
                    if (q < G) dst[q * D] = o[q];
            }
            if (p.amax_bits) {
#pragma unroll
                for (int q = 0; q < NC; ++q)
                    if (q < G) am = fmaxf(am, fabsf(o[q]));
            }
            if (p.out && p.out_f32) {
                float* dst = static_cast<float*>(p.out) + row0 * D + d;
#pragma unroll
                for (int q = 0; q < NC; ++q)
                    if (q < G) dst[q * D] = o[q];
            } else if (p.out) {
                uint16_t* dst = static_cast<uint16_t*>(p.out) + row0 * D + d;
#pragma unroll
                for (int q = 0; q < NC; ++q)
                    if (q < G) dst[q * D] = float_to_bf16_bits(o[q]);
            }
            return am;
        };
        // ---- epilogue: L = sum over the 128 key lanes, O = acc · (1 / L), lse = ln2 * (m + log2 L)
        if (!empty) {
            if (NC == 1) {
                const float s = warp_sum(l[0]);
                if (lane == 0) red_sum[ew][0] = s;
            } else {
                // butterflies over the lanes in which each round halves the columns a lane carries: the lane keeps
                // those whose bit matches its own and gives the others away (16 shuffles for 16 columns, not 80)
                float v[NC];
#pragma unroll
                for (int q = 0; q < NC; ++q) v[q] = l[q];
                int n = NC, col = 0;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) {
                    const bool up = lane & o;
                    if (n > 1) {
                        n >>= 1;
                        col += up ? n : 0;
#pragma unroll
                        for (int q = 0; q < NC / 2; ++q)
                            if (q < n) {
                                const float give = up ? v[q] : v[q + n], keep = up ? v[q + n] : v[q];
                                v[q] = keep + __shfl_xor_sync(0xffffffffu, give, o);
                            }
                    } else {
                        v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
                    }
                }
                if ((lane & (32 / NC - 1)) == 0) red_sum[ew][col] = v[0];
            }
        }
        // red_sum is complete, and every thread is past its reads of the previous item's
        // col_inv / col_lse (an empty item has no tile barriers in between)
        named_bar_sync(bar, 128);
        // one thread per column: L, then 1 / L and the LSE for every thread of the CTA
        if (tid < G) {
            const float Lq = empty ? 0.f : (red_sum[0][tid] + red_sum[1][tid]) + (red_sum[2][tid] + red_sum[3][tid]);
            float mq = m[0];
#pragma unroll
            for (int q = 1; q < NC; ++q)
                if (q == tid) mq = m[q];
            const bool none = Lq == 0.f;   // no visible key in this range; a NaN score makes L, the row and its LSE NaN
            col_inv[tid] = none ? 0.f : 1.f / Lq;
            col_lse[tid] = none ? -INFINITY : (mq + __log2f(Lq)) * kLn2;
        }
        // one abort decision for all four warps (named barriers and shuffles below)
        if (tid == 0) ep_abort = aborted(wc) ? 1 : 0;
        named_bar_sync(bar, 128);
        const bool lost = ep_abort != 0;
        // single-pass NVFP4 in split mode: whole units also go through the combine, which
        // encodes every row in parallel (encoding here would lengthen the CTAs holding many
        // short units)
        const bool final_here = it.whole && !(p.split && p.nv_codes) && !(REST && (it.after || !p.out));
        // An aborted CTA writes no result, but a partial that is counted goes out all the same, as one without a
        // visible key: a graph's replays carry one tag, so an arrival left out here would be made up for by the
        // next replay's first one.
        if (lost && !(p.fixup && !final_here)) return;
        float local_amax = 0.f;
        float o[NC];
#pragma unroll
        for (int q = 0; q < NC; ++q) o[q] = col_inv[q] != 0.f && !lost ? acc[q] * col_inv[q] : 0.f;   // 0: no visible key in this range
        if (final_here) {
            if (tid < D) {
                local_amax = write_rows(o, tid);
                if (p.nv_codes)   // single-pass NVFP4: a warp holds 32 consecutive columns of the row
#pragma unroll
                    for (int q = 0; q < NC; ++q)
                        if (q < G)
                            nvfp4_encode_lanes(o[q], nv_sg, tid, p.nv_codes + (row0 + q) * (D / 2), p.nv_scales + (row0 + q) * (D / 16));
            }
            if (tid < G && p.lse) p.lse[row0 + tid] = col_lse[tid];
        } else {
            if (tid < D) {
                float* dst = p.part_o + static_cast<size_t>(it.slot) * kN * D + tid;
#pragma unroll
                for (int q = 0; q < NC; ++q)
                    if (q < G) dst[q * D] = o[q];
            }
            if (tid < G) p.part_lse[static_cast<size_t>(it.slot) * kN + tid] = lost ? -INFINITY : col_lse[tid];
        }
        if (p.amax_bits && final_here) {
            const float wm = warp_max(local_amax);
            if (lane == 0 && wm > 0.f) atomicMax(p.amax_bits, __float_as_uint(wm));
        }
        if (p.fixup && !final_here) {
            // stream-K fixup: publish this partial, count the unit's arrivals, and let the CTA
            // that completes the unit merge it (O = sum exp(lse_i - lse) O_i, as the combine).
            // The CTA barrier orders every thread's partial stores before thread 0's device-scope
            // fence, which releases them all (release is cumulative) ahead of its arrival: one
            // fence waits for the stores instead of 128.
            named_bar_sync(bar, 128);
            if (tid == 0) {
                const int n = slots_ready ? fx_n : partial_slots(it);
                fx_n = n;
                __threadfence();
                const int arrived = n > 0 ? arrive_unit(p.unit_ctr + it.u, p.gen, n) : 0;
                // -1: the counter kept changing under us (another call on this workspace):
                // the unit may stay unmerged, so say so instead of failing silently
                if (arrived < 0) atomicExch(p.status, kDevMergeLost);
                fx_last = (arrived == n && n > 0) ? 1 : 0;
                // every arrival of this call is in: clear the counter for the next call.  A CUDA graph
                // replays a call with the same tag, so its arrivals must not be left over (0 carries
                // no call's tag: tags are never 0).
                if (fx_last) atomicExch(p.unit_ctr + it.u, 0ull);
            }
            named_bar_sync(bar, 128);
            if (fx_last) {
                __threadfence();
                const int ns = fx_n;
                float amax_m = 0.f;
                if (ns <= 4) {
                    // the usual case: this thread's element of every partial O of every column, and
                    // (threads q < G) column q's partial LSEs, all in flight at once, so the merge
                    // costs one L2 round trip whatever the number of columns (a round per few
                    // columns was one dependent trip each, slow while the other CTAs stream)
                    float ov[4][NC];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const bool use = i < ns && tid < D;
                        const float* src = p.part_o + static_cast<size_t>(fx_slot[i < ns ? i : 0]) * kN * D + tid;
#pragma unroll
                        for (int q = 0; q < NC; ++q) ov[i][q] = use && q < G ? __ldcg(src + q * D) : 0.f;
                    }
                    if (tid < G) {
                        float lv[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            lv[i] = i < ns ? __ldcg(p.part_lse + static_cast<size_t>(fx_slot[i]) * kN + tid) : -INFINITY;
                        const float mx = fmax_nan(fmax_nan(lv[0], lv[1]), fmax_nan(lv[2], lv[3]));
                        const bool any = mx != -INFINITY;   // partials without a visible key carry -inf
                        float sum = 0.f;
#pragma unroll
                        for (int i = 0; i < 4; ++i) sum += (any && i < ns) ? __expf(lv[i] - mx) : 0.f;
                        const float lse_all = any ? mx + __logf(sum) : -INFINITY;
#pragma unroll
                        for (int i = 0; i < 4; ++i) fx_w[tid][i] = (any && i < ns) ? __expf(lv[i] - lse_all) : 0.f;
                        fx_lse[tid] = lse_all;
                    }
                    named_bar_sync(bar, 128);
#pragma unroll
                    for (int q = 0; q < NC; ++q) {
                        o[q] = 0.f;
#pragma unroll
                        for (int i = 0; i < 4; ++i) o[q] = fmaf(fx_w[q][i], ov[i][q], o[q]);
                    }
                    if (tid < D) amax_m = write_rows(o, tid);
                } else {
                    // More partials (a long sequence over many CTAs): first their LSEs, a warp per column and a
                    // lane per partial, all columns' loads in flight together; then their O, four groups of lanes
                    // taking every fourth partial and eight lanes 32 columns of D, the groups' sums meeting in
                    // shuffles at the end.
                    constexpr int kCols = (NC + 3) / 4;
                    auto load_lse = [&](int c, int i) {
                        const int q = ew + 4 * c;
                        return q < G && i < ns ? __ldcg(p.part_lse + static_cast<size_t>(fx_slot[i]) * kN + q) : -INFINITY;
                    };
                    float lv[kCols], mx[kCols], all[kCols];
#pragma unroll
                    for (int c = 0; c < kCols; ++c) mx[c] = lv[c] = load_lse(c, lane);
                    for (int i = lane + kFixChunk; i < ns; i += kFixChunk)
#pragma unroll
                        for (int c = 0; c < kCols; ++c) mx[c] = fmax_nan(mx[c], load_lse(c, i));
#pragma unroll
                    for (int c = 0; c < kCols; ++c) {
                        mx[c] = redux_max_nan(mx[c]);
                        // partials without a visible key carry lse = -inf and weigh 0; all of them -> empty row
                        all[c] = mx[c] != -INFINITY ? __expf(lv[c] - mx[c]) : 0.f;
                    }
                    for (int i = lane + kFixChunk; i < ns; i += kFixChunk)
#pragma unroll
                        for (int c = 0; c < kCols; ++c)
                            if (mx[c] != -INFINITY) all[c] += __expf(load_lse(c, i) - mx[c]);
#pragma unroll
                    for (int x = 16; x > 0; x >>= 1)
#pragma unroll
                        for (int c = 0; c < kCols; ++c) all[c] += __shfl_xor_sync(0xffffffffu, all[c], x);
#pragma unroll
                    for (int c = 0; c < kCols; ++c) {
                        all[c] = mx[c] != -INFINITY ? mx[c] + __logf(all[c]) : -INFINITY;
                        if (lane == 0 && ew + 4 * c < NC) fx_lse[ew + 4 * c] = all[c];
                    }
                    const int d = ew * 32 + (lane & 7) * 4, first = lane >> 3;
                    float4 sum4[NC];
#pragma unroll
                    for (int q = 0; q < NC; ++q) sum4[q] = make_float4(0.f, 0.f, 0.f, 0.f);
                    for (int c0 = 0; c0 < ns; c0 += kFixChunk) {
                        if (c0) named_bar_sync(bar, 128);   // the previous run's weights have been used
#pragma unroll
                        for (int c = 0; c < kCols; ++c) {
                            const float x = c0 ? load_lse(c, c0 + lane) : lv[c];
                            if (ew + 4 * c < NC) fx_w[ew + 4 * c][lane] = all[c] != -INFINITY ? __expf(x - all[c]) : 0.f;
                        }
                        named_bar_sync(bar, 128);
                        const int nc = min(kFixChunk, ns - c0);
                        if (d < D) {
#pragma unroll(NC == 1 ? 8 : NC == 4 ? 4 : NC == 8 ? 2 : 1)
                            for (int i = first; i < nc; i += 4) {
                                const float* src = p.part_o + static_cast<size_t>(fx_slot[c0 + i]) * kN * D + d;
                                float4 v[NC];
#pragma unroll
                                for (int q = 0; q < NC; ++q)
                                    v[q] = q < G ? __ldcg(reinterpret_cast<const float4*>(src + q * D)) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                                for (int q = 0; q < NC; ++q) {
                                    const float w = fx_w[q][i];
                                    sum4[q].x = fmaf(w, v[q].x, sum4[q].x);
                                    sum4[q].y = fmaf(w, v[q].y, sum4[q].y);
                                    sum4[q].z = fmaf(w, v[q].z, sum4[q].z);
                                    sum4[q].w = fmaf(w, v[q].w, sum4[q].w);
                                }
                            }
                        }
                    }
#pragma unroll
                    for (int q = 0; q < NC; ++q) {
                        float x[4] = {sum4[q].x, sum4[q].y, sum4[q].z, sum4[q].w};
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            x[k] += __shfl_xor_sync(0xffffffffu, x[k], 8);
                            x[k] += __shfl_xor_sync(0xffffffffu, x[k], 16);
                        }
                        // the four lanes of a column group hold the same sums: each writes one column
                        o[q] = first == 0 ? x[0] : first == 1 ? x[1] : first == 2 ? x[2] : x[3];
                    }
                    if (d < D) amax_m = write_rows(o, d + first);
                }
                if (tid < G && p.lse) p.lse[row0 + tid] = fx_lse[tid];
                if (p.amax_bits) {
                    const float wm = warp_max(amax_m);
                    if (lane == 0 && wm > 0.f) atomicMax(p.amax_bits, __float_as_uint(wm));
                }
                named_bar_sync(bar, 128);   // every read of fx_slot is done before thread 0 refills it
            }
        }
    };

    // Each setmaxnreg dominates only its own role's code and is executed by whole warpgroups.
    if (warp >= tma_warp<EPI>()) {
        if constexpr (EPI) setmaxnreg_dec<kRegsCtl>();
      if (PAGED && (warp == tma_warp<EPI>() || warp == tma_warp<EPI>() + 2)) {
        // ------------------------------------------------ paged TMA producers: one warp for K, one for Q and V
        // A tile is filled in boxes of p.box keys, each inside one page, up to the request's length (rows behind
        // it keep what the buffer held: their scores are masked and their V rows zeroed).  Lane i of the warp
        // looks up the page of box i, a tile ahead (up to four ahead measured the same or slower), and issues
        // it.  A page outside the pool loads zeros (the tensor map's fill) and sets the status.  A box takes
        // its warp some 100 cycles, whoever issues it (one elected thread: twice that), hence two warps: in pages
        // of 16, B1 500 keys 9.2 -> 8.0 us, B8 Hkv16 0..2000 keys D64 19.8 -> 16.0.
        if constexpr (PAGED) {
            using L = TileLayout<D, PAGED>;
            const int lane = static_cast<int>(lane_id()), boxes = kTileKV >> p.box_log2;
            const bool is_k = warp == tma_warp<EPI>();
            const CUtensorMap* map = is_k ? &kmap : &vmap;
            uint64_t *full = is_k ? k_full : v_full, *empty = is_k ? k_empty : v_empty;
            uint8_t* ring = smem + (is_k ? C::kOffK : C::kOffV);
            const uint64_t pol = policy_evict_first();
            Ring qr(2), r(S);
            uint32_t cnt[S], qcnt[2] = {0, 0};
            for (int n = 0; n < S; ++n) cnt[n] = 0;
            // lane 0 waits for the buffer and announces `bytes`; the warp goes on unless the CTA has aborted
            auto claim = [&](uint64_t* free, uint64_t* filled, uint32_t phase, uint32_t bytes) {
                int go = 0;
                if (lane == 0) {
                    mbar_wait(free, phase ^ 1, wc);
                    go = aborted(wc) ? 0 : 1;
                    if (go) mbar_arrive_expect_tx(filled, bytes);
                }
                return __shfl_sync(0xffffffffu, go, 0) != 0;
            };
            while (sched.next(it)) {
                if (it.t1 <= it.t0) continue;
                const int32_t* row = p.table + static_cast<size_t>(it.b) * p.max_pages;
                // this lane's box of tile t starts at key first_key(t)
                auto first_key = [&](int t) { return t * kTileKV + lane * p.box; };
                auto look_up = [&](int t) {
                    const int j = first_key(t);
                    return t < it.t1 && lane < boxes && j < it.n ? row[p.by_page.div(j)] : 0;
                };
                int next_page = look_up(it.t0);
                if (!is_k) {
                    if (claim(&q_empty[qr.idx], &q_full[qr.idx], qr.phase, C::kQBytes)) {
                        if (lane < C::kAtoms)
                            tma_load_3d(smem + C::kOffQ + qr.idx * C::kQBytes + lane * (kN * 128), &qmap, &q_full[qr.idx], lane * 64,
                                        it.chunk * p.G, it.b * (p.Hkv / p.chunks) + it.head);
                        ++qcnt[qr.idx];
                    }
                    qr.advance();
                }
                for (int t = it.t0; t < it.t1; ++t) {
                    int page = next_page;
                    next_page = look_up(t + 1);
                    const int j = first_key(t), off = j - p.by_page.div(j) * p.page;
                    const bool mine = lane < boxes && j < it.n;
                    if (mine && (page < 0 || page >= p.num_pages)) {
                        page = p.num_pages;
                        report_bad_page(p.status);
                    }
                    const int used = (min(it.n - t * kTileKV, kTileKV) + p.box - 1) >> p.box_log2;
                    const uint32_t bytes = static_cast<uint32_t>((used << p.box_log2) * 128 * C::kAtoms);
                    if (claim(&empty[r.idx], &full[r.idx], r.phase, bytes)) {
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
        }
      } else if (!PAGED && warp == tma_warp<EPI>()) {
        // ------------------------------------------------ TMA producer
        if (lane_id() == 0) {
            tma_prefetch_desc(&qmap);
            tma_prefetch_desc(&kmap);
            tma_prefetch_desc(&vmap);
            const uint64_t pol = policy_evict_first();
            Ring qr(2), kr(S), vr(S);
            uint32_t kcnt[S], vcnt[S], qcnt[2] = {0, 0};
            for (int i = 0; i < S; ++i) kcnt[i] = vcnt[i] = 0;
            while (sched.next(it)) {
                if (it.t1 <= it.t0) continue;
                mbar_wait(&q_empty[qr.idx], qr.phase ^ 1, wc);
                if (!aborted(wc)) {
                    uint8_t* dst = smem + C::kOffQ + qr.idx * C::kQBytes;
                    mbar_arrive_expect_tx(&q_full[qr.idx], C::kQBytes);
                    for (int a = 0; a < C::kAtoms; ++a)
                        tma_load_3d(dst + a * (kN * 128), &qmap, &q_full[qr.idx], a * 64, 0, it.u);
                    ++qcnt[qr.idx];
                }
                qr.advance();
                for (int t = it.t0; t < it.t1; ++t) {
                    mbar_wait(&k_empty[kr.idx], kr.phase ^ 1, wc);
                    if (!aborted(wc)) {
                        uint8_t* dst = smem + C::kOffK + kr.idx * C::kKVBytes;
                        mbar_arrive_expect_tx(&k_full[kr.idx], C::kKVBytes);
                        for (int a = 0; a < C::kAtoms; ++a)
                            tma_load_3d_hint(dst + a * (kTileKV * 128), &kmap, &k_full[kr.idx], a * 64, t * kTileKV,
                                             it.u, pol);
                        ++kcnt[kr.idx];
                    }
                    kr.advance();
                    mbar_wait(&v_empty[vr.idx], vr.phase ^ 1, wc);
                    if (!aborted(wc)) {
                        uint8_t* dst = smem + C::kOffV + vr.idx * C::kKVBytes;
                        mbar_arrive_expect_tx(&v_full[vr.idx], C::kKVBytes);
                        for (int a = 0; a < C::kAtoms; ++a)
                            tma_load_3d_hint(dst + a * (kTileKV * 128), &vmap, &v_full[vr.idx], a * 64, t * kTileKV,
                                             it.u, pol);
                        ++vcnt[vr.idx];
                    }
                    vr.advance();
                }
            }
            // nothing may still be landing in shared memory when the CTA exits
            for (int i = 0; i < S; ++i) {
                if (kcnt[i]) drain_wait(&k_full[i], (kcnt[i] - 1) & 1, kDrainLimit);
                if (vcnt[i]) drain_wait(&v_full[i], (vcnt[i] - 1) & 1, kDrainLimit);
            }
            for (int i = 0; i < 2; ++i)
                if (qcnt[i]) drain_wait(&q_full[i], (qcnt[i] - 1) & 1, kDrainLimit);
        }
      } else if (warp == mma_warp<EPI>()) {
        // ------------------------------------------------ MMA issuer
        if (lane_id() == 0) {
            constexpr uint32_t idesc_qk = idesc_bf16_f32(128, kN, false, false);
            constexpr uint32_t idesc_pv = idesc_bf16_f32(128, PAGED && NC == 16 ? 2 * kN : kN, true, true);
            using L = TileLayout<D, PAGED>;
            constexpr uint32_t lbo_v = (D >= 128) ? L::kHalf : 0u;   // D = 64: M rows 64..127 repeat 0..63
            Ring qr(2), kr(S), vr(S), sr(2), pr(2), orr(2);
            auto pv = [&]() {
                mbar_wait(&p_full[pr.idx], pr.phase, wc);
                mbar_wait(&v_full[vr.idx], vr.phase, wc);
                tc_fence_after();
                if (!aborted(wc)) {
                    const uint32_t sV = smem_u32(smem + C::kOffV + vr.idx * C::kKVBytes);
                    const uint32_t sP = smem_u32(smem + C::kOffP + pr.idx * C::kPBytes);
                    const uint32_t dO = tmem + C::o_col(NC, PAGED, orr.idx);
#pragma unroll
                    for (int ks = 0; ks < kTileKV / 16; ++ks) {
                        const uint64_t da = sdesc_sw128(sV + ks * 2 * L::kGroup, lbo_v, L::kGroup);
                        const uint64_t db = sdesc_sw32(sP + ks * 512, 2 * C::kPBytes, 256);
                        mma_ss(dO, da, db, idesc_pv, ks > 0 ? 1u : 0u);
                    }
                    mma_commit(&o_full[orr.idx]);
                    mma_commit(&v_empty[vr.idx]);
                }
                pr.advance();
                vr.advance();
                orr.advance();
            };
            // QK of a tile is issued ahead of PV of the tile before it, across work items too, so that tile's
            // softmax overlaps it
            bool behind = false;
            while (sched.next(it)) {
                if (it.t1 <= it.t0) continue;
                mbar_wait(&q_full[qr.idx], qr.phase, wc);
                const uint32_t sQ = smem_u32(smem + C::kOffQ + qr.idx * C::kQBytes);
                for (int t = it.t0; t < it.t1; ++t) {
                    mbar_wait(&k_full[kr.idx], kr.phase, wc);
                    tc_fence_after();
                    if (!aborted(wc)) {
                        const uint32_t sK = smem_u32(smem + C::kOffK + kr.idx * C::kKVBytes);
                        const uint32_t dS = tmem + sr.idx * 16;
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk) {
                            const uint64_t da = sdesc_sw128(sK + (kk >> 2) * L::kHalf + (kk & 3) * 32, 16, L::kGroup);
                            const uint64_t db = sdesc_sw128(sQ + (kk >> 2) * (kN * 128) + (kk & 3) * 32, 16, 1024);
                            mma_ss(dS, da, db, idesc_qk, kk > 0 ? 1u : 0u);
                        }
                        mma_commit(&s_full[sr.idx]);
                        mma_commit(&k_empty[kr.idx]);
                        if (t + 1 == it.t1) mma_commit(&q_empty[qr.idx]);
                    }
                    kr.advance();
                    sr.advance();
                    if (behind) pv();
                    behind = true;
                }
                qr.advance();
            }
            if (behind) pv();
            mma_commit(&mma_done);
            drain_wait(&mma_done, 0, kDrainLimit);
        }
      }
    } else if (warp < 4) {
        if constexpr (EPI) setmaxnreg_inc<kRegsSm>();
        // ------------------------------------------------ softmax / correction (128 threads)
        const int tid = threadIdx.x;
        const int lane = static_cast<int>(lane_id());
        const uint32_t lane_base = static_cast<uint32_t>(warp * 32) << 16;
        Ring sr(2), pr(2), orr(2), vr(S), hr(2);
        float acc[NC], alpha_prev[NC];   // O of the tiles before the last, and what the last tile's max makes of it
        bool moved_prev = false;
        // O of the tile before: one tile late, so that its PV runs beside the softmax of the next
        auto consume = [&]() {
            mbar_wait(&o_full[orr.idx], orr.phase, wc);
            tc_fence_after();
            uint32_t ov[NC];
            tmem_ld<NC>(tmem + lane_base + C::o_col(NC, PAGED, orr.idx), ov);
            if constexpr (PAGED) {   // and what the roundings of P left (see store_p)
                uint32_t ow[NC];
                tmem_ld<NC>(tmem + lane_base + C::o_col(NC, PAGED, orr.idx) + (NC == 16 ? 16 : 8), ow);
                tmem_ld_wait(ov, ow);
#pragma unroll
                for (int q = 0; q < NC; ++q) ov[q] = __float_as_uint(__uint_as_float(ov[q]) + __uint_as_float(ow[q]));
            } else {
                tmem_ld_wait(ov);
            }
            orr.advance();
            if (moved_prev) {
#pragma unroll
                for (int q = 0; q < NC; ++q) acc[q] = fmaf(acc[q], alpha_prev[q], __uint_as_float(ov[q]));
            } else {
#pragma unroll
                for (int q = 0; q < NC; ++q) acc[q] += __uint_as_float(ov[q]);
            }
        };
        // DEFER: an item's last O is consumed beside the next item's first tile too (Hq32 Hkv8 D128: B128 0..200 keys
        // 21.1 -> 19.5 us, B32 0..300 10.9 -> 10.5, B32 0..1500 20.4 -> 20.0).  It publishes a partial later, which a
        // merge waits for: B4 0..6000 16.4 -> 16.6, and with 16 columns B17 Hq16 Hkv4 Sq4 D64 20.1 -> 21.7, dense
        // speculative decode (B8 Hq32 Hkv8 Sq4 8192 keys) 43.8 -> 45.6.  Deferring whole items alone takes most of
        // the gain away (21.0 for the first).
        constexpr bool DEFER = PAGED && NC <= 8;
        bool pending = false;   // an item whose last O is still to come
        // hands it to the epilogue warpgroup, with acc and the partial column sums through Tensor Memory (lane tid)
        // and the reference maxima through shared memory, the sums and maxima at the item's end; the softmax goes on
        // meanwhile.  Both sides walk the same item sequence and take part in every handoff whatever their waits
        // return (a timeout only drains).
        auto hand_off = [&]() {
            __syncwarp();   // tcgen05.st is warp-collective
            uint32_t hv[NC];
#pragma unroll
            for (int q = 0; q < NC; ++q) hv[q] = __float_as_uint(acc[q]);
            tmem_st<NC>(tmem + lane_base + 64 + hr.idx * 32, hv);
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ep_full[hr.idx]);
            hr.advance();
            pending = false;
#pragma unroll
            for (int q = 0; q < NC; ++q) acc[q] = 0.f;
        };
#pragma unroll
        for (int q = 0; q < NC; ++q) acc[q] = 0.f;
        for (;;) {
            const bool more = sched.next(it);
            if constexpr (DEFER) {
                if (pending && !(more && it.t1 > it.t0)) {   // no tile comes to consume the last O beside
                    consume();
                    hand_off();
                }
            }
            if (!more) break;
            const int G = unit_cols<PAGED>(p, it);
            float m[NC], l[NC];
            // keys visible to column q: 0 .. lim[q] - 1 (causal: query q % Sq sees keys up to
            // (q % Sq) + n - Sq; otherwise all n)
            int lim[NC];
#pragma unroll
            for (int q = 0; q < NC; ++q)
                lim[q] = CAUSAL ? it.n - p.Sq + 1 + (((PAGED ? it.chunk * p.G : 0) + q) % p.Sq) : it.n;
#pragma unroll
            for (int q = 0; q < NC; ++q) {
                m[q] = q < G ? -INFINITY : INFINITY;   // a column without a query: P = 0, never the largest
                l[q] = 0.f;
            }
            for (int t = it.t0; t < it.t1; ++t) {
                mbar_wait(&s_full[sr.idx], sr.phase, wc);
                tc_fence_after();
                uint32_t sv[NC];
                tmem_ld<NC>(tmem + lane_base + sr.idx * 16, sv);
                tmem_ld_wait(sv);
                sr.advance();

                const int kv = t * kTileKV + tid;
                const bool valid = kv < it.n;
                // Lazy column max (as the row-tile kernel's lazy rescale): the reference m[q] moves only
                // when some score of column q exceeds it by more than 2^8, so P <= 256 and the final
                // O = acc / L and LSE = m + log2 L are exact for any reference.  Usually no column
                // moves and no max is reduced: one barrier that also ORs a flag decides.
                float x[NC], pv[NC];
                bool above = false;
#pragma unroll
                for (int q = 0; q < NC; ++q) {
                    x[q] = (CAUSAL ? kv < lim[q] : valid) ? __uint_as_float(sv[q]) * p.c : -INFINITY;
                    above |= x[q] > m[q] + kRescaleD;
                }
                const bool moved = bar_any128(1, above);   // the same in all four warps
                float alpha[NC];
                if (moved) {
#pragma unroll
                    for (int q = 0; q < NC; ++q) {
                        const float mx = redux_max(x[q]);
                        if (lane == 0) red_max[warp][q] = mx;
                    }
                    named_bar_sync(1, 128);
#pragma unroll
                    for (int q = 0; q < NC; ++q) {
                        const float mt = fmaxf(fmaxf(red_max[0][q], red_max[1][q]), fmaxf(red_max[2][q], red_max[3][q]));
                        const bool up = mt > m[q] + kRescaleD;
                        // a column without a finite reference yet has nothing to rescale
                        alpha[q] = !up ? 1.f : m[q] == -INFINITY ? 0.f : ex2_approx(m[q] - mt);
                        m[q] = up ? mt : m[q];
                    }
                }
                // a column with no visible key so far keeps m = -inf: its scores are -inf, and so is x - 0
#pragma unroll
                for (int q = 0; q < NC; ++q) {
                    pv[q] = ex2_approx(x[q] - (m[q] == -INFINITY ? 0.f : m[q]));
                    l[q] = moved ? fmaf(l[q], alpha[q], pv[q]) : l[q] + pv[q];
                }
                // Keys at or beyond n in a partial tile: their V rows may hold anything (NaN in
                // padded memory) and P = 0 does not cancel NaN in the MMA, so zero those rows.
                // Whole 128-byte rows are zeroed, which the swizzle only permutes within, each thread its own in
                // an order that keeps a warp's stores on different banks.
                if ((t + 1) * kTileKV > it.n) {
                    mbar_wait(&v_full[vr.idx], vr.phase, wc);
                    if (!valid) {
                        uint8_t* rowp = smem + C::kOffV + vr.idx * C::kKVBytes + TileLayout<D, PAGED>::row(tid);
#pragma unroll
                        for (int a = 0; a < C::kAtoms; ++a)
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                reinterpret_cast<uint4*>(rowp + a * TileLayout<D, PAGED>::kHalf)[i ^ (tid & 7)] = make_uint4(0, 0, 0, 0);
                    }
                }
                vr.advance();
                // other columns of P keep what they held: they only reach columns of O that nobody reads
                uint8_t* sP = smem + C::kOffP + pr.idx * C::kPBytes;
                store_p<NC, PAGED>(sP, sP + 2 * C::kPBytes, tid, pv);
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[pr.idx]);
                pr.advance();
                if (t > it.t0 || (DEFER && pending)) consume();
                if (DEFER && pending) hand_off();
                moved_prev = moved;
                if (moved)
#pragma unroll
                    for (int q = 0; q < NC; ++q) alpha_prev[q] = alpha[q];
            }
            if constexpr (EPI) {
                mbar_wait(&ep_empty[hr.idx], hr.phase ^ 1, wc);
                tc_fence_after();
                __syncwarp();
                uint32_t hv[NC];
#pragma unroll
                for (int q = 0; q < NC; ++q) hv[q] = __float_as_uint(l[q]);
                tmem_st<NC>(tmem + lane_base + 64 + NC + hr.idx * 32, hv);
                if (tid == 0)
#pragma unroll
                    for (int q = 0; q < NC; ++q) ep_m[hr.idx][q] = m[q];
                if (DEFER && it.t1 > it.t0) {
                    pending = true;
                } else {
                    if (it.t1 > it.t0) consume();
                    hand_off();
                }
            } else {
                if (it.t1 > it.t0) consume();
                run_epilogue(it, it.t1 <= it.t0, m, l, acc, tid, warp, 1, false);
#pragma unroll
                for (int q = 0; q < NC; ++q) acc[q] = 0.f;
            }
        }
    } else {
      if constexpr (EPI) {
        setmaxnreg_inc<kRegsEpi>();
        // ------------------------------------------------ epilogue (128 threads): the items the softmax
        // warpgroup hands over, in order; thread tid owns O^T row tid (Tensor Memory lane tid)
        const int tid = threadIdx.x - 128;
        const int ew = warp - 4;
        const uint32_t lane_base = static_cast<uint32_t>(ew * 32) << 16;
        Ring hr(2);
        while (sched.next(it)) {   // the softmax warpgroup's sequence of items
            // a partial's slots (64-bit divisions) while the softmax warps still stream the item, off
            // the path from its last tile to its arrival count
            const bool partial = p.fixup && !(it.whole && !(p.split && p.nv_codes)) && it.t1 > it.t0;
            if (partial && tid == 0) fx_n = partial_slots(it);
            mbar_wait(&ep_full[hr.idx], hr.phase, wc);
            tc_fence_after();
            __syncwarp();   // tcgen05.ld is warp-collective
            const bool empty = it.t1 <= it.t0;
            float m[NC], l[NC], acc[NC];
            {
                uint32_t hv[2 * NC];
                tmem_ld<2 * NC>(tmem + lane_base + 64 + hr.idx * 32, hv);
                tmem_ld_wait(hv);
#pragma unroll
                for (int q = 0; q < NC; ++q) {
                    acc[q] = __uint_as_float(hv[q]);
                    l[q] = __uint_as_float(hv[NC + q]);
                    m[q] = ep_m[hr.idx][q];
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane_id() == 0) mbar_arrive(&ep_empty[hr.idx]);
            hr.advance();

            run_epilogue(it, empty, m, l, acc, tid, ew, 2, partial);
        }
      }
    }

    tc_fence_before();
    __syncthreads();
    if constexpr (!REST) {
        if (warp == mma_warp<EPI>()) tmem_dealloc(tmem, C::tmem_cols(NC, PAGED));
    }
    if constexpr (PAGED && !REST) {
        const int B = p.U / p.Hkv;
        if (cta == 0)
            for (int b = threadIdx.x; b < B; b += blockDim.x)
                if (p.seqlens[b] < 0 || p.seqlens[b] > p.cap) report_bad_page(p.status);
        if (p.fixup)   // no combine kernel runs: entries without keys are written here
            for (int b = cta; b < B; b += ctas)
                if (pre[b + 1] == pre[b]) write_empty_entry(p, b);
    }
}

template <int D, bool CAUSAL, int NC, bool PAGED = false>
__global__ void __launch_bounds__(decode_threads<has_epilogue_warps<NC, PAGED>()>(), 1)
    decode_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                  const __grid_constant__ CUtensorMap vmap, const __grid_constant__ DecodeParams p)
{
    extern __shared__ uint8_t smem_raw[];
    __shared__ DecodeShared<D, PAGED> sh;
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    decode_body<D, CAUSAL, NC, PAGED, false>(qmap, kmap, vmap, p, sh, smem, static_cast<int>(blockIdx.x), static_cast<int>(gridDim.x), RestPlan{});
}

// Exclusive prefix of per-unit tile counts (ragged keys), one block.
template <bool PAGED>
__global__ void __launch_bounds__(1024) tile_prefix_kernel(const __grid_constant__ DecodeParams p, int32_t* prefix)
{
    // dense: the units' tiles; paged: the batch entries' tiles
    const int U = PAGED ? p.U / p.Hkv : p.U, per_entry = PAGED ? 1 : p.Hkv;
    griddep_launch_dependents();
    griddep_wait();
    __shared__ int part[1024];
    const int per = (U + 1023) / 1024;
    const int b0 = threadIdx.x * per;
    int s = 0;
    int with_keys = 0;
    if constexpr (PAGED)
        for (int u = b0; u < min(U, b0 + per); ++u) with_keys += batch_keys<PAGED>(p, u) > 0 ? 1 : 0;
    for (int u = b0; u < min(U, b0 + per); ++u) s += (batch_keys<PAGED>(p, u / per_entry) + kTileKV - 1) / kTileKV;
    part[threadIdx.x] = s;
    __syncthreads();
    for (int off = 1; off < 1024; off <<= 1) {
        const int v = threadIdx.x >= off ? part[threadIdx.x - off] : 0;
        __syncthreads();
        part[threadIdx.x] += v;
        __syncthreads();
    }
    int run = threadIdx.x ? part[threadIdx.x - 1] : 0;
    for (int u = b0; u < min(U, b0 + per); ++u) {
        prefix[u] = run;
        run += (batch_keys<PAGED>(p, u / per_entry) + kTileKV - 1) / kTileKV;
    }
    if (threadIdx.x == 1023) prefix[U] = part[1023];
    if constexpr (PAGED) {   // and the CTAs that the tiles are split over
        const int total = part[1023];
        __syncthreads();
        part[threadIdx.x] = with_keys;
        __syncthreads();
        if (threadIdx.x == 0) {
            int n = 0;
            for (int i = 0; i < 1024; ++i) n += part[i];
            prefix[U + 1] = paged_ctas(total * p.Hkv, n * p.Hkv, p.ctas);
        }
    }
}

// Merges the partial results of units whose tiles were split over several CTAs, and writes the
// result of units without keys (O = 0, LSE = -inf).  One block of D threads per query row; warp 0
// finds the CTAs holding partials of the unit once per block (64-bit divisions).
constexpr int kMaxPartsD = 512;

template <bool PAGED = false>
__global__ void combine_kernel(const __grid_constant__ DecodeParams p, int nctas)
{
    __shared__ int slots[kMaxPartsD];
    __shared__ float weights[kMaxPartsD];
    __shared__ int nslots;
    __shared__ float lse_sh;
    griddep_launch_dependents();
    griddep_wait();
    const int row = blockIdx.x;
    const int u = row / p.G;
    const int q = row % p.G;
    Item it{};
    it.u = u;
    if constexpr (PAGED) {
        place_unit(p, it, u / p.Hkv, u % p.Hkv);
        if (q >= unit_cols<PAGED>(p, it)) return;   // the last chunk of a head may have fewer rows
    }
    const int d = threadIdx.x;
    const int D = p.D;
    if (threadIdx.x < 32) {
        int cnt = 0;
        if constexpr (PAGED) {
            if (threadIdx.x == 0) {
                const int B = p.U / p.Hkv;
                Line line;
                line.T = p.prefix[B] * p.Hkv;
                line.P = p.prefix[B + 1];
                cnt = paged_partial_slots(p, p.prefix, line, it.b, it.head * p.chunks + it.chunk, slots, kMaxPartsD);
            }
            cnt = __shfl_sync(0xffffffffu, cnt, 0);
            if (cnt == 1 && !p.nv_codes) cnt = -1;   // one CTA held the whole unit and wrote it
        } else {
            int tiles;
            long long Tu, T;
            if (p.prefix) {
                tiles = p.prefix[u + 1] - p.prefix[u];
                Tu = p.prefix[u];
                T = p.prefix[p.U];
            } else {
                tiles = p.tiles_uniform;
                Tu = static_cast<long long>(u) * tiles;
                T = static_cast<long long>(p.U) * tiles;
            }
            if (tiles > 0) {
                const long long P = nctas;
                const int c0 = static_cast<int>(min((((Tu + 1) * P) - 1) / T, P - 1));
                const int c1 = static_cast<int>(min((((Tu + tiles) * P) - 1) / T, P - 1));
                if (c0 == c1 && !p.nv_codes) {
                    cnt = -1;   // one CTA held the whole unit and wrote it
                } else {
                    for (int cw = c0; cw <= c1; cw += 32) {
                        const int c = cw + static_cast<int>(threadIdx.x);
                        // CTAs with an empty tile range (possible when T < P) hold no partial
                        const bool ok = c <= c1 && (c * T) / P != ((c + 1) * T) / P;
                        const unsigned m = __ballot_sync(0xffffffffu, ok);
                        if (ok) {
                            const int idx = cnt + __popc(m & ((1u << threadIdx.x) - 1u));
                            if (idx < kMaxPartsD) slots[idx] = u + c;
                        }
                        cnt += __popc(m);
                    }
                    cnt = min(cnt, kMaxPartsD);
                }
            }
        }
        __syncwarp();
        // LSE of the merged row and each partial's weight exp(lse_i - lse), once per block
        float mx = -INFINITY;
        for (int i = static_cast<int>(threadIdx.x); i < cnt; i += 32) mx = fmax_nan(mx, p.part_lse[static_cast<size_t>(slots[i]) * kN + q]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mx = fmax_nan(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        // partials without a visible key carry lse = -inf and weigh 0; all of them -> empty row
        const bool any = mx != -INFINITY;
        float sum = 0.f;
        if (any)
            for (int i = static_cast<int>(threadIdx.x); i < cnt; i += 32) sum += __expf(p.part_lse[static_cast<size_t>(slots[i]) * kN + q] - mx);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        const float lse_all = (cnt > 0 && any) ? mx + __logf(sum) : -INFINITY;
        for (int i = static_cast<int>(threadIdx.x); i < cnt; i += 32)
            weights[i] = any ? __expf(p.part_lse[static_cast<size_t>(slots[i]) * kN + q] - lse_all) : 0.f;
        if (threadIdx.x == 0) {
            nslots = cnt;
            lse_sh = lse_all;
        }
    }
    __syncthreads();
    const int ns = nslots;
    if (ns < 0) return;
    float o = 0.f;
    const float lse_v = lse_sh;
#pragma unroll 4
    for (int i = 0; i < ns; ++i) o = fmaf(weights[i], p.part_o[(static_cast<size_t>(slots[i]) * kN + q) * D + d], o);
    const size_t r = unit_row0<PAGED>(p, it) + q;
    if (p.o_stage) p.o_stage[r * D + d] = o;
    if (p.out) {
        if (p.out_f32)
            static_cast<float*>(p.out)[r * D + d] = o;
        else
            static_cast<uint16_t*>(p.out)[r * D + d] = float_to_bf16_bits(o);
    }
    if (d == 0 && p.lse) p.lse[r] = lse_v;
    if (p.nv_codes) nvfp4_encode_lanes(o, *p.nv_sg, d, p.nv_codes + r * (D / 2), p.nv_scales + r * (D / 16));
    if (p.amax_bits) {
        const float wm = warp_max(fabsf(o));
        if ((threadIdx.x & 31) == 0 && wm > 0.f) atomicMax(p.amax_bits, __float_as_uint(wm));
    }
}

}  // namespace

}  // namespace atc_gb300
