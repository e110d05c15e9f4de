// How the key tiles of fmha_fwd_prefix are cut for its CTAs, and which pieces of a row's keys that makes: the attention kernel and
// the merge find out the same.
#pragma once
#include "paged_run.cuh"
#include "prefix.h"

namespace atc_gb300 {
namespace {

// What a unit costs: a key tile of it, and that there is one more (its queries, its first tile, its partials).  A cut leaves
// `least` tiles on either side, or the unit whole.
struct UnitCost {
    int tile = 1, start = 0, least = kMinPiece;
    __host__ __device__ int of(int nt) const { return start + nt * tile; }
};

// In 0.05 us, where memory does not bound it: least squares over the CTAs' times in 13 problems of Hq32 Hkv8 D128 and Hq16 Hkv4 D64
// (of D = 128 and D = 64).  The lines of units are cut where the costs are equal; by tiles alone the CTAs with the end of one unit
// and the beginning of the next were the last by 7 us.
// The least pieces, us a call from a graph (Hq32 Hkv8 D128): own keys of few rows of 4 tiles at least instead of 1, 64 requests behind
// 8192 keys 45.1 for 43.2; common ones of two row tiles of 1 or 3 instead of 2, 64 behind 2048 27.8 and 28.3 for 25.0; of one
// row tile of 2 instead of 3, 32 behind 4096 25.7 for 25.2, of 4, Hq16 Hkv4 Sq4 D64 16 groups of 4 behind up to 5001 36.5 for 34.2.
template <int D>
struct Cost {
    __host__ __device__ static UnitCost common(bool two)   // a row tile of each side, or one for both
    {
        return two ? UnitCost{D == 128 ? 42 : 37, D == 128 ? 105 : 50, 2} : UnitCost{D == 128 ? 22 : 16, D == 128 ? 80 : 40, 3};
    }
    __host__ __device__ static UnitCost own(bool many)     // more than 8 rows, which 16 columns hold
    {
        return {D == 128 ? (many ? 13 : 11) : (many ? 12 : 9), many ? 42 : 11, many ? kMinPiece : 1};
    }
    // A tile that each request reads for itself, from memory or from L2; a row in the merge.  Shared and one by one, us: groups of
    // requests 64 x 2 behind 500 to 1000 keys 68.9 and 56.6, behind 1000 to 2000 94.3 and 109.3, 256 x 2 behind 300 to 500 152.8 and
    // 140.7, behind 1000 265.2 and 320.3, 4 x 64 behind 128 63.5 and 52.0 (Hq32 Hkv8 D128); D = 64, 64 x 2 behind 1000 to 2000 72.8 and 65.0.
    static constexpr int kAgain = D == 128 ? 20 : 12, kMerge = 5;
    // what CTAs of common keys take more than those of own keys, whatever their part
    static constexpr float start(bool two) { return D == 128 ? (two ? 120.f : 80.f) : (two ? 60.f : 40.f); }
    static constexpr float kRead = D == 128 ? 0.18f : 0.09f;    // a tile from memory, with all SMs
    static constexpr float kFirst = D == 128 ? 240.f : 180.f;   // from the beginning of the reads to a CTA's common keys, and from these to its end
};
constexpr int kByTiles = 1 << 16;   // in the plan, beside the CTAs of a line that counts tiles
// With more tiles the sums of costs would pass 31 bits; each tile counts as one then
constexpr long long kMaxWeighed = 1 << 23;

// The cut at x, from the unit's place on: the first tile behind it of nt (0 or nt when it is not inside)
__device__ __forceinline__ int tile_at(int x, int nt, UnitCost u)
{
    if (x <= u.start) return 0;
    const int t = static_cast<int>(static_cast<unsigned>(x - u.start) / static_cast<unsigned>(u.tile));
    if (t >= nt) return nt;
    return 2 * t <= nt ? (t < u.least ? 0 : t) : (nt - t < u.least ? nt : t);
}

}  // namespace
}  // namespace atc_gb300
