// Sets of pages as bits in the shared memory of a cluster of eight CTAs: CTA r holds the pages
// [32 * words * r, 32 * words * (r + 1)), so a set of 2^20 pages takes 16 KB of each, and the eight SMs
// look at the lists and tables that fill it together.  What threads do to a set is an OR or an AND, whose
// order does not show.
#pragma once
#include "ptx.cuh"

namespace atc_gb300 {
namespace {

constexpr int kClusterCtas = 8;
constexpr int kMaxPoolPages = 1 << 20;

struct PageBits {
    uint32_t base;   // shared::cta address of this CTA's words
    int words;       // of each CTA

    // shared::cluster address of page's word
    __device__ __forceinline__ uint32_t at(int page) const
    {
        const int w = page >> 5, r = w / words;
        return mapa_shared(base + static_cast<uint32_t>(w - r * words) * 4, static_cast<uint32_t>(r));
    }
    __device__ __forceinline__ void set(int page) const
    {
        asm volatile("red.relaxed.cluster.shared::cluster.or.b32 [%0], %1;" ::"r"(at(page)), "r"(1u << (page & 31)) : "memory");
    }
    // sets it; was it set?
    __device__ __forceinline__ bool test_set(int page) const
    {
        uint32_t old;
        asm volatile("atom.relaxed.cluster.shared::cluster.or.b32 %0, [%1], %2;" : "=r"(old) : "r"(at(page)), "r"(1u << (page & 31)) : "memory");
        return (old >> (page & 31)) & 1;
    }
    // most pages that are cleared were not set: they cost a read
    __device__ __forceinline__ void clear(int page) const
    {
        const uint32_t a = at(page), bit = 1u << (page & 31);
        uint32_t v;
        asm volatile("ld.relaxed.cluster.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
        if (v & bit) asm volatile("red.relaxed.cluster.shared::cluster.and.b32 [%0], %1;" ::"r"(a), "r"(~bit) : "memory");
    }
};

__device__ __forceinline__ uint32_t ld_cluster(uint32_t caddr)
{
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(caddr) : "memory");
    return v;
}

__device__ __forceinline__ void st_cluster(uint32_t caddr, uint32_t v)
{
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(caddr), "r"(v) : "memory");
}

// Exclusive sum of v over the block's threads (a whole number of warps), and the total; sums: 32 ints.
// Every thread of the block takes part; ends with the barrier behind which `sums` is free again.
__device__ __forceinline__ int block_scan(int v, int* sums, int& total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    int inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += u;
    }
    if (lane == 31) sums[warp] = inc;
    __syncthreads();
    const int mine = lane < nw ? sums[lane] : 0;
    int all = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, all, o);
        if (lane >= o) all += u;
    }
    total = __shfl_sync(0xffffffffu, all, 31);
    const int before = __shfl_sync(0xffffffffu, all - mine, warp);
    __syncthreads();
    return before + inc - v;
}

}  // namespace
}  // namespace atc_gb300
