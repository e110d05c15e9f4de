// Sets of pages as bits in shared memory, filled by the CTAs of a cluster together: each marks what it reads in a
// whole set of its own, and the parts of the eight meet in an OR, a slice per CTA, so the order of the marks does not show.
// (Marks straight into a set spread over the cluster's memory cost one SM-to-SM atomic each: a compaction of 300,000 pages took
// 63.4 us so, 17.4 with this and the tables translated from new_ids; a fork of 512 beams of 16384 tokens 27.9, now 9.1.)
#pragma once
#include "ptx.cuh"

namespace atc_gb300 {
namespace {

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

// Every thread of the CTAs that work together
template <int CTAS>
__device__ __forceinline__ void sync_ctas()
{
    if constexpr (CTAS > 1)
        cluster_sync();
    else
        __syncthreads();
}

__device__ __forceinline__ void set_bit(uint32_t* bits, int i) { atomicOr(&bits[i >> 5], 1u << (i & 31)); }

// Word w of the OR of the CTAs' sets
template <int CTAS>
__device__ __forceinline__ uint32_t joined_word(const uint32_t* bits, int w)
{
    if constexpr (CTAS == 1) {
        return bits[w];
    } else {
        uint32_t v = 0;
#pragma unroll
        for (int r = 0; r < CTAS; ++r) v |= ld_cluster(mapa_shared(smem_u32(bits + w), static_cast<uint32_t>(r)));
        return v;
    }
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
