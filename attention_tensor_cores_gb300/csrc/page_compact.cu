// Used pages to the low ids (fmha_page_compact): where each goes, the block table that says so, the moves and
// the stack of free pages.
//
// With n free pages of N, U = N - n are used.  The k-th used page with an id of at least U (ascending) moves to the
// k-th free id below U; as many of either exist.  With f(x) the number of free pages below x, a used page x >= U is
// the (x - U - (f(x) - f(U)))-th to move, and f(U) pages move in all.
//
// One CTA, or clusters of eight.  Each reads the whole stack into a set of bits that every CTA of it gets a copy of, and sums
// it in blocks of 256 pages: f is a sum and up to eight popcounts, its inverse a binary search and as many, for each page that
// moves.  The stack names each page once if the set has as many bits as it has entries.  The tables' new entries are looked up
// in new_ids, by the one CTA or by a second launch (with f and its inverse for each entry: 13,000 cycles of 34,000).
// Bound: latency, stack -> set -> copy -> new ids -> tables.
#include <cuda_runtime.h>

#include "cluster_bits.cuh"
#include "fastdiv.cuh"
#include "paged.h"
#include "ptx.cuh"

namespace atc_gb300 {
namespace {

constexpr int kCompactThreads = 1024;
constexpr int kCompactCtas = 8;              // of a cluster
constexpr int kMaxCompactPages = 1 << 20;

struct CompactParams {
    const int32_t* seqlens;
    int B, page;
    FastDiv by_page;
    const int32_t* table;
    int max_pages;
    const int32_t* free_pages;
    const int32_t* free_count;
    int num_pages;
    int32_t* new_ids;
    int32_t* new_table;
    int32_t* src;
    int32_t* dst;
    int cap;
    int32_t* moves;
    int32_t* free_out;
    int* status;
    int blocks;   // runs of 256 pages, 8 words of the set each
};

// The rows' new entries from new_ids, by `step` threads of which this is the first-th: a warp for 128 entries at a time,
// several warps a row where there are more of them
__device__ __forceinline__ void translate_rows(const CompactParams& p, int first, int step)
{
    const int lane = static_cast<int>(lane_id()), warps = step / 32, shared = max(1, min((p.max_pages + 127) / 128, warps / max(p.B, 1)));
    const long long room = static_cast<long long>(p.max_pages) * p.page;
    bool odd = false;
    for (int v = first / 32; v < p.B * shared; v += warps) {
        const int b = v / shared;
        const long long len = p.seqlens[b], held_tokens = len < 0 ? 0 : len > room ? room : len;
        const int k = p.by_page.up(static_cast<int>(held_tokens));
        const size_t row = static_cast<size_t>(b) * p.max_pages;
        for (int s = v - b * shared; static_cast<long long>(s) * 128 < k; s += shared) {
            int x[4], to[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int j = s * 128 + u * 32 + lane;
                x[u] = j < k ? p.table[row + j] : 0;
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) to[u] = x[u] >= 0 && x[u] < p.num_pages ? __ldcg(p.new_ids + x[u]) : -1;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int j = s * 128 + u * 32 + lane;
                if (j >= k) continue;
                odd = odd || to[u] < 0;   // no page, or a free one
                p.new_table[row + j] = to[u] < 0 ? x[u] : to[u];
            }
        }
    }
    if (odd) report_bad_page(p.status);
}

template <int CTAS>
__global__ void __cluster_dims__(CTAS, 1, 1) __launch_bounds__(kCompactThreads, 1) page_compact_kernel(const __grid_constant__ CompactParams p)
{
    extern __shared__ uint32_t bits[];                                   // the set
    const int words = p.blocks * 8;
    uint32_t* slice = bits + words;                                      // this CTA's blocks of the joined one
    int* below = reinterpret_cast<int*>(slice + (CTAS > 1 ? p.blocks + 8 * CTAS : 0));   // free pages before each block
    __shared__ int sums[32];
    griddep_launch_dependents();
    const int tid = threadIdx.x, N = p.num_pages;
    const int rank = CTAS > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    for (int i = tid; i < words; i += kCompactThreads) bits[i] = 0;
    griddep_wait();
    __syncthreads();

    const int n = *p.free_count;
    const long long room = static_cast<long long>(p.max_pages) * p.page;
    bool bad = n < 0 || n > N;
    const auto fine = [&](int page) { return page >= 0 && page < N; };
    if (!bad)
#pragma unroll 8
        for (int i = rank * kCompactThreads + tid; i < n; i += CTAS * kCompactThreads) {
            const int x = p.free_pages[i];
            if (fine(x)) set_bit(bits, x);
        }
    for (int b = tid; b < p.B; b += kCompactThreads) {
        const int c = p.seqlens[b];
        bad = bad || c < 0 || c > room;
    }
    bad = __syncthreads_or(bad);
    if constexpr (CTAS > 1) {
        const int per = (words + CTAS - 1) / CTAS;
        cluster_sync();   // all sets are marked
        for (int i = tid; i < per; i += kCompactThreads) slice[i] = rank * per + i < words ? joined_word<CTAS>(bits, rank * per + i) : 0u;
        cluster_sync();   // all slices are joined, and nobody looks at the sets any more
        for (int i = tid; i < words; i += kCompactThreads) {
            const int r = i / per;
            bits[i] = ld_cluster(mapa_shared(smem_u32(slice + (i - r * per)), static_cast<uint32_t>(r)));
        }
        cluster_sync();   // nobody looks into another CTA's memory from here on
    }

    const auto count_block = [&](int k) {
        int c = 0;
#pragma unroll
        for (int w = 0; w < 8; ++w) c += __popc(bits[k * 8 + w]);
        return c;
    };
    const int per = (p.blocks + kCompactThreads - 1) / kCompactThreads;
    const int k0 = min(p.blocks, tid * per), k1 = min(p.blocks, k0 + per);
    int own = 0, total;
    for (int k = k0; k < k1; ++k) own += count_block(k);
    int at = block_scan(own, sums, total);
    for (int k = k0; k < k1; ++k) {
        below[k] = at;
        at += count_block(k);
    }
    __syncthreads();
    bad = bad || total != n;   // an entry that is no page, or twice the same

    const auto is_free = [&](int x) { return (bits[x >> 5] >> (x & 31)) & 1; };
    // free pages below x < N
    const auto free_below = [&](int x) {
        int c = below[x >> 8];
        for (int w = (x >> 8) * 8; w < x >> 5; ++w) c += __popc(bits[w]);
        return c + __popc(bits[x >> 5] & ((1u << (x & 31)) - 1));
    };
    // the k-th free page
    const auto nth_free = [&](int k) {
        int lo = 0, hi = p.blocks - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (below[mid] <= k) lo = mid; else hi = mid - 1;
        }
        k -= below[lo];
        int w = lo * 8;
        for (int c; k >= (c = __popc(bits[w])); ++w) k -= c;
        const uint32_t v = bits[w];
        int pos = 0;
#pragma unroll
        for (int h = 16; h > 0; h >>= 1) {
            const int c = __popc((v >> pos) & ((1u << h) - 1));
            if (k >= c) {
                k -= c;
                pos += h;
            }
        }
        return w * 32 + pos;
    };
    const int U = N - n;
    const int M = bad || U == N ? 0 : free_below(U);
    // a used page's place among those that move
    const auto mover = [&](int x) { return x - U - (free_below(x) - M); };

    const int first = blockIdx.x * kCompactThreads + tid, step = gridDim.x * kCompactThreads;
    for (int x = first; x < N; x += step) {
        int to = x;
        if (!bad) {
            if (is_free(x)) {
                to = -1;
            } else if (x >= U) {
                const int k = mover(x);
                to = nth_free(k);
                p.src[k] = x;
                p.dst[k] = to;
            }
        }
        p.new_ids[x] = to;
        if (x < n) p.free_out[x] = bad ? p.free_pages[x] : N - 1 - x;
    }
    for (int k = M + first; k < p.cap; k += step) p.src[k] = p.dst[k] = -1;
    if (first == 0) {
        *p.moves = M;
        if (bad) report_bad_page(p.status);
    }
    if constexpr (CTAS == 1) {
        __syncthreads();   // the new ids are written
        translate_rows(p, first, step);
    }
}

__global__ void __launch_bounds__(256) page_translate_kernel(const __grid_constant__ CompactParams p)
{
    griddep_launch_dependents();
    griddep_wait();
    translate_rows(p, blockIdx.x * 256 + threadIdx.x, gridDim.x * 256);
}

}  // namespace
}  // namespace atc_gb300

using namespace atc_gb300;

extern "C" int fmha_page_compact(const int32_t* seqlens, int B, int page_size, const int32_t* block_table, int max_pages,
                                 const int32_t* free_pages, const int32_t* free_count, int num_pages, int32_t* new_ids, int32_t* new_table,
                                 int32_t* copy_src, int32_t* copy_dst, int n_copies, int32_t* copy_count, int32_t* free_pages_out,
                                 fmha_stream_t stream)
{
    if (B < 0 || page_size < 1 || num_pages < 1 || max_pages < 1 || n_copies < num_pages / 2)
        return set_error(FMHA_ERR_INVALID, "fmha_page_compact: need B >= 0, page_size, num_pages and max_pages >= 1, n_copies >= num_pages / 2");
    if (!free_pages || !free_count || !new_ids || !copy_count || !free_pages_out || (n_copies > 0 && (!copy_src || !copy_dst)) ||
        (B > 0 && (!seqlens || !block_table || !new_table)))
        return set_error(FMHA_ERR_INVALID, "fmha_page_compact: NULL pointer");
    for (const void* x : {static_cast<const void*>(seqlens), static_cast<const void*>(block_table), static_cast<const void*>(free_pages),
                          static_cast<const void*>(free_count), static_cast<const void*>(new_ids), static_cast<const void*>(new_table),
                          static_cast<const void*>(copy_src), static_cast<const void*>(copy_dst), static_cast<const void*>(copy_count),
                          static_cast<const void*>(free_pages_out)})
        if (misaligned(x, 4)) return set_error(FMHA_ERR_INVALID, "fmha_page_compact: arrays must be 4-byte aligned");
    if (free_pages_out == free_pages || (B > 0 && new_table == block_table))
        return set_error(FMHA_ERR_INVALID, "fmha_page_compact: new_table and free_pages_out must not be block_table and free_pages");
    if (static_cast<long long>(max_pages) * page_size > (1LL << 31) - 256 || num_pages > kMaxCompactPages || n_copies > (1 << 30) || B > (1 << 24))
        return set_error(FMHA_ERR_UNSUPPORTED, "fmha_page_compact: max_pages * page_size past 2^31, more than 2^20 pages, 2^24 requests or 2^30 copies");
    int* status = device_status_ptr();
    if (!status) return set_error(FMHA_ERR_CUDA, "no CUDA device");
    const int blocks = (num_pages + 255) / 256;
    const CompactParams p{seqlens, B, page_size, FastDiv(static_cast<uint32_t>(page_size)), block_table, max_pages, free_pages, free_count,
                          num_pages, new_ids, new_table, copy_src, copy_dst, n_copies, copy_count, free_pages_out, status, blocks};
    // A CTA for up to 8192 pages and tables of as many entries; else a cluster for each 32768 pages, up to eight (more would not all be
    // on the GPU at a time: a cluster's SMs are neighbours)
    const long long entries = static_cast<long long>(B) * max_pages;
    const bool one = num_pages <= 8192 && entries <= 8192;
    const int clusters = 1 + num_pages / 32768 < 8 ? 1 + num_pages / 32768 : 8;
    const auto kernel = one ? page_compact_kernel<1> : page_compact_kernel<kCompactCtas>;
    const int smem = 36 * blocks + (one ? 0 : 4 * (blocks + 8 * kCompactCtas));
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    FMHA_CHECK_CUDA(set_smem_limit_once(reinterpret_cast<const void*>(kernel), 40 * (kMaxCompactPages / 256) + 4 * 8 * kCompactCtas));
    FMHA_CHECK_CUDA(launch_pdl(kernel, dim3(static_cast<unsigned>(one ? 1 : clusters * kCompactCtas)), dim3(kCompactThreads), static_cast<size_t>(smem), st, p));
    count_launch();
    if (!one && B > 0) {
        const long long most = 4LL * (num_sms() > 0 ? num_sms() : 1), want = (entries + 1023) / 1024;
        FMHA_CHECK_CUDA(launch_pdl(page_translate_kernel, dim3(static_cast<unsigned>(want < most ? want : most)), dim3(256), 0, st, p));
        count_launch();
    }
    return FMHA_OK;
}
