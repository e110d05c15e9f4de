// The next step's requests as children of this step's (fmha_page_fork): block table, pages given back and
// pages to be copied.
//
// Old request i of ctx_i tokens holds the first ceil(ctx_i / P) pages of its row.  With first_i its lowest
// child (none: the request ends):
//
//   kept = pages of rows with a child, gone = pages of rows without;   freed = gone \ kept, by ascending id
//   stack: free[n + r] = the r-th freed page
//   child b of i: row b = row i; if b > first_i and ctx_i % P != 0, its last page is one of its own,
//   taken(a) = free[n + R - 1 - a], a the number of such children before b, and is to be copied from row i's
//
// No reference counts are kept between calls: who holds a page stands in the tables.
//
// One launch.  A cluster of eight CTAs finds the freed pages in a set of bits that is spread over their
// shared memory (gone pages set, then kept pages cleared), counts them in the order of ids and hands out
// the copies' pages; more clusters, if the tables are large, copy the rows meanwhile.  Bound: latency, a chain
// of lengths and parents -> rows -> two or three cluster barriers -> stack -> last pages.
#include <cuda_runtime.h>

#include "cluster_bits.cuh"
#include "fastdiv.cuh"
#include "paged.h"
#include "ptx.cuh"

namespace atc_gb300 {
namespace {

constexpr int kMaxForkRequests = 8192;
constexpr int kForkThreads = 1024;

struct ForkParams {
    const int32_t* parents;
    int B;
    const int32_t* ctx;
    int Bo, page;
    FastDiv by_page;
    const int32_t* table;
    int max_pages;
    int32_t* free_pages;
    const int32_t* free_count;
    int num_pages;
    int32_t* new_table;
    int32_t* seqlens;
    int32_t* src;
    int32_t* dst;
    int32_t* tokens;
    int32_t* free_count_out;
    int* status;
    int words;   // of each CTA's part of the set
};

__global__ void __cluster_dims__(kClusterCtas, 1, 1) __launch_bounds__(kForkThreads, 1) page_fork_kernel(const __grid_constant__ ForkParams p)
{
    extern __shared__ int sh[];
    int* first = sh;                 // an old request's lowest child
    int* held_tokens = sh + p.Bo;    // and its tokens
    uint32_t* bits = reinterpret_cast<uint32_t*>(sh + 2 * p.Bo);
    __shared__ int sums[32], given[kClusterCtas];
    griddep_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, B = p.B, Bo = p.Bo, P = p.page;
    const int rank = static_cast<int>(cluster_ctarank()), cluster = blockIdx.x / kClusterCtas, clusters = gridDim.x / kClusterCtas;
    const bool counts = cluster == 0;   // this cluster finds the freed pages
    for (int i = tid; i < Bo; i += kForkThreads) first[i] = INT32_MAX;
    if (counts)
        for (int i = tid; i < p.words; i += kForkThreads) bits[i] = 0;
    griddep_wait();

    const long long room = static_cast<long long>(p.max_pages) * P;
    const int n = counts ? *p.free_count : 0;   // other clusters must not look: it may be updated in place
    bool bad = n < 0 || n > p.num_pages;
    for (int i = tid; i < Bo; i += kForkThreads) {
        const int c = p.ctx[i];
        held_tokens[i] = c;
        bad = bad || c < 0 || c > room;
    }
    __syncthreads();
    for (int b = tid; b < B; b += kForkThreads) {
        const int i = p.parents[b];
        bad = bad || i >= Bo;
        if (i >= 0 && i < Bo) atomicMin(&first[i], b);
    }
    bad = __syncthreads_or(bad);

    const auto held = [&](int i) { return p.by_page.up(held_tokens[i]); };
    const auto part = [&](int i) { return held_tokens[i] - p.by_page.div(held_tokens[i]) * P; };
    const auto copies = [&](int b, int i) { return i >= 0 && first[i] != b && part(i) != 0; };
    const auto fine = [&](int page) { return page >= 0 && page < p.num_pages; };
    const auto row = [&](int i) { return p.table + static_cast<size_t>(i) * p.max_pages; };
    const int warps = kForkThreads / 32, cluster_warp = rank * warps + (tid >> 5), cluster_warps = kClusterCtas * warps;

    // a warp per child: its row, up to a page that it gets for itself
    if (!bad && (clusters == 1 || !counts)) {
        const int step = clusters == 1 ? cluster_warps : (clusters - 1) * cluster_warps;
        for (int b = clusters == 1 ? cluster_warp : (cluster - 1) * cluster_warps + cluster_warp; b < B; b += step) {
            const int i = p.parents[b];
            if (i < 0) continue;
            const int k = held(i) - (copies(b, i) ? 1 : 0);
            const int32_t* from = row(i);
            int32_t* to = p.new_table + static_cast<size_t>(b) * p.max_pages;
            bool odd = false;
#pragma unroll 4
            for (int j = lane; j < k; j += 32) {
                const int x = from[j];
                odd = odd || !fine(x);
                to[j] = x;
            }
            if (odd) report_bad_page(p.status);
        }
    }
    if (!counts) return;

    // which pages go back
    const PageBits set{smem_u32(bits), p.words};
    int R = 0, before = 0, own = 0, at = 0;
    const int per = (p.words + kForkThreads - 1) / kForkThreads;
    const int w0 = min(p.words, tid * per), w1 = min(p.words, w0 + per);
    bool gone = false;
    if (!bad)
        for (int i = tid; i < Bo; i += kForkThreads) gone = gone || (first[i] == INT32_MAX && held_tokens[i] > 0);
    gone = __syncthreads_or(gone);
    if (gone) {
        cluster_sync();   // every CTA's words are zero
        bool odd = false;
        for (int i = cluster_warp; i < Bo; i += cluster_warps)
            if (first[i] == INT32_MAX)
#pragma unroll 4
                for (int j = lane; j < held(i); j += 32) {
                    const int x = row(i)[j];
                    if (fine(x))
                        set.set(x);
                    else
                        odd = true;
                }
        if (odd) report_bad_page(p.status);
        cluster_sync();
        for (int i = cluster_warp; i < Bo; i += cluster_warps)
            if (first[i] != INT32_MAX)
#pragma unroll 4
                for (int j = lane; j < held(i); j += 32) {
                    const int x = row(i)[j];
                    if (fine(x)) set.clear(x);
                }
        cluster_sync();
        for (int w = w0; w < w1; ++w) own += __popc(bits[w]);
        int total;
        at = block_scan(own, sums, total);
        if (tid < kClusterCtas) st_cluster(mapa_shared(smem_u32(&given[rank]), static_cast<uint32_t>(tid)), static_cast<uint32_t>(total));
        cluster_sync();
        for (int r = 0; r < kClusterCtas; ++r) {
            before += r < rank ? given[r] : 0;
            R += given[r];
        }
    }
    // children that get a page of their own, in a run per thread
    const int per_b = (B + kForkThreads - 1) / kForkThreads;
    const int b0 = min(B, tid * per_b), b1 = min(B, b0 + per_b);
    int mine = 0, A = 0;
    if (!bad)
        for (int b = b0; b < b1; ++b) mine += copies(b, p.parents[b]) ? 1 : 0;
    int a = block_scan(mine, sums, A);

    // all or nothing
    bad = bad || n + R > p.num_pages || A > n + R;
    if (bad) {
        cluster_sync();   // the stack's height has been read by all
        if (rank == 0) {
            for (int b = tid; b < B; b += kForkThreads) {
                p.seqlens[b] = 0;
                p.src[b] = p.dst[b] = -1;
                p.tokens[b] = 0;
            }
            if (tid == 0) {
                *p.free_count_out = n;
                report_bad_page(p.status);
            }
        }
        return;
    }
    if (R > 0) {
        int32_t* to = p.free_pages + n + before + at;
        for (int w = w0; w < w1; ++w)
            for (uint32_t v = bits[w]; v; v &= v - 1) *to++ = (rank * p.words + w) * 32 + __ffs(v) - 1;
    }
    cluster_sync();   // the stack is written, and its height read
    if (rank == 0 && tid == 0) *p.free_count_out = n + R - A;
    for (int b = b0; b < b1; ++b) {
        const int i = p.parents[b];
        const bool copy = copies(b, i);
        if (b % kClusterCtas == rank) {
            int from = -1, to = -1;
            if (copy) {
                const int last = held(i) - 1;
                from = row(i)[last];
                to = __ldcg(p.free_pages + (n + R - 1 - a));
                p.new_table[static_cast<size_t>(b) * p.max_pages + last] = to;
                if (!fine(from) || !fine(to)) report_bad_page(p.status);
            }
            p.seqlens[b] = i >= 0 ? held_tokens[i] : 0;
            p.src[b] = from;
            p.dst[b] = to;
            p.tokens[b] = copy ? part(i) : 0;
        }
        a += copy ? 1 : 0;
    }
}

}  // namespace
}  // namespace atc_gb300

using namespace atc_gb300;

extern "C" int fmha_page_fork(const int32_t* parents, int B, const int32_t* ctx_lens, int B_old, int page_size,
                              const int32_t* block_table, int max_pages, int32_t* free_pages, const int32_t* free_count,
                              int num_pages, int32_t* new_table, int32_t* seqlens, int32_t* copy_src, int32_t* copy_dst,
                              int32_t* copy_tokens, int32_t* free_count_out, fmha_stream_t stream)
{
    if (B < 0 || B_old < 0 || page_size < 1 || num_pages < 1 || max_pages < 1)
        return set_error(FMHA_ERR_INVALID, "fmha_page_fork: need B >= 0, B_old >= 0, page_size, num_pages and max_pages >= 1");
    if (!free_pages || !free_count || !free_count_out || (B_old > 0 && (!ctx_lens || !block_table)) ||
        (B > 0 && (!parents || !new_table || !seqlens || !copy_src || !copy_dst || !copy_tokens)))
        return set_error(FMHA_ERR_INVALID, "fmha_page_fork: NULL pointer");
    for (const void* x : {static_cast<const void*>(parents), static_cast<const void*>(ctx_lens), static_cast<const void*>(block_table),
                          static_cast<const void*>(free_pages), static_cast<const void*>(free_count), static_cast<const void*>(new_table),
                          static_cast<const void*>(seqlens), static_cast<const void*>(copy_src), static_cast<const void*>(copy_dst),
                          static_cast<const void*>(copy_tokens), static_cast<const void*>(free_count_out)})
        if (misaligned(x, 4)) return set_error(FMHA_ERR_INVALID, "fmha_page_fork: arrays must be 4-byte aligned");
    if (B > 0 && B_old > 0 && new_table == block_table)
        return set_error(FMHA_ERR_INVALID, "fmha_page_fork: new_table must not be block_table");
    if (B > kMaxForkRequests || B_old > kMaxForkRequests)
        return set_error(FMHA_ERR_UNSUPPORTED, "fmha_page_fork: more than 8192 requests");
    if (static_cast<long long>(max_pages) * page_size > (1LL << 31) - 256 || num_pages > kMaxPoolPages)
        return set_error(FMHA_ERR_UNSUPPORTED, "fmha_page_fork: max_pages * page_size past 2^31, or more than 2^20 pages");
    int* status = device_status_ptr();
    if (!status) return set_error(FMHA_ERR_CUDA, "no CUDA device");
    const int words = (num_pages + 32 * kClusterCtas - 1) / (32 * kClusterCtas);
    const ForkParams p{parents, B, ctx_lens, B_old, page_size, FastDiv(static_cast<uint32_t>(page_size)), block_table, max_pages,
                       free_pages, free_count, num_pages, new_table, seqlens, copy_src, copy_dst, copy_tokens, free_count_out, status, words};
    // clusters that copy rows: one for each 16384 entries that they may have
    const long long entries = static_cast<long long>(B) * max_pages;
    const int most = num_sms() / kClusterCtas - 1;
    const int copiers = entries <= 16384 ? 0 : static_cast<int>(entries / 16384 < most ? entries / 16384 : most);
    const int smem = 8 * B_old + 4 * words;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    FMHA_CHECK_CUDA(set_smem_limit_once(reinterpret_cast<const void*>(page_fork_kernel), 8 * kMaxForkRequests + kMaxPoolPages / 8 / kClusterCtas));
    FMHA_CHECK_CUDA(launch_pdl(page_fork_kernel, dim3(static_cast<unsigned>((1 + copiers) * kClusterCtas)), dim3(kForkThreads),
                               static_cast<size_t>(smem), st, p));
    count_launch();
    return FMHA_OK;
}
