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
// One launch.  A CTA, or a cluster of eight for larger tables, marks gone and kept pages in sets of bits, counts the freed
// ones in the order of ids and hands out the copies' pages; more clusters, if the tables are large, copy the rows meanwhile.
// Bound: latency, a chain of lengths and parents -> rows -> sets -> stack -> last pages.  2 groups of 4 beams 5.7 us, one request
// into 64 samples 5.2, 128 groups of 4 with 16384 tokens each at most 9.1 (from a CUDA graph).
#include <cuda_runtime.h>

#include "cluster_bits.cuh"
#include "fastdiv.cuh"
#include "paged.h"
#include "ptx.cuh"

namespace atc_gb300 {
namespace {

constexpr int kMaxForkRequests = 8192;
constexpr int kForkThreads = 1024;

constexpr int kMaxForkPages = 1 << 19;   // two sets of 64 KB
constexpr int kForkCtas = 8;             // of a cluster
constexpr int kSegment = 256;            // entries of a row that a warp takes at a time, eight loads a lane

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
    int words;      // of a set
    int segments;   // runs of kSegment entries of a row
};

template <int CTAS>
__global__ void __cluster_dims__(CTAS, 1, 1) __launch_bounds__(kForkThreads, 1) page_fork_kernel(const __grid_constant__ ForkParams p)
{
    extern __shared__ int sh[];
    int* first = sh;                 // an old request's lowest child
    int* held_tokens = sh + p.Bo;    // and its tokens
    uint32_t* gone = reinterpret_cast<uint32_t*>(sh + 2 * p.Bo);
    uint32_t* kept = gone + p.words;
    __shared__ int sums[32], given[CTAS];
    griddep_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, B = p.B, Bo = p.Bo, P = p.page;
    const int rank = CTAS > 1 ? static_cast<int>(cluster_ctarank()) : 0, cluster = blockIdx.x / CTAS, clusters = gridDim.x / CTAS;
    const bool counts = cluster == 0;   // this cluster finds the freed pages
    for (int i = tid; i < Bo; i += kForkThreads) first[i] = INT32_MAX;
    if (counts)
        for (int i = tid; i < 2 * p.words; i += kForkThreads) gone[i] = 0;
    griddep_wait();

    const long long room = static_cast<long long>(p.max_pages) * P;
    const int n = counts ? *p.free_count : 0;   // other clusters must not look: it may be updated in place
    bool bad = n < 0 || n > p.num_pages;
    for (int i = tid; i < Bo; i += kForkThreads) {
        const int c = p.ctx[i];
        held_tokens[i] = c;
        bad = bad || c < 0 || c > room;
    }
    // children in a run per thread; the first of them, the usual number, stays in a register
    const int per_b = (B + kForkThreads - 1) / kForkThreads;
    const int b0 = min(B, tid * per_b), b1 = min(B, b0 + per_b);
    const int parent0 = b0 < b1 ? p.parents[b0] : -1;
    const auto parent = [&](int b) { return b == b0 ? parent0 : p.parents[b]; };
    __syncthreads();
    for (int b = b0; b < b1; ++b) {
        const int i = parent(b);
        bad = bad || i >= Bo;
        if (i >= 0 && i < Bo) atomicMin(&first[i], b);
    }
    bad = __syncthreads_or(bad);

    const auto held = [&](int i) { return p.by_page.up(held_tokens[i]); };
    const auto part = [&](int i) { return held_tokens[i] - p.by_page.div(held_tokens[i]) * P; };
    const auto copies = [&](int b, int i) { return i >= 0 && first[i] != b && part(i) != 0; };
    const auto fine = [&](int page) { return page >= 0 && page < p.num_pages; };
    const auto row = [&](int i) { return p.table + static_cast<size_t>(i) * p.max_pages; };
    const int warps = kForkThreads / 32, cluster_warp = rank * warps + (tid >> 5), cluster_warps = CTAS * warps;
    // The first count(i) entries of rows 0 .. n - 1 by `nw` warps, this one the w-th: a warp per row, or several where there are
    // more of them.  put(row, entry, page)
    const auto walk = [&](int n, int w, int nw, auto&& from, auto&& count, auto&& put) {
        const int shared = max(1, min(p.segments, nw / max(n, 1)));   // warps of a row
        for (int v = w; v < n * shared; v += nw) {
            const int i = v / shared, k = count(i);
            for (int s = v - i * shared; static_cast<long long>(s) * kSegment < k; s += shared) {
                const int32_t* row = from(i);
                int x[kSegment / 32];
#pragma unroll
                for (int u = 0; u < kSegment / 32; ++u) {
                    const int j = s * kSegment + u * 32 + lane;
                    x[u] = j < k ? row[j] : 0;
                }
#pragma unroll
                for (int u = 0; u < kSegment / 32; ++u) {
                    const int j = s * kSegment + u * 32 + lane;
                    if (j < k) put(i, j, x[u]);
                }
            }
        }
    };

    bool odd = false;
    // the children's rows, up to a page that a child gets for itself
    if (!bad && (clusters == 1 || !counts)) {
        const int others = clusters == 1 ? 1 : clusters - 1, me = clusters == 1 ? 0 : cluster - 1;
        walk(B, me * cluster_warps + cluster_warp, others * cluster_warps, [&](int b) { return row(p.parents[b]); },
             [&](int b) {
                 const int i = p.parents[b];
                 return i < 0 ? 0 : held(i) - (copies(b, i) ? 1 : 0);
             },
             [&](int b, int j, int x) {
                 odd = odd || !fine(x);
                 p.new_table[static_cast<size_t>(b) * p.max_pages + j] = x;
             });
    }
    if (!counts) {
        if (odd) report_bad_page(p.status);
        return;
    }

    // which pages go back
    int R = 0, before = 0, at = 0;
    const int slice = (p.words + CTAS - 1) / CTAS, per = (slice + kForkThreads - 1) / kForkThreads;   // words of a CTA and of a thread
    const int w1 = min(p.words, min((rank + 1) * slice, rank * slice + (tid + 1) * per)), w0 = min(w1, rank * slice + tid * per);
    bool ends = false;
    if (!bad)
        for (int i = tid; i < Bo; i += kForkThreads) ends = ends || (first[i] == INT32_MAX && held_tokens[i] > 0);
    ends = __syncthreads_or(ends);
    if (ends) {
        walk(Bo, cluster_warp, cluster_warps, row, held, [&](int i, int, int x) {
            const bool last = first[i] == INT32_MAX;
            if (fine(x))
                set_bit(last ? gone : kept, x);
            else
                odd = odd || last;
        });
        sync_ctas<CTAS>();
        int own = 0, total;
        for (int w = w0; w < w1; ++w) own += __popc(joined_word<CTAS>(gone, w) & ~joined_word<CTAS>(kept, w));
        at = block_scan(own, sums, total);
        if constexpr (CTAS > 1) {
            if (tid < CTAS) st_cluster(mapa_shared(smem_u32(&given[rank]), static_cast<uint32_t>(tid)), static_cast<uint32_t>(total));
        } else if (tid == 0) {
            given[0] = total;
        }
        sync_ctas<CTAS>();
        for (int r = 0; r < CTAS; ++r) {
            before += r < rank ? given[r] : 0;
            R += given[r];
        }
    }
    if (odd) report_bad_page(p.status);
    // children that get a page of their own
    int mine = 0, A = 0;
    if (!bad)
        for (int b = b0; b < b1; ++b) mine += copies(b, parent(b)) ? 1 : 0;
    int a = block_scan(mine, sums, A);

    // all or nothing
    bad = bad || n + R > p.num_pages || A > n + R;
    if (bad) {
        sync_ctas<CTAS>();   // the stack's height has been read by all, and nobody looks into another CTA's memory
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
            for (uint32_t v = joined_word<CTAS>(gone, w) & ~joined_word<CTAS>(kept, w); v; v &= v - 1) *to++ = w * 32 + __ffs(v) - 1;
    }
    sync_ctas<CTAS>();   // the stack is written, and its height read
    if (rank == 0 && tid == 0) *p.free_count_out = n + R - A;
    for (int b = b0; b < b1; ++b) {
        const int i = parent(b);
        const bool copy = copies(b, i);
        if (b % CTAS == rank) {
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
    if (static_cast<long long>(max_pages) * page_size > (1LL << 31) - 256 || num_pages > kMaxForkPages)
        return set_error(FMHA_ERR_UNSUPPORTED, "fmha_page_fork: max_pages * page_size past 2^31, or more than 2^19 pages");
    int* status = device_status_ptr();
    if (!status) return set_error(FMHA_ERR_CUDA, "no CUDA device");
    const int words = (num_pages + 31) / 32, segments = (max_pages + kSegment - 1) / kSegment;
    const ForkParams p{parents, B, ctx_lens, B_old, page_size, FastDiv(static_cast<uint32_t>(page_size)), block_table, max_pages,
                       free_pages, free_count, num_pages, new_table, seqlens, copy_src, copy_dst, copy_tokens, free_count_out, status, words, segments};
    // Runs of 256 entries that the tables may have: two a warp of one CTA, or else a cluster (its barriers cost a small call about 2
    // us); beyond two a warp of that, up to seven clusters more, to copy rows (with more than eight not all would be on the GPU at a time)
    const long long work = static_cast<long long>(B > B_old ? B : B_old) * segments;
    constexpr int kTwo = 2 * kForkThreads / 32;
    const bool one = work <= kTwo;
    const int most = 7, want = static_cast<int>(work / (kTwo * kForkCtas) < most ? work / (kTwo * kForkCtas) : most);
    const auto kernel = one ? page_fork_kernel<1> : page_fork_kernel<kForkCtas>;
    const int ctas = one ? 1 : (1 + want) * kForkCtas;
    const int smem = 8 * B_old + 8 * words;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    FMHA_CHECK_CUDA(set_smem_limit_once(reinterpret_cast<const void*>(kernel), 8 * kMaxForkRequests + kMaxForkPages / 4));
    FMHA_CHECK_CUDA(launch_pdl(kernel, dim3(static_cast<unsigned>(ctas)), dim3(kForkThreads), static_cast<size_t>(smem), st, p));
    count_launch();
    return FMHA_OK;
}
