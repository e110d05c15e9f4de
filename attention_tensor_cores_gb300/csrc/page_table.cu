// Page allocation, block tables and slot maps from request lengths (fmha_page_table).
//
// For each request b with ctx_b tokens in the cache and new_b to come (new_b < 0: finished), and pages of
// P tokens: held_b = ceil(ctx_b / P), need_b = ceil((ctx_b + new_b) / P) - held_b, and a finished request
// gives its held_b pages back.  With exclusive sums over the requests (in order) of the tokens (cu), the
// pages taken (aoff) and the pages given back (roff), everything else is a lookup:
//
//   free[n + r]               = the r-th page given back          (n: pages on the stack before)
//   table[b][held_b + j]      = taken(aoff_b + j), taken(a) = free[n + R - 1 - a]
//   token t, request b, position pos = ctx_b + t - cu_b:  slot = table[b][pos / P] * P + pos % P
//
// taken(a) that falls on a page given back in this call is found through roff and the finished request's
// table row, not through the stack, so no thread reads what another one writes.  The lengths and the
// stack height may be updated in place: every CTA keeps them in shared memory before any is written.
//
// Bound: launch latency and a chain of dependent loads (lengths, table or stack entry) for a decoding
// step; 12 bytes written per token for prompts.
#include <cuda_runtime.h>

#include "paged.h"
#include "ptx.cuh"

namespace atc_gb300 {
namespace {

constexpr int kMaxRequests = 8192;   // 16 bytes of shared memory each
constexpr int kDevBadPage = 7;

struct PageTableParams {
    const int32_t* ctx;
    const int32_t* add;
    int B, page, num_pages;
    int32_t* free_pages;
    const int32_t* free_count;
    int32_t* table;
    int max_pages;
    int32_t* seqlens;
    int32_t* cu;
    int32_t* positions;
    int64_t* slots;
    int T;
    int32_t* free_count_out;
    int* status;
};

// last b with start[b] <= x (start non-decreasing, start[0] = 0): the request that item x belongs to
__device__ __forceinline__ int owner(const int* start, int B, int x)
{
    int lo = 0, hi = B - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (start[mid] <= x) lo = mid; else hi = mid - 1;
    }
    return lo;
}

struct Sums {
    long long add, need, back;
};

__global__ void __launch_bounds__(1024) page_table_kernel(const __grid_constant__ PageTableParams p)
{
    extern __shared__ int sh[];
    int* s_ctx = sh;                 // tokens held
    int* s_cu = sh + p.B;            // first new token
    int* s_aoff = sh + 2 * p.B;      // first page taken
    int* s_roff = sh + 3 * p.B;      // first page given back
    __shared__ Sums warp_sums[32], total;
    __shared__ int s_n;
    griddep_launch_dependents();
    griddep_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = blockDim.x >> 5;
    const int P = p.page, B = p.B;

    // each thread sums a run of requests; then a scan over the threads
    const int per = (B + blockDim.x - 1) / blockDim.x;
    const int b0 = min(B, tid * per), b1 = min(B, b0 + per);
    bool bad = false;
    Sums own{0, 0, 0};
    for (int b = b0; b < b1; ++b) {
        const int c = p.ctx[b], a = p.add[b];
        const long long held = (static_cast<long long>(c) + P - 1) / P;
        if (c < 0 || held > p.max_pages) bad = true;
        if (a < 0) {
            own.back += held;
        } else {
            const long long after = (static_cast<long long>(c) + a + P - 1) / P;
            if (after > p.max_pages) bad = true;
            own.add += a;
            own.need += after - held;
        }
    }
    if (tid == 0) s_n = *p.free_count;
    Sums inc = own;
    for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, inc.add, o), y = __shfl_up_sync(0xffffffffu, inc.need, o),
                        z = __shfl_up_sync(0xffffffffu, inc.back, o);
        if (lane >= o) {
            inc.add += x;
            inc.need += y;
            inc.back += z;
        }
    }
    if (lane == 31) warp_sums[warp] = inc;
    bad = __syncthreads_or(bad);
    if (tid == 0) {
        Sums run{0, 0, 0};
        for (int w = 0; w < nw; ++w) {
            const Sums v = warp_sums[w];
            warp_sums[w] = run;
            run.add += v.add;
            run.need += v.need;
            run.back += v.back;
        }
        total = run;
    }
    __syncthreads();
    const Sums tot = total;
    const int n = s_n;
    // all or nothing: without room for every request, or with a length that cannot be, nothing changes
    bad = bad || n < 0 || n + tot.back > p.num_pages || tot.need > n + tot.back || tot.add > p.T;
    if (!bad) {
        Sums at = warp_sums[warp];
        at.add += inc.add - own.add;
        at.need += inc.need - own.need;
        at.back += inc.back - own.back;
        for (int b = b0; b < b1; ++b) {
            const int c = p.ctx[b], a = p.add[b];
            const int held = static_cast<int>((static_cast<long long>(c) + P - 1) / P);
            s_ctx[b] = c;
            s_cu[b] = static_cast<int>(at.add);
            s_aoff[b] = static_cast<int>(at.need);
            s_roff[b] = static_cast<int>(at.back);
            if (a < 0) {
                at.back += held;
            } else {
                at.add += a;
                at.need += static_cast<int>((static_cast<long long>(c) + a + P - 1) / P) - held;
            }
        }
    } else {
        for (int b = b0; b < b1; ++b) s_ctx[b] = p.ctx[b];
    }
    // every CTA has read the lengths and the stack height: from here on they may be overwritten
    cluster_sync();

    const int first = blockIdx.x * blockDim.x + tid, step = gridDim.x * blockDim.x;
    if (bad) {
        for (int b = first; b <= B; b += step) {
            p.cu[b] = 0;
            if (b < B) p.seqlens[b] = s_ctx[b];
        }
        for (int t = first; t < p.T; t += step) {
            p.positions[t] = 0;
            p.slots[t] = -1;
        }
        if (first == 0) {
            *p.free_count_out = n;
            atomicExch(p.status, kDevBadPage);
        }
        return;
    }
    const int taken_n = static_cast<int>(tot.need), given_n = static_cast<int>(tot.back), tokens = static_cast<int>(tot.add);
    auto given = [&](int r) {
        const int b = owner(s_roff, B, r);
        return p.table[static_cast<size_t>(b) * p.max_pages + (r - s_roff[b])];
    };
    auto taken = [&](int a) {
        const int i = n + given_n - 1 - a;
        return i < n ? p.free_pages[i] : given(i - n);
    };
    auto held_of = [&](int b) { return static_cast<int>((static_cast<unsigned>(s_ctx[b]) + P - 1) / P); };
    for (int b = first; b <= B; b += step) {
        p.cu[b] = b < B ? s_cu[b] : tokens;
        if (b < B) {
            const bool done = (b + 1 < B ? s_roff[b + 1] : given_n) > s_roff[b];
            p.seqlens[b] = done ? 0 : s_ctx[b] + ((b + 1 < B ? s_cu[b + 1] : tokens) - s_cu[b]);
        }
    }
    for (int r = first; r < given_n; r += step) {
        const int page = given(r);
        p.free_pages[n + r] = page;
        if (page < 0 || page >= p.num_pages) atomicExch(p.status, kDevBadPage);
    }
    for (int a = first; a < taken_n; a += step) {
        const int b = owner(s_aoff, B, a);
        p.table[static_cast<size_t>(b) * p.max_pages + held_of(b) + (a - s_aoff[b])] = taken(a);
    }
    if (first == 0) *p.free_count_out = n + given_n - taken_n;
    for (int t = first; t < p.T; t += step) {
        int pos = 0;
        long long slot = -1;
        if (t < tokens) {
            const int b = owner(s_cu, B, t);
            pos = s_ctx[b] + (t - s_cu[b]);
            const int i = pos / P, held = held_of(b);
            const int page = i < held ? p.table[static_cast<size_t>(b) * p.max_pages + i] : taken(s_aoff[b] + i - held);
            if (page >= 0 && page < p.num_pages)
                slot = static_cast<long long>(page) * P + (pos - i * P);
            else
                atomicExch(p.status, kDevBadPage);
        }
        p.positions[t] = pos;
        p.slots[t] = slot;
    }
}

}  // namespace
}  // namespace atc_gb300

using namespace atc_gb300;

extern "C" int fmha_page_table(const int32_t* ctx_lens, const int32_t* new_lens, int B, int page_size, int32_t* free_pages,
                               const int32_t* free_count, int num_pages, int32_t* block_table, int max_pages, int32_t* seqlens,
                               int32_t* cu_new, int32_t* positions, int64_t* slots, int T, int32_t* free_count_out,
                               fmha_stream_t stream)
{
    if (B < 0 || T < 0 || page_size < 1 || num_pages < 1 || max_pages < 1)
        return set_error(FMHA_ERR_INVALID, "fmha_page_table: need B >= 0, T >= 0, page_size, num_pages and max_pages >= 1");
    if (!free_pages || !free_count || !free_count_out || !cu_new || (B > 0 && (!ctx_lens || !new_lens || !block_table || !seqlens)) ||
        (T > 0 && (!positions || !slots)))
        return set_error(FMHA_ERR_INVALID, "fmha_page_table: NULL pointer");
    if (misaligned(ctx_lens, 4) || misaligned(new_lens, 4) || misaligned(free_pages, 4) || misaligned(free_count, 4) ||
        misaligned(block_table, 4) || misaligned(seqlens, 4) || misaligned(cu_new, 4) || misaligned(positions, 4) ||
        misaligned(slots, 8) || misaligned(free_count_out, 4))
        return set_error(FMHA_ERR_INVALID, "fmha_page_table: slots 8-byte, the other arrays 4-byte aligned");
    if (B > kMaxRequests) return set_error(FMHA_ERR_UNSUPPORTED, "fmha_page_table: more than 8192 requests");
    if (static_cast<long long>(max_pages) * page_size > (1LL << 31) - 256 || T > (1 << 30) || num_pages > (1 << 30))
        return set_error(FMHA_ERR_UNSUPPORTED, "fmha_page_table: max_pages * page_size past 2^31, or T or num_pages past 2^30");
    int* status = device_status_ptr();
    if (!status) return set_error(FMHA_ERR_CUDA, "no CUDA device");
    const PageTableParams p{ctx_lens, new_lens, B,         page_size, num_pages, free_pages, free_count,     block_table,
                            max_pages, seqlens, cu_new,    positions, slots,     T,          free_count_out, status};
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const int smem = B * 16;
    FMHA_CHECK_CUDA(set_smem_limit_once(reinterpret_cast<const void*>(page_table_kernel), kMaxRequests * 16));
    FMHA_CHECK_CUDA(launch_pdl(page_table_kernel, dim3(1), dim3(1024), static_cast<size_t>(smem), st, p));
    count_launch();
    return FMHA_OK;
}
