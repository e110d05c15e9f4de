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
// table row, not through the stack, so no thread reads what another one writes, except that the lengths
// and the stack height may be updated in place: a CTA has them in shared memory before it writes them, and
// a launch of several CTAs leaves them to a second launch when they are.
//
// Bound: launch latency and a chain of dependent loads (lengths, table or stack entry) for a decoding
// step; 12 bytes written per token for prompts.  GPU time (without requests 1.8 us): 8 requests of a token 2.9 us,
// 256 requests of which 32 end 4.6 (one CTA 7.2), 32 prompts of 131,000 tokens 4.4 (one CTA 120, a cluster of
// eight 19).  An update in place is slower, as its CTAs may not write what others still read (separate arrays / in
// place, pages of 16, a token each): 8 requests 3.1 / 3.4, 256 (pages of 64, 77 of padding) 3.7 / 4.2, 1024
// 4.7 / 5.6, 2049 6.7 / 10.9; 32 prompts of 4000 tokens 4.0 / 6.9.
#include <cuda_runtime.h>

#include "fastdiv.cuh"
#include "paged.h"
#include "ptx.cuh"

namespace atc_gb300 {
namespace {

constexpr int kMaxRequests = 8192;   // 16 bytes of shared memory each

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
    FastDiv by_page;
    int top;      // the largest power of two below B
    int parts;    // kTables, kLengths or both
};

// What a launch writes: the tables and slots, or what may be updated in place (lengths and stack height).
enum : int { kTables = 1, kLengths = 2 };

// last b with start[b] <= x (start non-decreasing, start[0] = 0): the request that item x belongs to.  top: the
// largest power of two below B (0 for B = 1).
__device__ __forceinline__ int owner(const int* start, int B, int top, int x)
{
    int b = 0;
    for (int s = top; s > 0; s >>= 1)
        if (b + s < B && start[b + s] <= x) b += s;
    return b;
}

struct Sums {   // new tokens, pages taken, pages given back
    long long add, need, back;

    __device__ __forceinline__ Sums operator+(const Sums& o) const { return {add + o.add, need + o.need, back + o.back}; }
    __device__ __forceinline__ Sums operator-(const Sums& o) const { return {add - o.add, need - o.need, back - o.back}; }
};

// inclusive sums over the lanes of a warp
__device__ __forceinline__ Sums warp_scan(Sums v, int lane)
{
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Sums u{__shfl_up_sync(0xffffffffu, v.add, o), __shfl_up_sync(0xffffffffu, v.need, o), __shfl_up_sync(0xffffffffu, v.back, o)};
        if (lane >= o) v = v + u;
    }
    return v;
}

// What request b asks for; sets `bad` for lengths that cannot be.
__device__ __forceinline__ Sums request(const PageTableParams& p, int c, int a, bool& bad)
{
    Sums r{0, 0, 0};
    const long long room = static_cast<long long>(p.max_pages) * p.page;   // below 2^31
    if (c < 0 || c > room || (a > 0 && static_cast<long long>(c) + a > room)) {
        bad = true;
        return r;
    }
    const int held = p.by_page.up(c);
    if (a < 0) {
        r.back = held;
    } else {
        r.add = a;
        r.need = p.by_page.up(c + a) - held;
    }
    return r;
}

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
        const int c = p.ctx[b];
        s_ctx[b] = c;
        own = own + request(p, c, p.add[b], bad);
    }
    if (tid == 0) s_n = *p.free_count;
    const Sums inc = warp_scan(own, lane);
    if (lane == 31) warp_sums[warp] = inc;
    bad = __syncthreads_or(bad);
    if (warp == 0) {
        const Sums mine = lane < nw ? warp_sums[lane] : Sums{0, 0, 0};
        const Sums all = warp_scan(mine, lane);
        __syncwarp();
        if (lane < nw) warp_sums[lane] = all - mine;
        if (lane == 31) total = all;
    }
    __syncthreads();
    const Sums tot = total;
    const int n = s_n;
    // all or nothing: without room for every request, or with a length that cannot be, nothing changes
    bad = bad || n < 0 || n + tot.back > p.num_pages || tot.need > n + tot.back || tot.add > p.T;
    if (!bad) {
        Sums at = warp_sums[warp] + inc - own;
        for (int b = b0; b < b1; ++b) {
            s_cu[b] = static_cast<int>(at.add);
            s_aoff[b] = static_cast<int>(at.need);
            s_roff[b] = static_cast<int>(at.back);
            if (b + 1 < b1) at = at + request(p, s_ctx[b], p.add[b], bad);
        }
    }
    // the lengths and the stack height have been read: from here on they may be overwritten
    __syncthreads();

    const int first = blockIdx.x * blockDim.x + tid, step = gridDim.x * blockDim.x;
    if (bad) {
        if (p.parts & kTables) {
            for (int b = first; b <= B; b += step) p.cu[b] = 0;
            for (int t = first; t < p.T; t += step) {
                p.positions[t] = 0;
                p.slots[t] = -1;
            }
            if (first == 0) report_bad_page(p.status);
        }
        if (p.parts & kLengths) {
            for (int b = first; b < B; b += step) p.seqlens[b] = s_ctx[b];
            if (first == 0) *p.free_count_out = n;
        }
        return;
    }
    const int taken_n = static_cast<int>(tot.need), given_n = static_cast<int>(tot.back), tokens = static_cast<int>(tot.add);
    const auto row = [&](int b) { return p.table + static_cast<size_t>(b) * p.max_pages; };
    // where the r-th page given back, and the page of taken(a), are to be read
    const auto given = [&](int r) {
        const int b = owner(s_roff, B, p.top, r);
        return row(b) + (r - s_roff[b]);
    };
    const auto taken = [&](int a) {
        const int i = n + given_n - 1 - a;
        return i < n ? p.free_pages + i : given(i - n);
    };
    const auto fine = [&](int page) { return page >= 0 && page < p.num_pages; };

    if (p.parts & kTables) {
        // a token, a page taken and a page given back at a time: first all three are looked up, then written
        const int most = max(max(p.T, taken_n), given_n);
        for (int x = first; x < most; x += step) {
            int pos = 0, page = 0, to = 0, new_page = 0, old_page = 0;
            if (x < tokens) {
                const int b = owner(s_cu, B, p.top, x);
                pos = s_ctx[b] + (x - s_cu[b]);
                const int i = p.by_page.div(pos), held = p.by_page.up(s_ctx[b]);
                page = *(i < held ? row(b) + i : taken(s_aoff[b] + i - held));
            }
            if (x < taken_n) {
                to = owner(s_aoff, B, p.top, x);
                new_page = *taken(x);
            }
            if (x < given_n) old_page = *given(x);
            if (x < p.T) {
                const bool ok = x < tokens && fine(page);
                if (x < tokens && !ok) report_bad_page(p.status);
                p.positions[x] = pos;
                p.slots[x] = ok ? static_cast<long long>(page) * P + (pos - p.by_page.div(pos) * P) : -1;
            }
            if (x < taken_n) row(to)[p.by_page.up(s_ctx[to]) + (x - s_aoff[to])] = new_page;
            if (x < given_n) {
                p.free_pages[n + x] = old_page;
                if (!fine(old_page)) report_bad_page(p.status);
            }
        }
        for (int b = first; b <= B; b += step) p.cu[b] = b < B ? s_cu[b] : tokens;
    }
    if (p.parts & kLengths) {
        for (int b = first; b < B; b += step) {
            const bool done = (b + 1 < B ? s_roff[b + 1] : given_n) > s_roff[b];
            p.seqlens[b] = done ? 0 : s_ctx[b] + ((b + 1 < B ? s_cu[b + 1] : tokens) - s_cu[b]);
        }
        if (first == 0) *p.free_count_out = n + given_n - taken_n;
    }
}

int launch_table(PageTableParams& p, int parts, int ctas, int threads, cudaStream_t st)
{
    p.parts = parts;
    FMHA_CHECK_CUDA(set_smem_limit_once(reinterpret_cast<const void*>(page_table_kernel), kMaxRequests * 16));
    FMHA_CHECK_CUDA(launch_pdl(page_table_kernel, dim3(static_cast<unsigned>(ctas)), dim3(static_cast<unsigned>(threads)),
                               static_cast<size_t>(p.B) * 16, st, p));
    count_launch();
    return FMHA_OK;
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
    PageTableParams p{ctx_lens, new_lens, B, page_size, num_pages, free_pages, free_count, block_table, max_pages, seqlens, cu_new,
                      positions, slots, T, free_count_out, status, FastDiv(static_cast<uint32_t>(page_size)), 0, 0};
    while ((p.top ? 2 * p.top : 1) < B) p.top = p.top ? 2 * p.top : 1;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    // An item per thread: the tokens, or, as requests that end give back many pages, 32 per request (8: 32
    // requests 5.0 us against 4.1, 256 5.4 / 4.8).  Every CTA sums the lengths, so many requests take larger and
    // fewer ones (1024 requests with 256, 512, 1024 threads 6.5, 6.2, 7.1; 4096 45, 13.4, 9.8).  An update in
    // place has one CTA, or beyond 2048 tokens or requests a launch of its own after the others have read.
    // (Four items per thread, their loads in flight together: 131,000 tokens 5.9 against 4.6.)
    const bool in_place = seqlens == ctx_lens || free_count_out == free_count;
    const int most = T > B ? T : B;
    if (in_place && most <= 2048) return launch_table(p, kTables | kLengths, 1, most <= 256 ? 256 : 1024, st);
    const int threads = B > 2048 ? 1024 : B > 512 ? 512 : 256, items = T > 32 * B ? T : 32 * B, want = (items + threads - 1) / threads;
    const int limit = 1024 / threads * num_sms();
    const int rc = launch_table(p, in_place ? kTables : kTables | kLengths, want < 1 ? 1 : want < limit ? want : limit, threads, st);
    return rc || !in_place ? rc : launch_table(p, kLengths, 1, 1024, st);
}
