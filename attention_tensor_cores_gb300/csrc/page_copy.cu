// Copies of pages inside the pools of a model's layers (fmha_page_copy): the first tokens[i] tokens of page
// src[i], all heads, K and V, to page dst[i] of the same pool.
//
// Bound: HBM, every byte read and written once, or the launch: 1501 whole pages of 3 MB 1370 us, 6.9 TB/s; 64 partly filled ones
// 10.0 us, 5.0 TB/s.  A block takes up to kRows rows (a head's
// features of a token) of one pool of one pair, eight 16-byte loads in flight a thread; rows go in the order in
// which they lie in memory, tokens of a head or heads of a token innermost, whichever has the smaller stride.
#include <cuda_runtime.h>

#include "paged.h"
#include "ptx.cuh"

namespace atc_gb300 {
namespace {

constexpr int kCopyThreads = 256;
constexpr int kCopyLoads = 8;        // 16-byte loads in flight a thread
constexpr int kMaxCopyCaches = 128;  // of a launch: their pointers are kernel parameters

struct CopyParams {
    const int32_t* src;
    const int32_t* dst;
    const int32_t* tokens;
    const int32_t* count;
    int n, num_pages, page, Hkv, D;
    int64_t page_stride, head_stride, token_stride;
    int heads_inside;   // the heads of a token are innermost
    int* status;
    void* pool[2 * kMaxCopyCaches];   // K and V of each cache
};

template <int D>
__global__ void __launch_bounds__(kCopyThreads) page_copy_kernel(const __grid_constant__ CopyParams p)
{
    constexpr int kLanes = D / 8;   // threads of a row
    constexpr int kRows = kCopyThreads / kLanes * kCopyLoads;
    griddep_launch_dependents();
    griddep_wait();
    const int i = blockIdx.x;
    const bool report = blockIdx.y == 0 && blockIdx.z == 0 && threadIdx.x == 0;
    const int from = p.src[i], to = p.dst[i], wanted = p.tokens ? p.tokens[i] : p.page, c = p.count ? *p.count : p.n;
    if (report && i == 0 && (c < 0 || c > p.n)) report_bad_page(p.status);
    if (i >= c) return;
    if (from < 0 || to < 0) return;
    const int t = min(max(wanted, 0), p.page);
    const bool fine = from < p.num_pages && to < p.num_pages;
    if (report && (!fine || t != wanted)) report_bad_page(p.status);
    if (!fine) return;
    const int rows = t * p.Hkv, inner = p.heads_inside ? p.Hkv : t, r0 = blockIdx.z * kRows;
    if (r0 >= rows) return;
    const int64_t inner_stride = p.heads_inside ? p.head_stride : p.token_stride, outer_stride = p.heads_inside ? p.token_stride : p.head_stride;
    uint16_t* pool = static_cast<uint16_t*>(p.pool[blockIdx.y]);
    const uint16_t* a = pool + from * p.page_stride;
    uint16_t* b = pool + to * p.page_stride;
    const int lane = threadIdx.x % kLanes, first = r0 + threadIdx.x / kLanes;
    uint4 v[kCopyLoads];
    int64_t at[kCopyLoads];
#pragma unroll
    for (int k = 0; k < kCopyLoads; ++k) {
        const int r = first + k * (kCopyThreads / kLanes), o = static_cast<int>(static_cast<unsigned>(r) / static_cast<unsigned>(inner));
        at[k] = o * outer_stride + (r - o * inner) * inner_stride + lane * 8;
        if (r < rows) v[k] = __ldcs(reinterpret_cast<const uint4*>(a + at[k]));
    }
#pragma unroll
    for (int k = 0; k < kCopyLoads; ++k)
        if (first + k * (kCopyThreads / kLanes) < rows) __stcs(reinterpret_cast<uint4*>(b + at[k]), v[k]);
}

}  // namespace
}  // namespace atc_gb300

using namespace atc_gb300;

extern "C" int fmha_page_copy(const fmha_kv_cache* caches, int n_caches, const int32_t* src, const int32_t* dst, const int32_t* tokens, int n,
                              const int32_t* count, fmha_stream_t stream)
{
    if (n_caches < 0 || n < 0 || (n_caches > 0 && !caches)) return set_error(FMHA_ERR_INVALID, "fmha_page_copy: need n_caches >= 0, n >= 0 and caches");
    for (int i = 0; i < n_caches; ++i) {
        const int rc = check_cache(caches + i, "fmha_page_copy");
        if (rc) return rc;
        const fmha_kv_cache &a = caches[0], &b = caches[i];
        if (a.num_pages != b.num_pages || a.page_size != b.page_size || a.Hkv != b.Hkv || a.D != b.D || a.page_stride != b.page_stride ||
            a.head_stride != b.head_stride || a.token_stride != b.token_stride)
            return set_error(FMHA_ERR_INVALID, "fmha_page_copy: the caches must have the same sizes and strides");
    }
    if (n > 0 && (!src || !dst)) return set_error(FMHA_ERR_INVALID, "fmha_page_copy: NULL src/dst");
    if (misaligned(src, 4) || misaligned(dst, 4) || misaligned(tokens, 4) || misaligned(count, 4))
        return set_error(FMHA_ERR_INVALID, "fmha_page_copy: arrays must be 4-byte aligned");
    if (n_caches == 0 || n == 0) return FMHA_OK;
    const fmha_kv_cache& c = caches[0];
    if (static_cast<long long>(c.page_size) * c.Hkv >= (1LL << 22))
        return set_error(FMHA_ERR_UNSUPPORTED, "fmha_page_copy: pages of 2^22 rows or more");
    CopyParams p{};
    p.src = src;
    p.dst = dst;
    p.tokens = tokens;
    p.count = count;
    p.n = n;
    p.num_pages = c.num_pages;
    p.page = c.page_size;
    p.Hkv = c.Hkv;
    p.D = c.D;
    p.page_stride = c.page_stride;
    p.head_stride = c.head_stride;
    p.token_stride = c.token_stride;
    p.heads_inside = c.head_stride < c.token_stride;
    p.status = device_status_ptr();
    if (!p.status) return set_error(FMHA_ERR_CUDA, "no CUDA device");
    const auto kernel = c.D == 64 ? page_copy_kernel<64> : page_copy_kernel<128>;
    const int rows = c.page_size * c.Hkv, per = kCopyThreads / (c.D / 8) * kCopyLoads;
    for (int first = 0; first < n_caches; first += kMaxCopyCaches) {
        const int m = n_caches - first < kMaxCopyCaches ? n_caches - first : kMaxCopyCaches;
        for (int i = 0; i < m; ++i) {
            p.pool[2 * i] = caches[first + i].k;
            p.pool[2 * i + 1] = caches[first + i].v;
        }
        FMHA_CHECK_CUDA(launch_pdl(kernel, dim3(static_cast<unsigned>(n), static_cast<unsigned>(2 * m), static_cast<unsigned>((rows + per - 1) / per)),
                                   dim3(kCopyThreads), 0, reinterpret_cast<cudaStream_t>(stream), p));
        count_launch();
    }
    return FMHA_OK;
}
