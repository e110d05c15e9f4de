// Norms of the query and key heads, position rotation and the store of keys and values in the paged
// cache, in one pass over the projection's output (fmha_rope_append).
//
// For each token and head x of D features:  y = x / sqrt(mean(x^2) + eps) * w  (queries and keys; without
// weights y = x), then for the first R features the rotation of the pairs (y_i, y_j) by the angle of the
// token's position, y_i' = y_i c - y_j s, y_j' = y_j c + y_i s, with j = i + R / 2 or neighbouring pairs.
// Queries go to q_out, keys and values to the token's slot of the cache; values are copied.  Everything is
// FP32 from the BF16 inputs to the one rounding of each output.
//
// Bound: HBM (every element read once and written once; a decoding step is latency-bound).
#include <cuda_runtime.h>

#include "paged.h"
#include "ptx.cuh"

namespace atc_gb300 {
namespace {

constexpr int kDevBadPage = 7;

struct AppendParams {
    const uint16_t *q, *k, *v;
    int64_t q_stride, k_stride, v_stride;   // elements between tokens
    const uint16_t *wq, *wk;
    float eps;
    const float* cos_sin;                   // [max_pos][R]: R/2 cosines, R/2 sines
    int max_pos, R;
    const int32_t* positions;
    const int64_t* slots;
    uint16_t* q_out;
    uint16_t *kc, *vc;
    int64_t page_stride, head_stride, token_stride, num_slots;
    int page;
    int T, Hq, Hkv, Sq;
    int* status;
};

// Sixteen features of a head as two runs of eight: thread l of the D / 16 threads of a head holds the
// runs that it rotates against each other (l < R / 16), or two that pass.
struct Runs {
    int a, b;   // first feature of each run
};

template <bool PAIRS>
__device__ __forceinline__ Runs runs_of(int l, int R)
{
    if (PAIRS) return {16 * l, 16 * l + 8};
    const int m = R / 16;
    if (l < m) return {8 * l, 8 * (l + m)};
    return {16 * l, 16 * l + 8};
}

__device__ __forceinline__ void unpack8(const uint4& u, float* f)
{
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

__device__ __forceinline__ uint4 pack8(const float* f)
{
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}

template <int D, bool PAIRS>
__global__ void __launch_bounds__(256) rope_append_kernel(const __grid_constant__ AppendParams p)
{
    constexpr int L = D / 16;   // threads per head
    griddep_launch_dependents();
    griddep_wait();
    const int H = p.Hq + 2 * p.Hkv;
    const long long item = (static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) / L;
    const int l = threadIdx.x % L;
    const bool live = item < static_cast<long long>(p.T) * H;
    const int t = live ? static_cast<int>(item / H) : 0, h = live ? static_cast<int>(item % H) : 0;
    const long long slot = live ? p.slots[t] : -1;
    const int pos = live && p.R ? p.positions[t] : 0;
    bool store = slot >= 0;
    if (store && (slot >= p.num_slots || (p.R && (pos < 0 || pos >= p.max_pos)))) {
        store = false;
        atomicExch(p.status, kDevBadPage);
    }
    const bool is_q = h < p.Hq, is_v = h >= p.Hq + p.Hkv;
    const Runs r = is_v ? Runs{16 * l, 16 * l + 8} : runs_of<PAIRS>(l, p.R);
    uint4 ua = make_uint4(0, 0, 0, 0), ub = ua;
    if (store) {
        const uint16_t* x = is_q ? p.q + t * p.q_stride + static_cast<int64_t>(h) * D
                            : is_v ? p.v + t * p.v_stride + static_cast<int64_t>(h - p.Hq - p.Hkv) * D
                                   : p.k + t * p.k_stride + static_cast<int64_t>(h - p.Hq) * D;
        ua = *reinterpret_cast<const uint4*>(x + r.a);
        ub = *reinterpret_cast<const uint4*>(x + r.b);
    }
    if (!is_v) {
        float a[8], b[8];
        unpack8(ua, a);
        unpack8(ub, b);
        const uint16_t* w = is_q ? p.wq : p.wk;
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss += a[i] * a[i] + b[i] * b[i];
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if (w) {
            const float inv = rsqrtf(ss / D + p.eps);
            float wa[8], wb[8];
            unpack8(*reinterpret_cast<const uint4*>(w + r.a), wa);
            unpack8(*reinterpret_cast<const uint4*>(w + r.b), wb);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                a[i] = a[i] * inv * wa[i];
                b[i] = b[i] * inv * wb[i];
            }
        }
        if (store && l < p.R / 16) {
            // the thread's eight angles: features 8l .. 8l + 7 of either half, or its eight neighbouring pairs
            const float* cs = p.cos_sin + static_cast<int64_t>(pos) * p.R + 8 * l;
            float c[8], s[8];
#pragma unroll
            for (int i = 0; i < 8; i += 4) {
                *reinterpret_cast<float4*>(c + i) = *reinterpret_cast<const float4*>(cs + i);
                *reinterpret_cast<float4*>(s + i) = *reinterpret_cast<const float4*>(cs + p.R / 2 + i);
            }
            if (PAIRS) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float x0 = a[2 * i], x1 = a[2 * i + 1], z0 = b[2 * i], z1 = b[2 * i + 1];
                    a[2 * i] = x0 * c[i] - x1 * s[i];
                    a[2 * i + 1] = x1 * c[i] + x0 * s[i];
                    b[2 * i] = z0 * c[4 + i] - z1 * s[4 + i];
                    b[2 * i + 1] = z1 * c[4 + i] + z0 * s[4 + i];
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float x0 = a[i], x1 = b[i];
                    a[i] = x0 * c[i] - x1 * s[i];
                    b[i] = x1 * c[i] + x0 * s[i];
                }
            }
        }
        ua = pack8(a);
        ub = pack8(b);
    } else {
        // a warp may hold heads of both kinds: take part in the norm's shuffles
        float ss = 0.f;
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    }
    if (!store) return;
    uint16_t* y;
    if (is_q) {
        y = p.q_out + ((static_cast<int64_t>(t / p.Sq) * p.Hq + h) * p.Sq + t % p.Sq) * D;
    } else {
        const int head = is_v ? h - p.Hq - p.Hkv : h - p.Hq;
        const int64_t page = slot / p.page;
        y = (is_v ? p.vc : p.kc) + page * p.page_stride + head * p.head_stride + (slot - page * p.page) * p.token_stride;
    }
    *reinterpret_cast<uint4*>(y + r.a) = ua;
    *reinterpret_cast<uint4*>(y + r.b) = ub;
}

template <int D, bool PAIRS>
int run_append(const AppendParams& p, cudaStream_t st)
{
    const long long threads = static_cast<long long>(p.T) * (p.Hq + 2 * p.Hkv) * (D / 16);
    FMHA_CHECK_CUDA(launch_pdl(rope_append_kernel<D, PAIRS>, dim3(static_cast<unsigned>((threads + 255) / 256)), dim3(256), 0, st, p));
    count_launch();
    return FMHA_OK;
}

}  // namespace
}  // namespace atc_gb300

using namespace atc_gb300;

extern "C" int fmha_rope_append(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                                const void* q_weight, const void* k_weight, float eps, const float* cos_sin, int max_pos, int rope_dim,
                                int interleaved, const int32_t* positions, const int64_t* slots, void* q_out,
                                const fmha_kv_cache* cache, int T, int Hq, int Sq, fmha_stream_t stream)
{
    const int rc = check_cache(cache, "fmha_rope_append");
    if (rc) return rc;
    if (T != 0 && (!q || !k || !v || !slots || !q_out || (rope_dim != 0 && (!cos_sin || !positions))))
        return set_error(FMHA_ERR_INVALID, "fmha_rope_append: NULL q/k/v/slots/q_out, or cos_sin/positions with rope_dim > 0");
    if (T < 0 || Hq < 1 || Sq < 1 || T % Sq != 0 || Hq % cache->Hkv != 0)
        return set_error(FMHA_ERR_INVALID, "fmha_rope_append: need Hq a multiple of Hkv, Sq >= 1 and T >= 0 a multiple of Sq");
    if (rope_dim < 0 || rope_dim > cache->D || (rope_dim > 0 && max_pos < 1))
        return set_error(FMHA_ERR_INVALID, "fmha_rope_append: need 0 <= rope_dim <= D, and max_pos >= 1 with rope_dim > 0");
    if (rope_dim % 16 != 0) return set_error(FMHA_ERR_UNSUPPORTED, "fmha_rope_append: rope_dim must be a multiple of 16");
    if (!(eps >= 0.f) || !(eps < INFINITY)) return set_error(FMHA_ERR_INVALID, "fmha_rope_append: eps must be finite and not negative");
    if (misaligned(q, 16) || misaligned(k, 16) || misaligned(v, 16) || misaligned(q_weight, 16) || misaligned(k_weight, 16) ||
        misaligned(cos_sin, 16) || misaligned(q_out, 16) || misaligned(positions, 4) || misaligned(slots, 8))
        return set_error(FMHA_ERR_INVALID,
                         "fmha_rope_append: tensors 16-byte, positions 4-byte, slots 8-byte aligned");
    if (q_stride % 8 != 0 || k_stride % 8 != 0 || v_stride % 8 != 0 || q_stride < 0 || k_stride < 0 || v_stride < 0)
        return set_error(FMHA_ERR_INVALID, "fmha_rope_append: token strides must be non-negative multiples of 8 elements");
    if (static_cast<long long>(T) * (Hq + 2LL * cache->Hkv) >= (1LL << 31))
        return set_error(FMHA_ERR_UNSUPPORTED, "fmha_rope_append: more than 2^31 heads");
    int* status = device_status_ptr();
    if (!status) return set_error(FMHA_ERR_CUDA, "no CUDA device");
    if (T == 0) return FMHA_OK;
    AppendParams p{};
    p.q = static_cast<const uint16_t*>(q);
    p.k = static_cast<const uint16_t*>(k);
    p.v = static_cast<const uint16_t*>(v);
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.wq = static_cast<const uint16_t*>(q_weight);
    p.wk = static_cast<const uint16_t*>(k_weight);
    p.eps = eps;
    p.cos_sin = cos_sin;
    p.max_pos = max_pos;
    p.R = rope_dim;
    p.positions = positions;
    p.slots = slots;
    p.q_out = static_cast<uint16_t*>(q_out);
    p.kc = static_cast<uint16_t*>(cache->k);
    p.vc = static_cast<uint16_t*>(cache->v);
    p.page_stride = cache->page_stride;
    p.head_stride = cache->head_stride;
    p.token_stride = cache->token_stride;
    p.page = cache->page_size;
    p.num_slots = static_cast<int64_t>(cache->num_pages) * cache->page_size;
    p.T = T;
    p.Hq = Hq;
    p.Hkv = cache->Hkv;
    p.Sq = Sq;
    p.status = status;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (cache->D == 64) return interleaved ? run_append<64, true>(p, st) : run_append<64, false>(p, st);
    return interleaved ? run_append<128, true>(p, st) : run_append<128, false>(p, st);
}
