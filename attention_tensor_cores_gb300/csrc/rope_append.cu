// Norms of the query and key heads, position rotation and the store of keys and values in the paged
// cache, in one pass over the projection's output (fmha_rope_append).
//
// For each token and head x of D features:  y = x / sqrt(mean(x^2) + eps) * w  (queries and keys; without
// weights y = x), then for the first R features the rotation of the pairs (y_i, y_j) by the angle of the
// token's position, y_i' = y_i c - y_j s, y_j' = y_j c + y_i s, with j = i + R / 2 or neighbouring pairs.
// Queries go to q_out, keys and values to the token's slot of the cache; values are copied.  Everything is
// FP32 from the BF16 inputs to the one rounding of each output.
//
// Bound: HBM (every element read once and written once; a decoding step is latency-bound).  A CTA's life is
// two dependent DRAM accesses (slot and position, then angles; the heads beside them) and little arithmetic, so
// occupancy and loads in flight set the rate.  8192 tokens, 32 + 8 + 8 heads of 128, norm and rotation: 34.8 to
// 35.4 us, 5.8 TB/s = 0.85 to 0.87 of the copy bandwidth.  On the way there: one head per group of threads 55.7 us; four heads in
// flight 48; the weights drawn into the angles, packed FP32 and five CTAs per SM 38.3 (four 41.5, six with
// spills 43); the next heads fetched into L2 34.8.  8 tokens: 2.2 us of GPU time.
#include <cuda_runtime.h>

#include "fastdiv.cuh"
#include "paged.h"
#include "ptx.cuh"

namespace atc_gb300 {
namespace {

constexpr int kThreads = 128, kCtas = 5;   // per CTA, and CTAs per SM that the registers allow

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
    int q_sets, kv_sets;               // sets of heads of a token, of queries and of keys (or values)
    int ahead;                         // tokens between one and the one whose heads are fetched into L2 with it
    FastDiv by_sets, by_page, by_sq;   // all of a token's sets, page and Sq
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

__device__ __forceinline__ uint64_t fmul2(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// Eight BF16 as four pairs of FP32, and back
__device__ __forceinline__ void unpack8(const uint4& u, uint64_t (&f)[4])
{
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = f32x2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}

__device__ __forceinline__ uint4 pack8(const uint64_t (&f)[4])
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float lo, hi;
        f32x2_split(f[i], lo, hi);
        w[i] = pack_bf16x2(lo, hi);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ uint64_t swap2(uint64_t v)
{
    float lo, hi;
    f32x2_split(v, lo, hi);
    return f32x2(hi, lo);
}

// A group of D / 16 threads takes up to HEADS consecutive heads of one kind (queries, keys or values) of a
// token: their loads are in flight together, and the token's slot, position and angles are read once for
// them.  With the weights drawn into the angles, w the head's and c, s the angle's cosine and sine, a pair is
//   y_i = (x_i (w_i c) + x_j (-w_j s)) / rms     y_j = (x_j (w_j c) + x_i (w_i s)) / rms
// three packed operations for two outputs.
template <int D, bool PAIRS, int HEADS>
__global__ void __launch_bounds__(kThreads, kCtas) rope_append_kernel(const __grid_constant__ AppendParams p)
{
    constexpr int L = D / 16;   // threads per head
    griddep_launch_dependents();
    griddep_wait();
    const int item = static_cast<int>((static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) / L);   // below 2^31
    const int l = threadIdx.x % L;
    const uint32_t group = ((1u << L) - 1u) << (threadIdx.x & 31 & ~(L - 1));   // the lanes of this head
    const int t = p.by_sets.div(item), set = item - t * static_cast<int>(p.by_sets.d);
    if (t >= p.T) return;
    const int64_t slot = p.slots[t];
    const int pos = p.R ? p.positions[t] : 0;
    const int kind = set < p.q_sets ? 0 : set < p.q_sets + p.kv_sets ? 1 : 2;
    const int h0 = (kind == 0 ? set : kind == 1 ? set - p.q_sets : set - p.q_sets - p.kv_sets) * HEADS;
    const int heads = min(HEADS, (kind == 0 ? p.Hq : p.Hkv) - h0);
    const Runs r = kind == 2 ? Runs{16 * l, 16 * l + 8} : runs_of<PAIRS>(l, p.R);

    const int64_t stride = kind == 0 ? p.q_stride : kind == 1 ? p.k_stride : p.v_stride;
    const uint16_t* x = (kind == 0 ? p.q : kind == 1 ? p.k : p.v) + t * stride + static_cast<int64_t>(h0) * D;
    uint4 u[HEADS][2];
#pragma unroll
    for (int k = 0; k < HEADS; ++k)
        if (k < heads) {
            u[k][0] = *reinterpret_cast<const uint4*>(x + k * D + r.a);
            u[k][1] = *reinterpret_cast<const uint4*>(x + k * D + r.b);
        }
    // the same heads of a token that a later CTA takes: into L2 meanwhile, a line per thread
    if (HEADS > 1 && t + p.ahead < p.T && l * 64 < heads * D)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(x + p.ahead * stride + l * 64));

    if (slot < 0) return;
    if (slot >= p.num_slots || (p.R && (pos < 0 || pos >= p.max_pos))) {
        report_bad_page(p.status);
        return;
    }
    uint16_t* y;
    int64_t step;   // from a head to the next
    if (kind == 0) {
        const int n = p.by_sq.div(t);
        step = static_cast<int64_t>(p.Sq) * D;
        y = p.q_out + (static_cast<int64_t>(n) * p.Hq + h0) * step + static_cast<int64_t>(t - n * p.Sq) * D;
    } else {
        const int64_t page = p.by_page.div(static_cast<int>(slot));
        step = p.head_stride;
        y = (kind == 1 ? p.kc : p.vc) + page * p.page_stride + (slot - page * p.page) * p.token_stride + h0 * step;
    }
    if (kind == 2) {
#pragma unroll
        for (int k = 0; k < HEADS; ++k)
            if (k < heads) {
                *reinterpret_cast<uint4*>(y + k * step + r.a) = u[k][0];
                *reinterpret_cast<uint4*>(y + k * step + r.b) = u[k][1];
            }
        return;
    }

    const uint16_t* w = kind == 0 ? p.wq : p.wk;
    const bool turn = l < p.R / 16;
    uint64_t pa[4], pb[4], qa[4], qb[4];   // what x_i and its partner are multiplied with, both runs
    if (w) {
        unpack8(*reinterpret_cast<const uint4*>(w + r.a), pa);
        unpack8(*reinterpret_cast<const uint4*>(w + r.b), pb);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) pa[i] = pb[i] = f32x2(1.f, 1.f);
    }
    if (turn) {
        // the thread's eight angles: features 8l .. 8l + 7 of either half, or its eight neighbouring pairs
        const float* cs = p.cos_sin + static_cast<int64_t>(pos) * p.R + 8 * l;
        const float4 c0 = *reinterpret_cast<const float4*>(cs), c1 = *reinterpret_cast<const float4*>(cs + 4);
        const float4 s0 = *reinterpret_cast<const float4*>(cs + p.R / 2), s1 = *reinterpret_cast<const float4*>(cs + p.R / 2 + 4);
        const float c[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
        const float s[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (PAIRS) {   // angle i turns the i-th pair of run a, angle 4 + i that of run b
                qa[i] = fmul2(swap2(pa[i]), f32x2(-s[i], s[i]));
                qb[i] = fmul2(swap2(pb[i]), f32x2(-s[4 + i], s[4 + i]));
                pa[i] = fmul2(pa[i], f32x2(c[i], c[i]));
                pb[i] = fmul2(pb[i], f32x2(c[4 + i], c[4 + i]));
            } else {
                qa[i] = fmul2(pb[i], f32x2(-s[2 * i], -s[2 * i + 1]));
                qb[i] = fmul2(pa[i], f32x2(s[2 * i], s[2 * i + 1]));
                pa[i] = fmul2(pa[i], f32x2(c[2 * i], c[2 * i + 1]));
                pb[i] = fmul2(pb[i], f32x2(c[2 * i], c[2 * i + 1]));
            }
        }
    }
#pragma unroll
    for (int k = 0; k < HEADS; ++k) {
        if (k >= heads) break;
        uint64_t a[4], b[4];
        unpack8(u[k][0], a);
        unpack8(u[k][1], b);
        float inv = 1.f;
        if (w) {
            uint64_t s0 = fmul2(a[0], a[0]), s1 = fmul2(b[0], b[0]);
#pragma unroll
            for (int i = 1; i < 4; ++i) {
                s0 = ffma2(a[i], a[i], s0);
                s1 = ffma2(b[i], b[i], s1);
            }
            float lo, hi;
            f32x2_split(fadd2(s0, s1), lo, hi);
            float ss = lo + hi;
#pragma unroll
            for (int o = L / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(group, ss, o);
            inv = rsqrtf(ss * (1.f / D) + p.eps);
        }
        const uint64_t inv2 = f32x2(inv, inv);
        uint64_t ya[4], yb[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            ya[i] = fmul2(a[i], pa[i]);
            yb[i] = fmul2(b[i], pb[i]);
        }
        if (turn) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                ya[i] = ffma2(PAIRS ? swap2(a[i]) : b[i], qa[i], ya[i]);
                yb[i] = ffma2(PAIRS ? swap2(b[i]) : a[i], qb[i], yb[i]);
            }
        }
        if (w) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                ya[i] = fmul2(ya[i], inv2);
                yb[i] = fmul2(yb[i], inv2);
            }
        }
        *reinterpret_cast<uint4*>(y + k * step + r.a) = pack8(ya);
        *reinterpret_cast<uint4*>(y + k * step + r.b) = pack8(yb);
    }
}

template <int D, bool PAIRS, int HEADS>
int launch_append(AppendParams& p, cudaStream_t st)
{
    p.q_sets = (p.Hq + HEADS - 1) / HEADS;
    p.kv_sets = (p.Hkv + HEADS - 1) / HEADS;
    const int sets = p.q_sets + 2 * p.kv_sets;
    p.by_sets = FastDiv(static_cast<uint32_t>(sets));
    p.ahead = num_sms() * kCtas * kThreads / (D / 16) / sets / 2 + 1;   // half of what the GPU holds
    const long long threads = static_cast<long long>(p.T) * sets * (D / 16);
    FMHA_CHECK_CUDA(launch_pdl(rope_append_kernel<D, PAIRS, HEADS>, dim3(static_cast<unsigned>((threads + kThreads - 1) / kThreads)), dim3(kThreads), 0, st, p));
    count_launch();
    return FMHA_OK;
}

// Four heads per group of threads once the threads of one head each would more than fill the GPU; below that one
// head each, which is the shorter chain (48 heads of 128, one head against four: 256 tokens 2.9 us against 3.6,
// 512 4.2 / 4.0, 1024 6.2 / 6.0, 2048 10.4 / 8.8, 8192 49.7 / 35.1).
template <int D, bool PAIRS>
int run_append(AppendParams& p, cudaStream_t st)
{
    const long long threads = static_cast<long long>(p.T) * (p.Hq + 2 * p.Hkv) * (D / 16);
    return threads > 2048LL * num_sms() ? launch_append<D, PAIRS, 4>(p, st) : launch_append<D, PAIRS, 1>(p, st);
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
    if (static_cast<long long>(T) * (Hq + 2LL * cache->Hkv) >= (1LL << 31) - 256)
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
    p.by_page = FastDiv(static_cast<uint32_t>(cache->page_size));
    p.by_sq = FastDiv(static_cast<uint32_t>(Sq));
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (cache->D == 64) return interleaved ? run_append<64, true>(p, st) : run_append<64, false>(p, st);
    return interleaved ? run_append<128, true>(p, st) : run_append<128, false>(p, st);
}
