/*
 * fmha.h - C ABI of the GB300 (sm_103a) fused attention library, libfmha.so.
 *
 * Computes O = softmax(scale * Q K^T) V over BF16 Q/K/V, with an online (running max / sum)
 * softmax and O rescale across key/value tiles, a split-KV decode path with a combine step,
 * and optional NVFP4 quantisation of O.  Sources:
 *   - "NVFP4-1.1_RAW_CUDA_CPP_APPROACH.md" (nvfp4-megamoe-kernel), kernel plan items 1-7:
 *     TMA loads of Q/K/V, tcgen05 MMA with a Tensor Memory accumulator, in-kernel softmax with
 *     O rescale, multi-KV-tile support, FP4 quantisation for NVFP4;
 *   - "CURRENT_ISSUE.md" @4b129c1, QK verify kernel: tensors laid out (B, H, S, D) contiguous;
 *   - "CURRENT_ISSUE.md" @57d67e6, "The 4x Bug": the raw S = Q K^T check (fmha_qk_gemm).
 *
 * Conventions shared by every entry point:
 *   - All tensor pointers are DEVICE pointers owned by the caller; the library never allocates
 *     or frees device memory, never synchronises (except fmha_check_status) and launches only
 *     on `stream`.  Inputs are read-only; outputs must not alias inputs.
 *   - Kernels are launched with programmatic dependent launch (except while `stream` is being
 *     captured into a graph): a call's kernel may be placed on the SMs while the previous kernel of
 *     `stream` finishes, but touches no global memory until that kernel has completed, so calls keep
 *     plain stream order (a call may read what the previous kernel wrote, or overwrite what it read).
 *   - Layouts are contiguous, row-major: Q/O [B][Hq][Sq][D], K/V [B][Hkv][Skv][D], LSE [B][Hq][Sq].
 *   - Grouped-query attention: query head hq reads key/value head hq / (Hq / Hkv).
 *   - LSE is the natural logarithm of sum_j exp(scale * q.k_j) (scale included), FP32.
 *   - A key set of size 0 (seqlens_k[b] == 0) gives O = 0 and LSE = -inf.
 *   - Tensor pointers must be 16-byte aligned (LSE, seqlens_k, nvfp4_scale_in and out_amax:
 *     4-byte; the workspace: 256-byte).  D must be 64, 128 or 512 (16 is also accepted by
 *     fmha_qk_gemm).
 *   - Return value: FMHA_OK or an fmha_status code; nothing aborts or throws.  A failed call
 *     leaves a message for fmha_error_string(code) / fmha_last_error() of the calling thread.
 *   - Asynchronous device-side failures (a bounded wait inside a kernel that timed out) are
 *     reported by fmha_check_status().
 */
#ifndef FMHA_H_
#define FMHA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* cudaStream_t without pulling in the CUDA headers; NULL = the legacy default stream. */
typedef struct CUstream_st* fmha_stream_t;

typedef enum {
    FMHA_OK = 0,
    FMHA_ERR_INVALID = 1,     /* bad argument: NULL pointer, Hq % Hkv != 0, unsupported D, misalignment */
    FMHA_ERR_UNSUPPORTED = 2, /* valid request that this library does not implement */
    FMHA_ERR_WORKSPACE = 3,   /* workspace missing or smaller than fmha_workspace_size() */
    FMHA_ERR_CUDA = 4,        /* a CUDA runtime/driver call or kernel launch failed */
    FMHA_ERR_TIMEOUT = 5,     /* a kernel's bounded wait expired (see fmha_check_status) */
    FMHA_ERR_RACE = 6,        /* a split-KV merge counter never settled: calls sharing one
                                 workspace (or the allocation-free scratch) overlapped on the
                                 GPU, so some output rows may be unmerged (see fmha_check_status).
                                 Make the call once eagerly before a captured one of that workspace
                                 is replayed: that clears the arrivals a replay would take up */
    FMHA_ERR_PAGES = 7        /* a paged-cache call met data out of bounds on the device: a length, page,
                                 slot or position, or too few free pages (see fmha_check_status) */
} fmha_status;

typedef enum {
    FMHA_OUT_BF16 = 0,  /* out: BF16 [B,Hq,Sq,D] */
    FMHA_OUT_F32 = 1,   /* out: FP32 [B,Hq,Sq,D] */
    FMHA_OUT_NVFP4 = 2  /* out: packed E2M1 codes [B,Hq,Sq,D/2] (element 2i in bits 3:0),
                           plus out_scales / out_tensor_scale below */
} fmha_out_kind;

typedef struct {
    int out_kind;             /* fmha_out_kind; default FMHA_OUT_BF16 */
    const int32_t* seqlens_k; /* device int32[B], 0 <= seqlens_k[b] <= Skv: keys at or beyond
                                 seqlens_k[b] are never read (ragged batches); NULL = all Skv */
    int num_splits;           /* 0 = automatic split-KV; 1 = no split (each (b, kv-head) handled
                                 by one CTA, or by one CTA pair for D = 512; no workspace needed
                                 for BF16/F32 output).  With 0 and
                                 a workspace, causal or ragged problems on the 128-row path (more
                                 than 16 query rows per key/value head) also take their work items
                                 from a counter in the workspace (balanced across SMs); with 1, or
                                 no workspace, in a fixed order.  0 without a workspace acts as 1 */
    void* workspace;          /* device scratch of at least fmha_workspace_size() bytes (256-B
                                 aligned); contents on entry do not matter */
    size_t workspace_bytes;
    uint8_t* out_scales;      /* NVFP4: E4M3 block scales [B,Hq,Sq,D/16] */
    float* out_tensor_scale;  /* NVFP4: device float[1], the per-tensor scale s_g */
    float* out_f32;           /* optional, NVFP4 only: the FP32 O that was quantised */
    int causal;               /* 1: bottom-right aligned causal mask: with n keys, query i of Sq sees
                                 keys 0 .. i + n - Sq (a query that sees none gets O = 0,
                                 LSE = -inf); 0 = all keys */
    const float* nvfp4_scale_in; /* NVFP4, optional: device float[1], a given per-tensor scale s_g
                                 (e.g. an earlier step's max|O| / 2688).  Set: single pass, the
                                 attention epilogues write codes and block scales with this s_g
                                 directly; no amax pass, no FP32 staging, no workspace for NVFP4.
                                 Blocks beyond 6 * 448 * s_g saturate; an s_g that is not a
                                 positive finite number gives all-zero codes and scales;
                                 *out_tensor_scale receives s_g.  NULL: s_g = fp32(max|O| / 2688)
                                 of this O (two passes) */
    float* out_amax;          /* optional, NVFP4 only: device float[1], receives max|O| (FP32) of
                                 this call (with two passes it is also the max the quantiser uses) */
    int wide_variant;         /* D = 512 kernel (fmha_wide_variant); results agree within rounding */
} fmha_opts;

/* Kernel variants for D = 512 (the value columns are split over a pair of CTAs either way). */
typedef enum {
    FMHA_WIDE_AUTO = 0,        /* the faster one measured on GB300: FMHA_WIDE_INDEPENDENT */
    FMHA_WIDE_INDEPENDENT = 1, /* two independent CTAs: each loads every K tile, computes the full S */
    FMHA_WIDE_PAIR = 2         /* a cluster of two CTAs running pair MMAs (tcgen05 cta_group::2): each
                                  CTA loads half of every K tile, the PV product runs over a doubled
                                  contraction; dense keys only (with seqlens_k the independent CTAs
                                  run) */
} fmha_wide_variant;

/*
 * Attention forward with default options (BF16 output, dense keys, no workspace, no split).
 *   q: BF16 [B,Hq,Sq,D]; k, v: BF16 [B,Hkv,Skv,D]; out: BF16 [B,Hq,Sq,D];
 *   lse: FP32 [B,Hq,Sq] or NULL; scale: multiplies Q K^T before the softmax, a positive finite number
 *   (FMHA_ERR_INVALID otherwise: the kernels scale each row's maximum score after taking it).
 * Same as fmha_fwd_ex(..., opts = NULL): every (b, kv-head) unit is handled whole by one CTA (for
 * D = 512 by one CTA pair, each CTA writing its half of the value columns), so nothing needs a
 * workspace.  Decode shapes with few units leave SMs idle this way; fmha_fwd_ex with a workspace
 * splits the keys over every SM instead.
 */
int fmha_fwd(const void* q, const void* k, const void* v, void* out, float* lse, int B, int Hq, int Hkv,
             int Sq, int Skv, int D, float scale, fmha_stream_t stream);

/*
 * Attention forward with options (output kind, ragged key lengths, causal mask, split-KV, NVFP4).
 * opts == NULL means all defaults.  Split-KV, the balanced work-item order and NVFP4 output need
 * opts->workspace; calls that share one workspace must be ordered on one stream.
 */
int fmha_fwd_ex(const void* q, const void* k, const void* v, void* out, float* lse, int B, int Hq, int Hkv,
                int Sq, int Skv, int D, float scale, fmha_stream_t stream, const fmha_opts* opts);

/* Bytes of workspace fmha_fwd_ex needs for this problem and these options (0 if none). */
size_t fmha_workspace_size(int B, int Hq, int Hkv, int Sq, int Skv, int D, const fmha_opts* opts);

/*
 * Attention from host memory: copies Q, K and V to the device, runs fmha_fwd_ex, and copies O and
 * the LSE back, all ordered after the work already on `stream`.  Returns once everything is
 * enqueued: synchronise `stream` before reading out_host / lse_host.
 *   q_host, k_host, v_host: host BF16 arrays in the fmha_fwd layouts; out_host: host O, BF16 or
 *   (opts->out_kind == FMHA_OUT_F32) FP32 [B,Hq,Sq,D]; lse_host: host FP32 [B,Hq,Sq] or NULL.
 *   Page-locked host memory (cudaHostAlloc, cudaHostRegister) makes the copies asynchronous;
 *   pageable memory works, but the copies then hold up the calling thread.
 *   dev_buf: device memory of at least fmha_host_buffer_size() bytes, 256-byte aligned, owned by the
 *   caller; it stages Q, K, V, O and the LSE and holds the attention workspace, so the call
 *   allocates nothing.  Calls that share dev_buf must be ordered on one stream.
 *   opts: as for fmha_fwd_ex, limited to out_kind (BF16 or F32), num_splits, causal and
 *   wide_variant; seqlens_k, the NVFP4 fields and the workspace fields must be NULL / 0
 *   (FMHA_ERR_UNSUPPORTED otherwise).  opts == NULL: BF16 output, automatic split-KV.
 * With B >= 2 the batch runs in up to four chunks of whole batch entries, so that the copy of one
 * chunk's inputs overlaps the attention of the one before (an internal copy stream per device, joined
 * back to `stream` through events; calls from several host threads are serialised while they
 * enqueue).  Errors: FMHA_ERR_INVALID (NULL or bad arguments), FMHA_ERR_WORKSPACE (dev_buf missing,
 * misaligned or too small), FMHA_ERR_UNSUPPORTED, FMHA_ERR_CUDA; with an error nothing is enqueued,
 * except for FMHA_ERR_CUDA from a failing copy or launch, after which out_host is unspecified.
 */
int fmha_fwd_host(const void* q_host, const void* k_host, const void* v_host, void* out_host, float* lse_host, int B,
                  int Hq, int Hkv, int Sq, int Skv, int D, float scale, fmha_stream_t stream, const fmha_opts* opts,
                  void* dev_buf, size_t dev_buf_bytes);

/* Bytes of device memory fmha_fwd_host needs for this problem and these options (0 if invalid). */
size_t fmha_host_buffer_size(int B, int Hq, int Hkv, int Sq, int Skv, int D, const fmha_opts* opts);

/*
 * NVFP4 quantisation of an FP32 tensor x[n], n % 16 == 0 (the NVFP4 step of the pages' kernel
 * plan, "FP4 quantization for NVFP4-1.1"):
 *   s_g = fp32(amax / (6 * 448)); per block of 16: sc = E4M3(amax_block / (6 s_g)) (round to
 *   nearest even, saturating at 448); code_i = E2M1(x_i / (sc * s_g)) (nearest even, saturating
 *   at 6, sign copied).  amax == 0 gives all-zero codes and scales.
 *   q: uint8[n/2] codes, element 2i in bits 3:0 and 2i+1 in bits 7:4.
 *   scales: nvfp4_scales_bytes(n) bytes: E4M3 scales [n/16], then at byte offset
 *   align16(n/16) the FP32 s_g, then 12 bytes the call uses as scratch.
 */
int nvfp4_quantize(const float* x, uint8_t* q, uint8_t* scales, int64_t n, fmha_stream_t stream);

/* Size in bytes of the `scales` buffer nvfp4_quantize needs for n values. */
size_t nvfp4_scales_bytes(int64_t n);

/*
 * NVFP4 encoding of x[n] (n % 16 == 0) with a given per-tensor scale: tensor_scale is a device
 * float[1] holding s_g.  q: n/2 bytes of E2M1 codes (as nvfp4_quantize); scales: n/16 bytes of
 * E4M3 block scales (no trailing s_g).  Same roundings as nvfp4_quantize; blocks beyond
 * 6 * 448 * s_g saturate and an s_g that is not a positive finite number gives all zeros.
 * Errors: FMHA_ERR_INVALID for NULL pointers, n < 0, n % 16 != 0, or x not 16-byte, q not 8-byte
 * or tensor_scale not 4-byte aligned.
 */
int nvfp4_quantize_scaled(const float* x, uint8_t* q, uint8_t* scales, int64_t n, const float* tensor_scale,
                          fmha_stream_t stream);

/*
 * ---- Paged key/value cache -----------------------------------------------------------------------
 * Keys and values of many requests of growing lengths in pools of equal pages: page p, key/value head
 * h, token t of the page and feature d are at element p * page_stride + h * head_stride +
 * t * token_stride + d of either pool.  Heads outside tokens ([pages][Hkv][page_size][D]) and tokens
 * outside heads ([pages][page_size][Hkv][D]) are both strides of this form; a dense [B][Hkv][Skv][D]
 * tensor is a cache of B pages of Skv tokens.  A request's tokens j = 0, 1, .. are in the pages of its
 * row of a block table: page block_table[b][j / page_size], token j % page_size of it.  A slot is a
 * token's place in the pool, page * page_size + token.
 *
 * A step of serving is fmha_page_table (pages and slots for the new tokens), then in every layer
 * fmha_rope_append (queries, and keys and values into the cache) and fmha_fwd_paged.  Where several
 * requests continue one prompt, fmha_page_fork and fmha_page_copy go before them, the requests hold the
 * pages of their common beginning together, and fmha_fwd_prefix reads those once.  All are
 * stream-ordered, allocate nothing and can be captured.  Data on the device that is out of bounds (a
 * length, page, slot or position) is never followed: the call does what its text says and
 * fmha_check_status reports FMHA_ERR_PAGES.
 */
typedef struct {
    void* k;              /* device BF16 pools, 16-byte aligned */
    void* v;
    int num_pages;        /* >= 1; num_pages * page_size below 2^31 */
    int page_size;        /* tokens per page, >= 1 (fmha_fwd_paged: a multiple of 8) */
    int Hkv;              /* key/value heads */
    int D;                /* 64 or 128 */
    int64_t page_stride;  /* elements; each a multiple of 8, at least D, below 2^38 */
    int64_t head_stride;
    int64_t token_stride;
} fmha_kv_cache;

/*
 * Pages, block tables and slots from request lengths, for one step of B requests (at most 8192), in
 * one launch (two for an update in place of more than 2048 tokens or requests).
 *   ctx_lens: int32[B], tokens request b has in the cache; new_lens: int32[B], tokens to come (0: none),
 *   or a negative number: the request is done and its pages go back.
 *   free_pages: int32[num_pages], a stack of free pages whose height is *free_count.  First the pages of
 *   done requests are pushed, in request order and page order; then every other request with more tokens
 *   than pages is given pages from the top, in request order.
 *   block_table: int32[B][max_pages]; the entries of new pages are written, no other is.
 * Outputs: seqlens[b] = ctx + new (0 for a done request); cu_new: int32[B + 1], first new token of each
 *   request and their total; positions[t] and slots[t], t < T, of the new tokens in request order; behind
 *   the last one positions 0 and slots -1 (T may be larger than the total, e.g. a captured size);
 *   *free_count_out, the stack's new height.
 * seqlens may be the ctx_lens array and free_count_out may be free_count (an update in place); no other
 * arrays may overlap.  With a length that is negative or passes the table row, a stack height outside
 * 0..num_pages, too few free pages, or more than T new tokens, nothing is given or taken: seqlens =
 * ctx_lens, cu_new 0, positions 0, slots -1, the stack as it was, and FMHA_ERR_PAGES from
 * fmha_check_status.  An id that is not one of the pool's pages is handed on like any other: a token on
 * such a page gets slot -1, and a done request's goes on the stack with its other pages, both with the
 * same report.  It stays in the pool until the program takes it out.
 * All pointers device memory; slots 8-byte, the others 4-byte aligned.
 */
int fmha_page_table(const int32_t* ctx_lens, const int32_t* new_lens, int B, int page_size, int32_t* free_pages,
                    const int32_t* free_count, int num_pages, int32_t* block_table, int max_pages, int32_t* seqlens,
                    int32_t* cu_new, int32_t* positions, int64_t* slots, int T, int32_t* free_count_out,
                    fmha_stream_t stream);

/*
 * Norms of the query and key heads, position rotation and the store in the cache, in one pass.
 *   q: BF16, head h of token t at q + t * q_stride + h * D (strides in elements, multiples of 8); k, v
 *   alike with the cache's Hkv heads: the three may be parts of one projection's rows.
 *   q_weight, k_weight: BF16[D], y = x / sqrt(mean(x^2) + eps) * weight per head; NULL: y = x.
 *   cos_sin: FP32 [max_pos][rope_dim], rope_dim / 2 cosines and then as many sines of each position;
 *   positions: int32[T].  The first rope_dim features of queries and keys are rotated: feature i with
 *   i + rope_dim / 2, or (interleaved != 0) 2i with 2i + 1.  rope_dim: a multiple of 16 up to D, 0 = none
 *   (cos_sin and positions are not read).
 *   slots: int64[T], distinct; a negative slot is padding: that token's rows of q, k and v, which are there, may
 *   hold anything, and nothing of it is written.
 *   q_out: BF16 [T / Sq][Hq][Sq][D], token t = n * Sq + s at [n][h][s] (Sq = 1: [T][Hq][D]).
 * Keys and values go to their slots of `cache` (values as they are).  FP32 throughout, one rounding to
 * BF16 per output.  A token with a slot or position out of bounds is left out like padding and reported.
 * Pointers 16-byte aligned (positions 4, slots 8).
 */
int fmha_rope_append(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                     const void* q_weight, const void* k_weight, float eps, const float* cos_sin, int max_pos, int rope_dim,
                     int interleaved, const int32_t* positions, const int64_t* slots, void* q_out,
                     const fmha_kv_cache* cache, int T, int Hq, int Sq, fmha_stream_t stream);

/*
 * Attention of the last Sq tokens of each request over its pages: fmha_fwd_ex with K and V row j of
 * request b taken from the cache through block_table (int32 [B][max_pages]) and seqlens[b] keys (device
 * int32[B], 0 <= seqlens[b] <= max_pages * page_size).  q, out, lse as in fmha_fwd; D and Hkv are the
 * cache's; page_size a multiple of 8; with D = 128 page_stride a multiple of 8 * token_stride.
 *   opts (NULL: defaults): out_kind, num_splits, workspace, causal and the NVFP4 fields as for fmha_fwd_ex;
 *   seqlens_k must be NULL.  With a workspace of fmha_paged_workspace_size() bytes the keys are split over
 *   every SM, without one each (request, kv-head) is one CTA's.
 * Made for up to 16 query rows per key/value head, (Hq / Hkv) * Sq; more rows run in chunks of at most 16,
 * each reading the keys again.  Entries of the block table behind the last key are not read.  Queries, keys and
 * values are finite (a score of NaN or +infinity makes its row and that row's LSE NaN, however the keys are
 * split); pool rows behind a request's length may hold anything (NaN too).  A page out of the pool
 * reads as zero keys and values, a length out of bounds is clamped, and both are reported.
 */
int fmha_fwd_paged(const void* q, const fmha_kv_cache* cache, const int32_t* block_table, int max_pages,
                   const int32_t* seqlens, void* out, float* lse, int B, int Hq, int Sq, float scale,
                   fmha_stream_t stream, const fmha_opts* opts);

/* Bytes of workspace fmha_fwd_paged needs for this problem and these options (0 if none or invalid). */
size_t fmha_paged_workspace_size(int B, int Hq, int Sq, const fmha_kv_cache* cache, const fmha_opts* opts);

/*
 * ---- Pages that requests share ---------------------------------------------------------------------
 * Requests that continue one prompt (parallel samples, beams, a common system prompt) may have the same
 * pages at the beginning of their rows of the block table.  Who holds a page stands in the table alone:
 * there are no reference counts.  Pages that several requests hold are full and are not written any more;
 * a partly filled page belongs to one request.  fmha_page_fork keeps it so.  Requests that share pages end
 * through fmha_page_fork, as fmha_page_table gives back every page of a request that ends.
 */

/*
 * Attention of the last Sq tokens of each request over its pages, as fmha_fwd_paged, with the common
 * beginning of the requests of a group read once for all of them.
 *   cu_groups: int32[N + 1], first request of each group and B; N >= 1 groups (at most 8192) of neighbouring
 *   requests, in order, that make up the batch; a group may have one request, or none.
 *   prefix_lens: int32[N], tokens that the group's requests have in the same pages: the rows of the block table
 *   agree there, as far as each request's tokens reach (a request may end inside, and an empty slot has none).
 *   They are read through the row of the group's first request, so as far as its tokens reach (the other requests
 *   read what is left through their own rows): a group whose first slot is empty shares nothing, so a request with all of
 *   the prefix goes first (64 samples behind 8192 keys: 43 us, 157 with an empty first slot).
 *   q, cache, block_table, max_pages, seqlens, out, lse, scale: as in fmha_fwd_paged, and the same results within
 *   rounding.  The call is fmha_fwd_paged's and does not look at the groups with more than 64 rows per key/value head,
 *   (Hq / Hkv) * Sq, or at most 6000 tiles of 128 keys in all heads if every table row were full: the table's width decides, not
 *   the lengths, which are on the device.  (Behind a wide table a few short requests take about 8 us longer than behind a narrow
 *   one, or than in fmha_fwd_paged.)
 *   Of the others a group's keys are read once where that takes less than its requests' own reads, in whole tiles of 128.
 *   opts: out_kind, workspace (always needed: fmha_prefix_workspace_size() bytes), causal and the NVFP4 fields;
 *   num_splits 0 (or above 1); seqlens_k must be NULL.
 * Lengths and pages out of bounds as in fmha_fwd_paged; with cu_groups that is no such list nothing is
 * shared; each is reported.  A prefix length below 0 is 0.
 */
int fmha_fwd_prefix(const void* q, const fmha_kv_cache* cache, const int32_t* block_table, int max_pages,
                    const int32_t* seqlens, const int32_t* cu_groups, const int32_t* prefix_lens, int N, void* out, float* lse,
                    int B, int Hq, int Sq, float scale, fmha_stream_t stream, const fmha_opts* opts);

/* Bytes of workspace fmha_fwd_prefix needs for this problem and these options (0 if none or invalid). */
size_t fmha_prefix_workspace_size(int B, int Hq, int Sq, const fmha_kv_cache* cache, const fmha_opts* opts);

/*
 * The next step's B requests as children of this step's B_old (at most 8192 each), in one launch: the
 * choice of a beam search, a prompt forked into samples, requests that end, a batch put in another order.
 *   parents: int32[B], the request that child b continues, or a negative number: an empty slot.
 *   ctx_lens: int32[B_old], tokens in the cache; block_table: int32[B_old][max_pages]; page_size.
 *   free_pages, free_count, num_pages (at most 2^19): the stack of free pages, as in fmha_page_table.
 * A child has its parent's tokens and pages, except that of several children of one parent all but the first
 * get a page of their own in place of a partly filled last one, whose tokens are to be copied (fmha_page_copy).
 * A request without children ends.  First the pages that rows of ended requests name and no row of a
 * continued one does are pushed, in the order of their ids; then the copies' pages are taken from the top,
 * in the order of the children.
 * Outputs: new_table: int32[B][max_pages], the entries of each child's pages (no other is written); seqlens[b];
 *   copy_src[b], copy_dst[b] and copy_tokens[b]: the page to be copied, to which, and how many tokens of it (-1, -1, 0:
 *   none); *free_count_out, the stack's new height (may be free_count; no other arrays may overlap).
 * With a parent that is not one of the B_old, a length that is negative or passes the table row, a stack height
 * outside 0..num_pages or passing it, or too few free pages, the stack stays as it was, seqlens are 0, the copies none,
 * new_table holds nothing of use, and FMHA_ERR_PAGES is reported: the old table still stands.  An id that is not one
 * of the pool's pages is handed on to children, not given back, and reported.
 * All arrays device memory, 4-byte aligned.
 */
int fmha_page_fork(const int32_t* parents, int B, const int32_t* ctx_lens, int B_old, int page_size, const int32_t* block_table,
                   int max_pages, int32_t* free_pages, const int32_t* free_count, int num_pages, int32_t* new_table,
                   int32_t* seqlens, int32_t* copy_src, int32_t* copy_dst, int32_t* copy_tokens, int32_t* free_count_out,
                   fmha_stream_t stream);

/*
 * Copies pages inside each of n_caches caches (a model's layers, of one size and the same strides; the array is read
 * on the host): the first tokens[i] tokens (NULL: all) of page src[i], all heads, keys and values, to page dst[i],
 * i < n, or i < *count if count is given (device int32[1], 0..n).  A pair with a negative page is left out.
 * No page may be a destination twice, or source and destination.  A page outside the pool is left out, a
 * number of tokens or pairs outside its range clamped, and each is reported.
 * src, dst, tokens: int32[n], device memory, 4-byte aligned.
 */
int fmha_page_copy(const fmha_kv_cache* caches, int n_caches, const int32_t* src, const int32_t* dst, const int32_t* tokens, int n,
                   const int32_t* count, fmha_stream_t stream);

/*
 * Used pages to the low ids, in one launch or two: with n = *free_count of num_pages (at most 2^20) pages free, the used ones
 * end up in 0 .. num_pages - n - 1.  The k-th used page behind them moves to the k-th free page among them.  The data
 * moves with fmha_page_copy(copy_src, copy_dst, NULL, n_copies, copy_count) in every layer.
 *   seqlens: int32[B], tokens of each request; block_table: int32[B][max_pages]; free_pages: int32[num_pages].
 * A page that is not on the stack is used, whether or not a request names it.
 * Outputs: new_ids: int32[num_pages], where each page goes (itself if it stays; -1: free); new_table: int32[B][max_pages],
 *   block_table's entries of each request's pages with their new ids (no other is written); copy_src, copy_dst: int32[n_copies],
 *   n_copies >= num_pages / 2, the *copy_count moves, and -1 behind them; free_pages_out: the stack, the lowest free page
 *   on top, the same number of pages (its entries above are not written).  No arrays may overlap.
 * With a stack height outside 0..num_pages, an entry that is not one of the pool's pages or is twice on the stack, or a
 * length that is negative or passes the table row, nothing moves (new_ids, tables and stack as they are, no copies)
 * and FMHA_ERR_PAGES is reported.  An entry of the table that is no page of the pool, or a free one, is
 * handed on and reported.
 * All arrays device memory, 4-byte aligned.
 */
int fmha_page_compact(const int32_t* seqlens, int B, int page_size, const int32_t* block_table, int max_pages,
                      const int32_t* free_pages, const int32_t* free_count, int num_pages, int32_t* new_ids, int32_t* new_table,
                      int32_t* copy_src, int32_t* copy_dst, int n_copies, int32_t* copy_count, int32_t* free_pages_out,
                      fmha_stream_t stream);

/*
 * Test hook: raw S = Q K^T in FP32, no scale ("CURRENT_ISSUE.md" @57d67e6, "The 4x Bug":
 * the single tcgen05 MMA product checked against a scalar dot product).
 *   q: BF16 [Sq,D], k: BF16 [Skv,D], s: FP32 [Sq,Skv]; D in {16, 64, 128, 512}.
 */
int fmha_qk_gemm(const void* q, const void* k, float* s, int Sq, int Skv, int D, fmha_stream_t stream);

/*
 * Test hook: layout self-checks of the building blocks.  Each writes its results to `out`
 * (device, `out_bytes` bytes, see the test-suite for the layouts) from inputs in `in`:
 *   which = 1: Tensor Memory round trip (tcgen05.st then tcgen05.ld, 32x32b shape);
 *   which = 2: O^T = V^T P^T with V^T an MN-major shared-memory operand (decode PV form);
 *   which = 3: O = P V with P in Tensor Memory and V MN-major in shared memory (TS form).
 */
int fmha_selftest(int which, const void* in, void* out, size_t out_bytes, int param, fmha_stream_t stream);

/*
 * Waits for `stream`, then returns FMHA_ERR_TIMEOUT if any kernel of this library timed out
 * in a bounded wait since the last call, FMHA_ERR_RACE if a split-KV merge found its arrival
 * counter changing under it (overlapping calls on one workspace), FMHA_ERR_PAGES if a paged-cache
 * call met device data out of bounds, clearing that state in all three cases.  Of several, the
 * latest of TIMEOUT and RACE is reported, and PAGES only after neither: the results of calls that met data
 * out of bounds are defined, those of the other two are not.  FMHA_ERR_CUDA if the stream reports an error; else FMHA_OK.
 */
int fmha_check_status(fmha_stream_t stream);

/* Bounded-wait limit in SM clock cycles for later launches (0 = default, about 2 s). */
void fmha_set_wait_limit(long long cycles);

/*
 * Split-KV decode that allocates nothing.  The pages have no counterpart: it serves callers that
 * cannot hand the library a workspace, such as plug-ins and foreign-language bindings that see
 * only tensor pointers and have no allocator to ask, or latency-critical loops that must not call
 * cudaMalloc (it can synchronise the device and its latency is unbounded).
 *   Same arguments and results as fmha_fwd (BF16 out, optional LSE) plus seqlens_k (device
 *   int32[B] or NULL, as in fmha_opts); at most 16 query rows per key/value head, D = 64 or 128.
 *   The split-KV scratch (partials and tile prefix) is a fixed array of FMHA_NOALLOC_SCRATCH_BYTES
 *   inside the library, held by every GPU that loads it until the process exits; a problem that
 *   needs more returns FMHA_ERR_WORKSPACE with the size in fmha_last_error().  The library calls
 *   no allocation routine.  The first call on a device looks up that device's address of the
 *   array (make it before any stream capture).  All calls on a device share the array: calls that
 *   overlap on the GPU race and must be ordered by the caller.
 */
#define FMHA_NOALLOC_SCRATCH_BYTES (8u * 1024u * 1024u)
int fmha_fwd_decode_noalloc(const void* q, const void* k, const void* v, void* out, float* lse, int B, int Hq,
                            int Hkv, int Sq, int Skv, int D, float scale, const int32_t* seqlens_k,
                            fmha_stream_t stream);

/* Number of kernels this library has launched in this process (all devices, all threads). */
long long fmha_launch_count(void);

/*
 * Timing hook, one-shot and per calling thread: the next attention / quantisation call records
 * `start_event` on its stream immediately before launching its dominant kernel (the attention
 * kernel; the quantiser for nvfp4_quantize) and `stop_event` right after it.  Both are
 * cudaEvent_t handles owned by the caller; NULL, NULL clears the hook.
 */
void fmha_time_next_call(void* start_event, void* stop_event);

/* Static text for a status code. */
const char* fmha_error_string(int code);

/* Message of the last failing call on this thread ("" if none). */
const char* fmha_last_error(void);

/* Number of SMs of the current device as the library sees it (0 on failure). */
int fmha_num_sms(void);

#ifdef __cplusplus
}
#endif
#endif /* FMHA_H_ */
