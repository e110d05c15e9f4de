"""GB300 (sm_103a) fused multi-head attention: Python binding of libfmha.so.

Thin marshalling only (ctypes; the paged cache's entry points through the native _binding.so, whose
checks and calls take a microsecond): every step of attention, split-KV combine and NVFP4 quantisation
runs in the library's CUDA kernels.  torch tensors supply device memory and the current stream.
There is no CPU path: if libfmha.so is missing or cannot load, every call raises.

Function names match the C ABI in include/fmha.h.
"""
from __future__ import annotations

import ctypes
import os
import re
import threading

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libfmha.so")
HEADER = os.path.join(os.path.dirname(PKG), "include", "fmha.h")

FMHA_OK = 0
FMHA_ERR_INVALID = 1
FMHA_ERR_UNSUPPORTED = 2
FMHA_ERR_WORKSPACE = 3
FMHA_ERR_CUDA = 4
FMHA_ERR_TIMEOUT = 5
FMHA_ERR_RACE = 6
FMHA_ERR_PAGES = 7
FMHA_OUT_BF16 = 0
FMHA_OUT_F32 = 1
FMHA_OUT_NVFP4 = 2
FMHA_WIDE_AUTO = 0
FMHA_WIDE_INDEPENDENT = 1
FMHA_WIDE_PAIR = 2

_lock = threading.Lock()
_lib = None


class FmhaError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"[{code}] {msg}")
        self.code = code


class fmha_opts(ctypes.Structure):
    _fields_ = [
        ("out_kind", ctypes.c_int),
        ("seqlens_k", ctypes.c_void_p),
        ("num_splits", ctypes.c_int),
        ("workspace", ctypes.c_void_p),
        ("workspace_bytes", ctypes.c_size_t),
        ("out_scales", ctypes.c_void_p),
        ("out_tensor_scale", ctypes.c_void_p),
        ("out_f32", ctypes.c_void_p),
        ("causal", ctypes.c_int),
        ("nvfp4_scale_in", ctypes.c_void_p),
        ("out_amax", ctypes.c_void_p),
        ("wide_variant", ctypes.c_int),
    ]


class fmha_kv_cache(ctypes.Structure):
    _fields_ = [
        ("k", ctypes.c_void_p),
        ("v", ctypes.c_void_p),
        ("num_pages", ctypes.c_int),
        ("page_size", ctypes.c_int),
        ("Hkv", ctypes.c_int),
        ("D", ctypes.c_int),
        ("page_stride", ctypes.c_int64),
        ("head_stride", ctypes.c_int64),
        ("token_stride", ctypes.c_int64),
    ]
    device = None   # index of the pools' CUDA device (make_kv_cache), compared with the other tensors' at every call


def header_functions() -> list[str]:
    """Names of the functions include/fmha.h declares."""
    txt = open(HEADER).read()
    txt = re.sub(r"/\*.*?\*/", "", txt, flags=re.S)
    return sorted(set(re.findall(r"\b(fmha_\w+|nvfp4_\w+)\s*\(", txt)) - {"fmha_fwd_ex_"})


def load(path: str | None = None):
    """Load libfmha.so (built by build.py / __graft_entry__.build()); raises if absent."""
    global _lib
    lib = _lib
    if lib is not None:
        return lib
    with _lock:
        if _lib is not None:
            return _lib
        p = path or LIB_PATH
        if not os.path.exists(p):
            raise FmhaError(FMHA_ERR_CUDA, f"{p} not built: run attention_tensor_cores_gb300/build.py")
        lib = ctypes.CDLL(p)
        V, I, I64, S, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
        sig = {
            "fmha_fwd": ([V, V, V, V, V, I, I, I, I, I, I, F, V], I),
            "fmha_fwd_ex": ([V, V, V, V, V, I, I, I, I, I, I, F, V, ctypes.POINTER(fmha_opts)], I),
            "fmha_workspace_size": ([I, I, I, I, I, I, ctypes.POINTER(fmha_opts)], S),
            "fmha_fwd_host": ([V, V, V, V, V, I, I, I, I, I, I, F, V, ctypes.POINTER(fmha_opts), V, S], I),
            "fmha_host_buffer_size": ([I, I, I, I, I, I, ctypes.POINTER(fmha_opts)], S),
            "nvfp4_quantize": ([V, V, V, I64, V], I),
            "nvfp4_quantize_scaled": ([V, V, V, I64, V, V], I),
            "nvfp4_scales_bytes": ([I64], S),
            "fmha_qk_gemm": ([V, V, V, I, I, I, V], I),
            "fmha_selftest": ([I, V, V, S, I, V], I),
            "fmha_check_status": ([V], I),
            "fmha_set_wait_limit": ([ctypes.c_longlong], None),
            "fmha_error_string": ([I], ctypes.c_char_p),
            "fmha_last_error": ([], ctypes.c_char_p),
            "fmha_num_sms": ([], I),
            "fmha_launch_count": ([], ctypes.c_longlong),
            "fmha_time_next_call": ([V, V], None),
            "fmha_page_table": ([V, V, I, I, V, V, I, V, I, V, V, V, V, I, V, V], I),
            "fmha_rope_append": ([V, I64, V, I64, V, I64, V, V, F, V, I, I, I, V, V, V, ctypes.POINTER(fmha_kv_cache), I, I, I, V], I),
            "fmha_fwd_paged": ([V, ctypes.POINTER(fmha_kv_cache), V, I, V, V, V, I, I, I, F, V, ctypes.POINTER(fmha_opts)], I),
            "fmha_paged_workspace_size": ([I, I, I, ctypes.POINTER(fmha_kv_cache), ctypes.POINTER(fmha_opts)], S),
            "fmha_fwd_prefix": ([V, ctypes.POINTER(fmha_kv_cache), V, I, V, V, V, I, V, V, I, I, I, F, V, ctypes.POINTER(fmha_opts)], I),
            "fmha_prefix_workspace_size": ([I, I, I, ctypes.POINTER(fmha_kv_cache), ctypes.POINTER(fmha_opts)], S),
            "fmha_page_fork": ([V, I, V, I, I, V, I, V, V, I, V, V, V, V, V, V, V], I),
            "fmha_page_copy": ([ctypes.POINTER(fmha_kv_cache), I, V, V, V, I, V, V], I),
            "fmha_page_compact": ([V, I, I, V, I, V, V, I, V, V, V, V, I, V, V, V], I),
            "fmha_fwd_decode_noalloc": ([V, V, V, V, V, I, I, I, I, I, I, F, V, V], I),
        }
        for name, (args, res) in sig.items():
            fn = getattr(lib, name, None)
            if fn is None:
                continue
            fn.argtypes = args
            fn.restype = res
        _lib = lib
        return lib


def _check(rc: int, what: str):
    if rc != FMHA_OK:
        lib = load()
        raise FmhaError(rc, f"{what}: {lib.fmha_last_error().decode()} ({lib.fmha_error_string(rc).decode()})")


def _stream(stream=None):
    """Raw cudaStream_t of `stream`, else of the current stream on the current device."""
    import torch
    if stream is not None:
        return stream.cuda_stream
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    if raw is not None:
        return raw(torch.cuda.current_device())
    return torch.cuda.current_stream().cuda_stream


def _ptr(t):
    return None if t is None else t.data_ptr()


def _need_cuda(*ts):
    for t in ts:
        if t is not None and not t.is_cuda:
            raise FmhaError(FMHA_ERR_INVALID, "tensors must be on a CUDA device")
        if t is not None and not t.is_contiguous():
            raise FmhaError(FMHA_ERR_INVALID, "tensors must be contiguous")


# ------------------------------------------------------------------------------------------------
# entry points (same names as the C ABI)
# ------------------------------------------------------------------------------------------------
def fmha_fwd(q, k, v, out, lse, scale: float, stream=None):
    """O = softmax(scale Q K^T) V with BF16 output; q [B,Hq,Sq,D], k/v [B,Hkv,Skv,D]."""
    _need_cuda(q, k, v, out, lse)
    B, Hq, Sq, D = q.shape
    Hkv, Skv = k.shape[1], k.shape[2]
    rc = load().fmha_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, Hq, Hkv, Sq, Skv, D,
                         float(scale), _stream(stream))
    _check(rc, "fmha_fwd")


def make_opts(out_kind=FMHA_OUT_BF16, seqlens_k=None, num_splits=0, workspace=None,
              out_scales=None, out_tensor_scale=None, out_f32=None, causal=False,
              nvfp4_scale_in=None, out_amax=None, wide_variant=FMHA_WIDE_AUTO) -> fmha_opts:
    """Options of a call; they keep the tensors they name alive."""
    o = fmha_opts()
    o.tensors = (seqlens_k, workspace, out_scales, out_tensor_scale, out_f32, nvfp4_scale_in, out_amax)
    o.wide_variant = wide_variant
    o.causal = 1 if causal else 0
    o.nvfp4_scale_in = None if nvfp4_scale_in is None else nvfp4_scale_in.data_ptr()
    o.out_amax = None if out_amax is None else out_amax.data_ptr()
    o.out_kind = out_kind
    o.seqlens_k = None if seqlens_k is None else seqlens_k.data_ptr()
    o.num_splits = num_splits
    o.workspace = None if workspace is None else workspace.data_ptr()
    o.workspace_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    o.out_scales = None if out_scales is None else out_scales.data_ptr()
    o.out_tensor_scale = None if out_tensor_scale is None else out_tensor_scale.data_ptr()
    o.out_f32 = None if out_f32 is None else out_f32.data_ptr()
    return o


def fmha_workspace_size(B, Hq, Hkv, Sq, Skv, D, opts: fmha_opts | None = None) -> int:
    return int(load().fmha_workspace_size(B, Hq, Hkv, Sq, Skv, D,
                                          None if opts is None else ctypes.byref(opts)))


def fmha_fwd_ex(q, k, v, out, lse, scale: float, opts: fmha_opts | None = None, stream=None):
    """Attention with options (see make_opts); tensors as in fmha_fwd, `out` per opts.out_kind."""
    _need_cuda(q, k, v, out, lse)
    B, Hq, Sq, D = q.shape
    Hkv, Skv = k.shape[1], k.shape[2]
    rc = load().fmha_fwd_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, Hq, Hkv, Sq, Skv, D,
                            float(scale), _stream(stream), None if opts is None else ctypes.byref(opts))
    _check(rc, "fmha_fwd_ex")


def fmha_host_buffer_size(B, Hq, Hkv, Sq, Skv, D, opts: fmha_opts | None = None) -> int:
    return int(load().fmha_host_buffer_size(B, Hq, Hkv, Sq, Skv, D, None if opts is None else ctypes.byref(opts)))


def fmha_fwd_host(q, k, v, out, lse, scale: float, dev_buf, opts: fmha_opts | None = None, stream=None):
    """Attention from host memory: q/k/v/out/lse are CPU tensors (page-locked for asynchronous copies,
    lse may be None), dev_buf a CUDA byte tensor of at least fmha_host_buffer_size() bytes.  Returns
    once enqueued on `stream`; synchronise before reading out / lse."""
    for t in (q, k, v, out, lse):
        if t is not None and (t.is_cuda or not t.is_contiguous()):
            raise FmhaError(FMHA_ERR_INVALID, "q/k/v/out/lse must be contiguous host tensors")
    _need_cuda(dev_buf)
    B, Hq, Sq, D = q.shape
    Hkv, Skv = k.shape[1], k.shape[2]
    rc = load().fmha_fwd_host(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, Hq, Hkv, Sq, Skv, D, float(scale),
                              _stream(stream), None if opts is None else ctypes.byref(opts), _ptr(dev_buf),
                              dev_buf.numel() * dev_buf.element_size())
    _check(rc, "fmha_fwd_host")


def nvfp4_scales_bytes(n: int) -> int:
    return int(load().nvfp4_scales_bytes(n))


def nvfp4_quantize(x, q, scales, stream=None):
    """x: FP32 [n] (n % 16 == 0), q: uint8 [n/2], scales: uint8 [nvfp4_scales_bytes(n)]."""
    _need_cuda(x, q, scales)
    rc = load().nvfp4_quantize(_ptr(x), _ptr(q), _ptr(scales), x.numel(), _stream(stream))
    _check(rc, "nvfp4_quantize")


def nvfp4_quantize_scaled(x, q, scales, tensor_scale, stream=None):
    """x: FP32 [n] (n % 16 == 0), q: uint8 [n/2], scales: uint8 [n/16], tensor_scale: FP32 [1] (s_g)."""
    _need_cuda(x, q, scales, tensor_scale)
    rc = load().nvfp4_quantize_scaled(_ptr(x), _ptr(q), _ptr(scales), x.numel(), _ptr(tensor_scale), _stream(stream))
    _check(rc, "nvfp4_quantize_scaled")


def fmha_qk_gemm(q, k, s, stream=None):
    """Raw S = Q K^T (FP32, no scale); q [Sq,D], k [Skv,D] BF16, s [Sq,Skv] FP32."""
    _need_cuda(q, k, s)
    Sq, D = q.shape
    Skv = k.shape[0]
    rc = load().fmha_qk_gemm(_ptr(q), _ptr(k), _ptr(s), Sq, Skv, D, _stream(stream))
    _check(rc, "fmha_qk_gemm")


def fmha_selftest(which: int, inp, out, param: int = 0, stream=None):
    _need_cuda(inp, out)
    rc = load().fmha_selftest(which, _ptr(inp), _ptr(out), out.numel() * out.element_size(), param,
                              _stream(stream))
    _check(rc, f"fmha_selftest({which})")


def fmha_check_status(stream=None) -> int:
    return int(load().fmha_check_status(_stream(stream)))


def fmha_set_wait_limit(cycles: int):
    load().fmha_set_wait_limit(int(cycles))


def fmha_num_sms() -> int:
    return int(load().fmha_num_sms())


def fmha_launch_count() -> int:
    return int(load().fmha_launch_count())


def fmha_time_next_call(start_event, stop_event):
    """torch.cuda.Event pair (enable_timing=True, already recorded once so the handle exists)."""
    load().fmha_time_next_call(ctypes.c_void_p(start_event.cuda_event), ctypes.c_void_p(stop_event.cuda_event))


def fmha_fwd_decode_noalloc(q, k, v, out, lse, scale: float, seqlens_k=None, stream=None):
    """Split-KV decode whose scratch is the library's fixed device array (nothing is allocated)."""
    _need_cuda(q, k, v, out, lse, seqlens_k)
    B, Hq, Sq, D = q.shape
    Hkv, Skv = k.shape[1], k.shape[2]
    rc = load().fmha_fwd_decode_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, Hq, Hkv, Sq, Skv, D,
                                        float(scale), _ptr(seqlens_k), _stream(stream))
    _check(rc, "fmha_fwd_decode_noalloc")


# ------------------------------------------------------------------------------------------------
# paged key/value cache
# ------------------------------------------------------------------------------------------------
_ext = None


def _native():
    """The native binding of the functions below (built with libfmha.so); raises if absent."""
    global _ext
    if _ext is None:
        lib = load()
        import torch  # noqa: F401  (its libraries first)
        try:
            from . import _binding as ext
        except ImportError as e:
            raise FmhaError(FMHA_ERR_CUDA, f"_binding.so not built for this torch: run attention_tensor_cores_gb300/build.py ({e})")
        ext.bind(FmhaError, *(ctypes.cast(f, ctypes.c_void_p).value for f in (
            lib.fmha_page_table, lib.fmha_rope_append, lib.fmha_fwd_paged, lib.fmha_fwd_prefix, lib.fmha_page_fork, lib.fmha_page_copy,
            lib.fmha_page_compact, lib.fmha_last_error, lib.fmha_error_string)))
        _ext = ext
    return _ext


def _need(cond, what: str):
    if not cond:
        raise FmhaError(FMHA_ERR_INVALID, what)


def make_kv_cache(k, v) -> fmha_kv_cache:
    """Descriptor of a paged cache: k and v are BF16 CUDA tensors [pages, Hkv, page_size, D] of the same
    strides (the last 1; the others multiples of 8), e.g. a [pages, page_size, Hkv, D] pool permuted.
    It keeps k and v alive."""
    import torch
    _need(k.is_cuda and v.device == k.device and k.dtype == v.dtype == torch.bfloat16,
          "cache pools must be BF16 tensors on one CUDA device")
    _need(k.dim() == 4 and k.shape == v.shape, "cache pools must have one shape [pages, Hkv, page_size, D]")
    D = k.shape[3]

    def strides(t):   # of a dimension of size 1 nothing is read, and torch may say anything
        return [s if n > 1 else D for n, s in zip(t.shape[:3], t.stride()[:3])]
    _need(k.stride(3) == 1 and v.stride(3) == 1 and strides(k) == strides(v), "cache pools must have the same strides, the last 1")
    c = fmha_kv_cache()
    c.k, c.v = k.data_ptr(), v.data_ptr()
    c.num_pages, c.Hkv, c.page_size, c.D = k.shape
    c.page_stride, c.head_stride, c.token_stride = strides(k)
    c.pools, c.device = (k, v), k.get_device()
    return c


def fmha_page_table(ctx_lens, new_lens, page_size: int, free_pages, free_count, block_table, seqlens, cu_new, positions, slots,
                    free_count_out, stream=None):
    """Gives pages of the stack free_pages [num_pages] to requests whose tokens outgrow theirs, takes back
    those of requests with new_lens < 0, and writes block_table [B, max_pages], seqlens [B], cu_new [B + 1],
    positions [T], slots [T] and free_count_out [1]; slots is int64, all others int32."""
    (_ext or _native()).page_table(ctx_lens, new_lens, page_size, free_pages, free_count, block_table, seqlens, cu_new, positions,
                                    slots, free_count_out, stream)


def fmha_rope_append(q, k, v, q_weight, k_weight, eps: float, cos_sin, positions, slots, q_out, cache: fmha_kv_cache,
                     interleaved: bool = False, stream=None):
    """Norm (weights [D] or None), rotation (cos_sin FP32 [max_pos, rope_dim] or None) and store: q [T, Hq, D],
    k and v [T, Hkv, D] may be slices of one projection; q_out [T / Sq, Hq, Sq, D] or [T, Hq, D]."""
    (_ext or _native()).rope_append(q, k, v, q_weight, k_weight, eps, cos_sin, positions, slots, q_out, cache, interleaved, stream)


def fmha_paged_workspace_size(B, Hq, Sq, cache: fmha_kv_cache, opts: fmha_opts | None = None) -> int:
    return int(load().fmha_paged_workspace_size(B, Hq, Sq, ctypes.byref(cache), None if opts is None else ctypes.byref(opts)))


def fmha_fwd_paged(q, cache: fmha_kv_cache, block_table, seqlens, out, lse, scale: float, opts: fmha_opts | None = None, stream=None):
    """Attention of q [B, Hq, Sq, D] over the first seqlens[b] tokens of each request's pages, block_table
    int32 [B, max_pages]; out per opts.out_kind, lse FP32 [B, Hq, Sq] or None (see make_opts, make_kv_cache)."""
    (_ext or _native()).fwd_paged(q, cache, block_table, seqlens, out, lse, scale, opts, stream)


# ------------------------------------------------------------------------------------------------
# pages that requests share
# ------------------------------------------------------------------------------------------------
def fmha_prefix_workspace_size(B, Hq, Sq, cache: fmha_kv_cache, opts: fmha_opts | None = None) -> int:
    return int(load().fmha_prefix_workspace_size(B, Hq, Sq, ctypes.byref(cache), None if opts is None else ctypes.byref(opts)))


def fmha_fwd_prefix(q, cache: fmha_kv_cache, block_table, seqlens, cu_groups, prefix_lens, out, lse, scale: float,
                    opts: fmha_opts | None = None, stream=None):
    """fmha_fwd_paged for groups of requests, cu_groups int32 [N + 1], whose first prefix_lens [N] tokens are in the same
    pages: those are read once for the group.  opts needs a workspace of fmha_prefix_workspace_size bytes."""
    (_ext or _native()).fwd_prefix(q, cache, block_table, seqlens, cu_groups, prefix_lens, out, lse, scale, opts, stream)


def fmha_page_fork(parents, ctx_lens, page_size: int, block_table, free_pages, free_count, new_table, seqlens, copy_src, copy_dst,
                   copy_tokens, free_count_out, stream=None):
    """The requests parents [B] (negative: an empty slot) of this step's ctx_lens [B_old], block_table [B_old, max_pages] as the next
    step's: new_table [B, max_pages], seqlens [B], the pages to be copied (copy_src, copy_dst, copy_tokens [B]) and the stack of
    free pages; all int32."""
    (_ext or _native()).page_fork(parents, ctx_lens, page_size, block_table, free_pages, free_count, new_table, seqlens, copy_src,
                                  copy_dst, copy_tokens, free_count_out, stream)


def fmha_page_copy(caches, src, dst, tokens=None, count=None, stream=None):
    """Copies the first tokens[i] tokens (None: all) of page src[i] to page dst[i], int32 [n], in each of the caches (a list: a
    model's layers); only the first count [1] pairs if given."""
    (_ext or _native()).page_copy(caches, src, dst, tokens, count, stream)


def fmha_page_compact(seqlens, page_size: int, block_table, free_pages, free_count, new_ids, new_table, copy_src, copy_dst, copy_count,
                      free_pages_out, stream=None):
    """Used pages to the low ids: new_ids [num_pages], new_table [B, max_pages], the moves (copy_src, copy_dst of at least num_pages / 2
    entries, copy_count [1]) and free_pages_out [num_pages]; all int32."""
    (_ext or _native()).page_compact(seqlens, page_size, block_table, free_pages, free_count, new_ids, new_table, copy_src, copy_dst,
                                     copy_count, free_pages_out, stream)
