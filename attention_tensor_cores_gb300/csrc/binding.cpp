// Python entry points of the paged key/value cache: checks of the tensors and the call of libfmha.so, in one
// native call.  A decoding step makes two of these calls per layer on kernels of a few microseconds, which
// marshalling through ctypes (10 to 14 us a call) would outlast; this takes about 1 us plus the launch.
//
// The functions take the arguments of the Python functions of the same names and raise FmhaError.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <exception>
#include <vector>

#include "../../include/fmha.h"

namespace {

// libfmha.so's functions (addresses from the package, which has loaded it) and the package's exception
struct Library {
    decltype(&fmha_page_table) page_table;
    decltype(&fmha_rope_append) rope_append;
    decltype(&fmha_fwd_paged) fwd_paged;
    decltype(&fmha_fwd_prefix) fwd_prefix;
    decltype(&fmha_page_fork) page_fork;
    decltype(&fmha_page_copy) page_copy;
    decltype(&fmha_page_compact) page_compact;
    decltype(&fmha_last_error) last_error;
    decltype(&fmha_error_string) error_string;
    PyObject* error;
} lib;

struct Refused {
    int code;
    const char* what;
};

void need(bool ok, const char* what)
{
    if (!ok) throw Refused{FMHA_ERR_INVALID, what};
}

void raise(int code, PyObject* text)
{
    if (text) {
        if (PyObject* e = PyObject_CallFunction(lib.error, "iO", code, text)) {
            PyErr_SetObject(lib.error, e);
            Py_DECREF(e);
        }
        Py_DECREF(text);
    }
}

PyObject* result(int rc, const char* name)
{
    if (rc == FMHA_OK) Py_RETURN_NONE;
    raise(rc, PyUnicode_FromFormat("%s: %s (%s)", name, lib.last_error(), lib.error_string(rc)));
    return nullptr;
}

const at::Tensor& tensor(PyObject* o, const char* what)
{
    need(THPVariable_Check(o), what);
    return THPVariable_Unpack(o);
}

int device_of(const at::Tensor& t)
{
    need(t.is_cuda() && t.get_device() == c10::cuda::current_device(), "tensors must be on the current CUDA device");
    return t.get_device();
}

// A contiguous tensor of this type on the device; what: the message otherwise
const at::Tensor& plain(PyObject* o, int device, at::ScalarType type, const char* what)
{
    const at::Tensor& t = tensor(o, what);
    need(t.scalar_type() == type && t.is_cuda() && t.get_device() == device && t.is_contiguous(), what);
    return t;
}

template <typename T>
T* data(const at::Tensor& t)
{
    return static_cast<T*>(t.data_ptr());
}

fmha_stream_t stream_of(PyObject* o, int device)
{
    if (o == Py_None) return reinterpret_cast<fmha_stream_t>(c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream());
    PyObject* raw = PyObject_GetAttrString(o, "cuda_stream");
    if (!raw) throw std::exception();
    void* s = PyLong_AsVoidPtr(raw);
    Py_DECREF(raw);
    if (PyErr_Occurred()) throw std::exception();
    return static_cast<fmha_stream_t>(s);
}

int integer(PyObject* o, const char* what)
{
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        need(false, what);
    }
    need(v >= INT32_MIN && v <= INT32_MAX, what);
    return static_cast<int>(v);
}

float number(PyObject* o)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw std::exception();
    return static_cast<float>(v);
}

// The C structure inside a ctypes Structure of the package
template <typename T>
T structure(PyObject* o, const char* what)
{
    Py_buffer b;
    if (PyObject_GetBuffer(o, &b, PyBUF_SIMPLE) != 0) {
        PyErr_Clear();
        need(false, what);
    }
    const bool fits = b.len == static_cast<Py_ssize_t>(sizeof(T));
    T v{};
    if (fits) memcpy(&v, b.buf, sizeof(T));
    PyBuffer_Release(&b);
    need(fits, what);
    return v;
}

// The cache's descriptor.  Its pools are bare pointers, so the device that make_kv_cache saw them on goes along as an
// attribute; a descriptor filled by hand has None there and is taken at its word.
fmha_kv_cache cache_of(PyObject* o, int device)
{
    const fmha_kv_cache c = structure<fmha_kv_cache>(o, "cache must be a fmha_kv_cache (make_kv_cache)");
    static PyObject* const name = PyUnicode_InternFromString("device");
    PyObject* at = PyObject_GetAttr(o, name);
    if (!at) PyErr_Clear();
    const bool here = !at || at == Py_None || PyLong_AsLong(at) == device;
    if (PyErr_Occurred()) PyErr_Clear();
    Py_XDECREF(at);
    need(here, "the cache's pools must be on the device of the other tensors");
    return c;
}

template <typename F>
PyObject* guarded(F&& body)
{
    try {
        return body();
    } catch (const Refused& r) {
        raise(r.code, PyUnicode_FromString(r.what));
    } catch (const std::exception& e) {
        if (!PyErr_Occurred()) raise(FMHA_ERR_INVALID, PyUnicode_FromString(e.what()));
    }
    return nullptr;
}

template <typename F>
int unlocked(F&& call)
{
    int rc;
    Py_BEGIN_ALLOW_THREADS;
    rc = call();
    Py_END_ALLOW_THREADS;
    return rc;
}

bool counted(PyObject*, Py_ssize_t n, Py_ssize_t want)
{
    if (n == want) return true;
    PyErr_Format(PyExc_TypeError, "%zd arguments expected, %zd given", want, n);
    return false;
}

// ctx_lens, new_lens, page_size, free_pages, free_count, block_table, seqlens, cu_new, positions, slots, free_count_out, stream
PyObject* page_table(PyObject* self, PyObject* const* a, Py_ssize_t n)
{
    if (!counted(self, n, 12)) return nullptr;
    return guarded([&] {
        constexpr auto i32 = at::kInt;
        const char* types = "slots must be int64, all other tensors int32, contiguous and on one CUDA device";
        const at::Tensor& free_pages = tensor(a[3], types);
        const int dev = device_of(free_pages);
        plain(a[3], dev, i32, types);
        const at::Tensor &ctx = plain(a[0], dev, i32, types), &add = plain(a[1], dev, i32, types), &count = plain(a[4], dev, i32, types),
                         &table = plain(a[5], dev, i32, types), &lens = plain(a[6], dev, i32, types), &cu = plain(a[7], dev, i32, types),
                         &pos = plain(a[8], dev, i32, types), &slots = plain(a[9], dev, at::kLong, types),
                         &out = plain(a[10], dev, i32, types);
        const int64_t B = ctx.numel(), T = slots.numel();
        need(add.numel() == B && lens.numel() == B && cu.numel() == B + 1 && pos.numel() == T && table.dim() == 2 && table.size(0) == B &&
                 count.numel() == 1 && out.numel() == 1,
             "need new_lens [B], seqlens [B], cu_new [B + 1], block_table [B, max_pages], positions [T], free counts [1]");
        need(B < INT32_MAX && T <= INT32_MAX && free_pages.numel() <= INT32_MAX && table.size(1) <= INT32_MAX, "sizes pass 2^31");
        const int page = integer(a[2], "page_size must be an integer");
        const fmha_stream_t st = stream_of(a[11], dev);
        return result(unlocked([&] {
                          return lib.page_table(data<int32_t>(ctx), data<int32_t>(add), static_cast<int>(B), page, data<int32_t>(free_pages),
                                                data<int32_t>(count), static_cast<int>(free_pages.numel()), data<int32_t>(table),
                                                static_cast<int>(table.size(1)), data<int32_t>(lens), data<int32_t>(cu), data<int32_t>(pos),
                                                data<int64_t>(slots), static_cast<int>(T), data<int32_t>(out), st);
                      }),
                      "fmha_page_table");
    });
}

// q, k, v, q_weight, k_weight, eps, cos_sin, positions, slots, q_out, cache, interleaved, stream
PyObject* rope_append(PyObject* self, PyObject* const* a, Py_ssize_t n)
{
    if (!counted(self, n, 13)) return nullptr;
    return guarded([&] {
        constexpr auto bf16 = at::kBFloat16;
        const at::Tensor& slots = tensor(a[8], "slots must be an int64 tensor");
        const int dev = device_of(slots);
        plain(a[8], dev, at::kLong, "slots must be a contiguous int64 tensor");
        const fmha_kv_cache cache = cache_of(a[10], dev);
        const char* shapes = "q must be BF16 [T, Hq, D], k and v [T, Hkv, D], with contiguous heads, on the device of slots";
        const at::Tensor &q = tensor(a[0], shapes), &k = tensor(a[1], shapes), &v = tensor(a[2], shapes);
        need(q.dim() == 3, shapes);
        const int64_t T = q.size(0), Hq = q.size(1), D = cache.D;
        const at::Tensor* three[3] = {&q, &k, &v};
        for (int i = 0; i < 3; ++i) {
            const at::Tensor& t = *three[i];
            const int64_t H = i ? cache.Hkv : Hq;
            need(t.scalar_type() == bf16 && t.is_cuda() && t.get_device() == dev && t.dim() == 3 && t.size(0) == T && t.size(1) == H &&
                     t.size(2) == D && (t.numel() == 0 || (t.stride(2) == 1 && (H == 1 || t.stride(1) == D))),
                 shapes);
        }
        const void* w[2] = {nullptr, nullptr};
        for (int i = 0; i < 2; ++i)
            if (a[3 + i] != Py_None) {
                const at::Tensor& t = plain(a[3 + i], dev, bf16, "weights must be contiguous BF16 tensors or None");
                need(t.numel() == D, "weights must have D values");
                w[i] = t.data_ptr();
            }
        const at::Tensor& out = plain(a[9], dev, bf16, "q_out must be a contiguous BF16 tensor");
        const int64_t Sq = out.dim() == 4 ? out.size(2) : 1;
        need(slots.numel() == T && out.numel() == T * Hq * D && (out.dim() == 3 || out.dim() == 4) && out.size(1) == Hq &&
                 out.size(out.dim() - 1) == D,
             "need slots [T] and q_out [T / Sq, Hq, Sq, D] or [T, Hq, D]");
        const float* cos_sin = nullptr;
        const int32_t* positions = nullptr;
        int64_t max_pos = 0, R = 0;
        if (a[6] != Py_None) {
            const at::Tensor &c = plain(a[6], dev, at::kFloat, "cos_sin must be a contiguous FP32 tensor or None"),
                             &p = plain(a[7], dev, at::kInt, "positions must be a contiguous int32 tensor");
            need(c.dim() == 2 && p.numel() == T, "need cos_sin [max_pos, rope_dim] and positions [T]");
            cos_sin = data<float>(c);
            positions = data<int32_t>(p);
            max_pos = c.size(0);
            R = c.size(1);
        }
        need(T <= INT32_MAX && Hq <= INT32_MAX && Sq <= INT32_MAX && max_pos <= INT32_MAX && R <= INT32_MAX, "sizes pass 2^31");
        const float eps = number(a[5]);
        const int pairs = PyObject_IsTrue(a[11]);
        if (pairs < 0) throw std::exception();
        const auto step = [T](const at::Tensor& t) { return T > 1 ? t.stride(0) : 0; };   // of one token, torch may say anything
        const fmha_stream_t st = stream_of(a[12], dev);
        return result(unlocked([&] {
                          return lib.rope_append(q.data_ptr(), step(q), k.data_ptr(), step(k), v.data_ptr(), step(v), w[0], w[1], eps,
                                                 cos_sin, static_cast<int>(max_pos), static_cast<int>(R), pairs, positions,
                                                 data<int64_t>(slots), out.data_ptr(), &cache, static_cast<int>(T), static_cast<int>(Hq),
                                                 static_cast<int>(Sq), st);
                      }),
                      "fmha_rope_append");
    });
}

// What the two attentions over pages have in common
struct Attention {
    const at::Tensor *q, *table, *lens, *out;
    int dev;
    fmha_kv_cache cache;
    fmha_opts opts{};
    bool has_opts;
    float* lse = nullptr;

    Attention(PyObject* q_, PyObject* cache_, PyObject* table_, PyObject* lens_, PyObject* out_, PyObject* lse_, PyObject* opts_)
        : q(&tensor(q_, "q must be a tensor")), dev(device_of(*q)), cache((plain(q_, dev, at::kBFloat16, "q must be a contiguous BF16 tensor"), cache_of(cache_, dev))),
          has_opts(opts_ != Py_None)
    {
        if (has_opts) opts = structure<fmha_opts>(opts_, "opts must be a fmha_opts (make_opts) or None");
        table = &plain(table_, dev, at::kInt, "block_table must be a contiguous int32 tensor on q's device");
        lens = &plain(lens_, dev, at::kInt, "seqlens must be a contiguous int32 tensor on q's device");
        need(q->dim() == 4 && q->size(3) == cache.D && table->dim() == 2 && table->size(0) == q->size(0) && lens->numel() == q->size(0),
             "need q [B, Hq, Sq, D] with the cache's D, block_table [B, max_pages] and seqlens [B]");
        const bool nvfp4 = opts.out_kind == FMHA_OUT_NVFP4;
        out = &plain(out_, dev, nvfp4 ? at::kByte : opts.out_kind == FMHA_OUT_F32 ? at::kFloat : at::kBFloat16,
                     "out must be contiguous, on q's device and BF16, FP32 or uint8 as opts.out_kind says");
        need(out->numel() * (nvfp4 ? 2 : 1) == q->numel(), "out must have q's size (NVFP4: a byte for two values)");
        if (lse_ != Py_None) {
            const at::Tensor& t = plain(lse_, dev, at::kFloat, "lse must be a contiguous FP32 tensor on q's device or None");
            need(t.numel() * cache.D == q->numel(), "lse must be [B, Hq, Sq]");
            lse = data<float>(t);
        }
        need(q->size(0) <= INT32_MAX && q->size(1) <= INT32_MAX && q->size(2) <= INT32_MAX && table->size(1) <= INT32_MAX, "sizes pass 2^31");
    }
    int size(int i) const { return static_cast<int>(q->size(i)); }
};

// q, cache, block_table, seqlens, out, lse, scale, opts, stream
PyObject* fwd_paged(PyObject* self, PyObject* const* a, Py_ssize_t n)
{
    if (!counted(self, n, 9)) return nullptr;
    return guarded([&] {
        const Attention x(a[0], a[1], a[2], a[3], a[4], a[5], a[7]);
        const float scale = number(a[6]);
        const fmha_stream_t st = stream_of(a[8], x.dev);
        return result(unlocked([&] {
                          return lib.fwd_paged(x.q->data_ptr(), &x.cache, data<int32_t>(*x.table), static_cast<int>(x.table->size(1)),
                                               data<int32_t>(*x.lens), x.out->data_ptr(), x.lse, x.size(0), x.size(1), x.size(2), scale, st,
                                               x.has_opts ? &x.opts : nullptr);
                      }),
                      "fmha_fwd_paged");
    });
}

// q, cache, block_table, seqlens, cu_groups, prefix_lens, out, lse, scale, opts, stream
PyObject* fwd_prefix(PyObject* self, PyObject* const* a, Py_ssize_t n)
{
    if (!counted(self, n, 11)) return nullptr;
    return guarded([&] {
        const Attention x(a[0], a[1], a[2], a[3], a[6], a[7], a[9]);
        const char* types = "cu_groups and prefix_lens must be contiguous int32 tensors on q's device";
        const at::Tensor &cu = plain(a[4], x.dev, at::kInt, types), &prefix = plain(a[5], x.dev, at::kInt, types);
        need(cu.numel() == prefix.numel() + 1 && cu.numel() <= INT32_MAX, "need cu_groups [N + 1] and prefix_lens [N]");
        const float scale = number(a[8]);
        const fmha_stream_t st = stream_of(a[10], x.dev);
        return result(unlocked([&] {
                          return lib.fwd_prefix(x.q->data_ptr(), &x.cache, data<int32_t>(*x.table), static_cast<int>(x.table->size(1)),
                                                data<int32_t>(*x.lens), data<int32_t>(cu), data<int32_t>(prefix), static_cast<int>(prefix.numel()),
                                                x.out->data_ptr(), x.lse, x.size(0), x.size(1), x.size(2), scale, st,
                                                x.has_opts ? &x.opts : nullptr);
                      }),
                      "fmha_fwd_prefix");
    });
}

// parents, ctx_lens, page_size, block_table, free_pages, free_count, new_table, seqlens, copy_src, copy_dst, copy_tokens, free_count_out, stream
PyObject* page_fork(PyObject* self, PyObject* const* a, Py_ssize_t n)
{
    if (!counted(self, n, 13)) return nullptr;
    return guarded([&] {
        const char* types = "all tensors must be int32, contiguous and on one CUDA device";
        const int dev = device_of(tensor(a[4], types));
        const auto i32 = [&](int i) -> const at::Tensor& { return plain(a[i], dev, at::kInt, types); };
        const at::Tensor &parents = i32(0), &ctx = i32(1), &table = i32(3), &free_pages = i32(4), &count = i32(5), &new_table = i32(6),
                         &lens = i32(7), &src = i32(8), &dst = i32(9), &tokens = i32(10), &out = i32(11);
        const int64_t B = parents.numel(), Bo = ctx.numel();
        need(table.dim() == 2 && table.size(0) == Bo && new_table.dim() == 2 && new_table.size(0) == B && new_table.size(1) == table.size(1) &&
                 lens.numel() == B && src.numel() == B && dst.numel() == B && tokens.numel() == B && count.numel() == 1 && out.numel() == 1,
             "need block_table [B_old, max_pages], new_table [B, max_pages], seqlens, copy_src, copy_dst and copy_tokens [B], free counts [1]");
        need(B <= INT32_MAX && Bo <= INT32_MAX && free_pages.numel() <= INT32_MAX && table.size(1) <= INT32_MAX, "sizes pass 2^31");
        const int page = integer(a[2], "page_size must be an integer");
        const fmha_stream_t st = stream_of(a[12], dev);
        return result(unlocked([&] {
                          return lib.page_fork(data<int32_t>(parents), static_cast<int>(B), data<int32_t>(ctx), static_cast<int>(Bo), page,
                                               data<int32_t>(table), static_cast<int>(table.size(1)), data<int32_t>(free_pages),
                                               data<int32_t>(count), static_cast<int>(free_pages.numel()), data<int32_t>(new_table),
                                               data<int32_t>(lens), data<int32_t>(src), data<int32_t>(dst), data<int32_t>(tokens),
                                               data<int32_t>(out), st);
                      }),
                      "fmha_page_fork");
    });
}

// caches (a list), src, dst, tokens, count, stream
PyObject* page_copy(PyObject* self, PyObject* const* a, Py_ssize_t n)
{
    if (!counted(self, n, 6)) return nullptr;
    return guarded([&] {
        const char* types = "src, dst, tokens and count must be contiguous int32 tensors on one CUDA device";
        const int dev = device_of(tensor(a[1], types));
        const at::Tensor &src = plain(a[1], dev, at::kInt, types), &dst = plain(a[2], dev, at::kInt, types);
        const int64_t pairs = src.numel();
        need(dst.numel() == pairs && pairs <= INT32_MAX, "need src and dst of one size");
        const int32_t *tokens = nullptr, *count = nullptr;
        if (a[3] != Py_None) {
            const at::Tensor& t = plain(a[3], dev, at::kInt, types);
            need(t.numel() == pairs, "need a number of tokens for each pair");
            tokens = data<int32_t>(t);
        }
        if (a[4] != Py_None) {
            const at::Tensor& t = plain(a[4], dev, at::kInt, types);
            need(t.numel() == 1, "need count [1]");
            count = data<int32_t>(t);
        }
        const char* list = "caches must be a list or tuple of fmha_kv_cache (make_kv_cache)";
        need(PyList_Check(a[0]) || PyTuple_Check(a[0]), list);
        std::vector<fmha_kv_cache> caches;
        const Py_ssize_t m = PySequence_Fast_GET_SIZE(a[0]);
        need(m <= INT32_MAX, list);
        caches.reserve(static_cast<size_t>(m));
        for (Py_ssize_t i = 0; i < m; ++i) caches.push_back(cache_of(PySequence_Fast_GET_ITEM(a[0], i), dev));
        const fmha_stream_t st = stream_of(a[5], dev);
        return result(unlocked([&] {
                          return lib.page_copy(caches.data(), static_cast<int>(m), data<int32_t>(src), data<int32_t>(dst), tokens,
                                               static_cast<int>(pairs), count, st);
                      }),
                      "fmha_page_copy");
    });
}

// seqlens, page_size, block_table, free_pages, free_count, new_ids, new_table, copy_src, copy_dst, copy_count, free_pages_out, stream
PyObject* page_compact(PyObject* self, PyObject* const* a, Py_ssize_t n)
{
    if (!counted(self, n, 12)) return nullptr;
    return guarded([&] {
        const char* types = "all tensors must be int32, contiguous and on one CUDA device";
        const int dev = device_of(tensor(a[3], types));
        const auto i32 = [&](int i) -> const at::Tensor& { return plain(a[i], dev, at::kInt, types); };
        const at::Tensor &lens = i32(0), &table = i32(2), &free_pages = i32(3), &count = i32(4), &ids = i32(5), &new_table = i32(6), &src = i32(7),
                         &dst = i32(8), &moves = i32(9), &out = i32(10);
        const int64_t B = lens.numel(), N = free_pages.numel();
        need(table.dim() == 2 && table.size(0) == B && new_table.dim() == 2 && new_table.size(0) == B && new_table.size(1) == table.size(1) &&
                 ids.numel() == N && out.numel() == N && src.numel() == dst.numel() && count.numel() == 1 && moves.numel() == 1,
             "need block_table and new_table [B, max_pages], new_ids and free_pages_out [num_pages], copy_src and copy_dst of one size, counts [1]");
        need(B <= INT32_MAX && N <= INT32_MAX && table.size(1) <= INT32_MAX && src.numel() <= INT32_MAX, "sizes pass 2^31");
        const int page = integer(a[1], "page_size must be an integer");
        const fmha_stream_t st = stream_of(a[11], dev);
        return result(unlocked([&] {
                          return lib.page_compact(data<int32_t>(lens), static_cast<int>(B), page, data<int32_t>(table), static_cast<int>(table.size(1)),
                                                  data<int32_t>(free_pages), data<int32_t>(count), static_cast<int>(N), data<int32_t>(ids),
                                                  data<int32_t>(new_table), data<int32_t>(src), data<int32_t>(dst), static_cast<int>(src.numel()),
                                                  data<int32_t>(moves), data<int32_t>(out), st);
                      }),
                      "fmha_page_compact");
    });
}

// bind(error class, addresses of page_table, rope_append, fwd_paged, fwd_prefix, page_fork, page_copy, page_compact, last_error, error_string)
PyObject* bind(PyObject* self, PyObject* const* a, Py_ssize_t n)
{
    if (!counted(self, n, 10)) return nullptr;
    void* f[9];
    for (int i = 0; i < 9; ++i) {
        f[i] = PyLong_AsVoidPtr(a[i + 1]);
        if (PyErr_Occurred()) return nullptr;
    }
    Py_INCREF(a[0]);
    lib = {reinterpret_cast<decltype(lib.page_table)>(f[0]), reinterpret_cast<decltype(lib.rope_append)>(f[1]),
           reinterpret_cast<decltype(lib.fwd_paged)>(f[2]), reinterpret_cast<decltype(lib.fwd_prefix)>(f[3]),
           reinterpret_cast<decltype(lib.page_fork)>(f[4]), reinterpret_cast<decltype(lib.page_copy)>(f[5]),
           reinterpret_cast<decltype(lib.page_compact)>(f[6]), reinterpret_cast<decltype(lib.last_error)>(f[7]),
           reinterpret_cast<decltype(lib.error_string)>(f[8]), a[0]};
    Py_RETURN_NONE;
}

#define METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(bind), METHOD(page_table), METHOD(rope_append), METHOD(fwd_paged), METHOD(fwd_prefix), METHOD(page_fork),
                         METHOD(page_copy), METHOD(page_compact), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
