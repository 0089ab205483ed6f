// binding.cpp -- the paged cache's calls for Python: checks the tensors,
// takes their addresses, sizes and strides, and calls the C entry point of the
// same name (include/think.h) with the tensors' device current.
//
// A decode step makes these calls with a few microseconds of work on the GPU
// each, so that the host's share counts: marshalling a dozen tensors through
// ctypes takes 13 to 21 us a call, this module a few.  The entry points come as addresses
// from the library that the package has loaded (bind), so that release and
// debug builds are both served.
#include <Python.h>

#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <string>

#include "think.h"

namespace {

decltype(&think_extend_pages) f_extend;
decltype(&think_norm_rope_append) f_rope;
decltype(&think_paged_attn) f_attn;
decltype(&think_gather_pages) f_gather;

// A refusal: becomes a ThinkError with THINK_ERR_INVALID_ARG.
struct Refused {
    std::string why;
};

[[noreturn]] void refuse(const char *why) { throw Refused{why}; }

// The arguments of one call, and the device that all its tensors share.
struct Args {
    PyObject *const *a;
    Py_ssize_t n;
    int device = -1;

    const at::Tensor &tensor(int i)
    {
        if (!THPVariable_Check(a[i])) refuse("expected a tensor");
        const at::Tensor &t = THPVariable_Unpack(a[i]);
        if (!t.is_cuda()) refuse("every tensor must lie on one GPU");
        const int d = t.get_device();
        if (device >= 0 && d != device) refuse("every tensor must lie on one GPU");
        device = d;
        return t;
    }
    bool none(int i) const { return a[i] == Py_None; }
    int64_t integer(int i) const
    {
        const long long v = PyLong_AsLongLong(a[i]);
        if (v == -1 && PyErr_Occurred()) {
            PyErr_Clear();
            refuse("expected an integer");
        }
        return v;
    }
    int int32(int i) const
    {
        const int64_t v = integer(i);
        if (v < INT32_MIN || v > INT32_MAX) refuse("an integer is out of range");
        return (int)v;
    }
    double number(int i) const
    {
        const double v = PyFloat_AsDouble(a[i]);
        if (v == -1.0 && PyErr_Occurred()) {
            PyErr_Clear();
            refuse("expected a number");
        }
        return v;
    }
    bool truth(int i) const
    {
        const int v = PyObject_IsTrue(a[i]);
        if (v < 0) {
            PyErr_Clear();
            refuse("expected a truth value");
        }
        return v != 0;
    }
    // the stream: an object with a cuda_stream, or None for the device's current one
    void *stream(int i) const
    {
        if (a[i] == Py_None) return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream();
        PyObject *s = PyObject_GetAttrString(a[i], "cuda_stream");
        if (!s) {
            PyErr_Clear();
            refuse("expected a stream");
        }
        void *p = PyLong_AsVoidPtr(s);
        Py_DECREF(s);
        if (!p && PyErr_Occurred()) {
            PyErr_Clear();
            refuse("expected a stream");
        }
        return p;
    }
};

think_dtype_t dtype_of(const at::Tensor &t)
{
    if (t.scalar_type() == at::kBFloat16) return THINK_BF16;
    if (t.scalar_type() == at::kFloat) return THINK_F32;
    refuse("dtypes are bfloat16 and float32");
}

int size32(const at::Tensor &t, int i)
{
    if (t.size(i) > INT32_MAX) refuse("a tensor is too large");
    return (int)t.size(i);
}

// a contiguous vector of n elements
template <typename P = int32_t>
P *vector(const at::Tensor &t, at::ScalarType dt, int64_t n, const char *why)
{
    if (t.scalar_type() != dt || t.dim() != 1 || t.size(0) != n || (n > 1 && t.stride(0) != 1)) refuse(why);
    return static_cast<P *>(t.data_ptr());
}

// [T,H,d] rows with contiguous channels: strides of the token and the head
struct Rows {
    int64_t s[2];
    explicit Rows(const at::Tensor &t)
    {
        if (t.dim() != 3 || (t.size(2) > 1 && t.stride(2) != 1)) refuse("expected a [T,H,d] tensor with contiguous channels");
        s[0] = t.stride(0), s[1] = t.stride(1);
    }
};

// [pages,Hkv,page_size,d] pool: strides of the page, the head and the row
struct Pool {
    int64_t s[3];
    explicit Pool(const at::Tensor &t)
    {
        if (t.dim() != 4 || (t.size(3) > 1 && t.stride(3) != 1))
            refuse("expected a [pages,Hkv,page_size,d] tensor with contiguous channels");
        for (int i = 0; i < 3; ++i) s[i] = t.stride(i);
    }
};

// [B,max_blocks] block table: the distance of its rows
int64_t table_ld(const at::Tensor &t, int64_t B)
{
    if (t.scalar_type() != at::kInt || t.dim() != 2 || t.size(0) != B || (t.size(1) > 1 && t.stride(1) != 1))
        refuse("expected a [B,max_blocks] int32 block table with contiguous rows");
    return B > 1 ? t.stride(0) : std::max(t.stride(0), t.size(1));
}

size_t bytes_of(const at::Tensor &t)
{
    if (!t.is_contiguous()) refuse("the workspace must be contiguous");
    return (size_t)t.nbytes();
}

int extend_pages(Args &x)
{
    const at::Tensor &new_lens = x.tensor(0), &kv_lens = x.tensor(1), &table = x.tensor(2), &free_pages = x.tensor(3),
                     &free_count = x.tensor(4), &lens_out = x.tensor(6), &count_out = x.tensor(7), &q_start = x.tensor(8),
                     &positions = x.tensor(9), &slots = x.tensor(10), &ws = x.tensor(11);
    if (new_lens.dim() != 1 || positions.dim() != 1 || free_pages.dim() != 1) refuse("lengths, positions and pages are vectors");
    const int B = size32(new_lens, 0);
    const int64_t T = positions.size(0), F = free_pages.size(0);
    const char *why = "lengths, pages and positions are contiguous int32 vectors of B, B + 1, T or 1 elements, slots int64";
    const int32_t *nl = vector(new_lens, at::kInt, B, why), *kl = vector(kv_lens, at::kInt, B, why);
    const int32_t *fp = vector(free_pages, at::kInt, F, why), *fc = vector(free_count, at::kInt, 1, why);
    int32_t *lo = vector(lens_out, at::kInt, B, why), *co = vector(count_out, at::kInt, 1, why);
    int32_t *qs = vector(q_start, at::kInt, (int64_t)B + 1, why), *ps = vector(positions, at::kInt, T, why);
    int64_t *sl = vector<int64_t>(slots, at::kLong, T, why);
    const int64_t ld = table_ld(table, B);
    c10::cuda::OptionalCUDAGuard guard((c10::DeviceIndex)x.device);
    return f_extend(nl, kl, B, x.int32(5), static_cast<int32_t *>(table.data_ptr()), ld, size32(table, 1), fp, size32(free_pages, 0),
                    fc, T, lo, co, qs, ps, sl, ws.data_ptr(), bytes_of(ws), x.stream(12));
}

int norm_rope_append(Args &x)
{
    const at::Tensor &q = x.tensor(0), &k = x.tensor(1), &v = x.tensor(2), &positions = x.tensor(8), &slots = x.tensor(9),
                     &q_out = x.tensor(10), &k_cache = x.tensor(11), &v_cache = x.tensor(12);
    const Rows rq(q), rk(k), rv(v), ro(q_out);
    const Pool pk(k_cache), pv(v_cache);
    const int64_t T = q.size(0), d = q.size(2);
    const int Hq = size32(q, 1), Hkv = size32(k, 1);
    const think_dtype_t dt = dtype_of(q);
    for (const at::Tensor *t : {&k, &v, &q_out, &k_cache, &v_cache})
        if (t->scalar_type() != q.scalar_type()) refuse("q, k, v, q_out and the caches must be of one dtype");
    if (k.size(0) != T || k.size(2) != d || v.sizes() != k.sizes() || q_out.sizes() != q.sizes() || k_cache.size(1) != Hkv ||
        k_cache.size(3) != d || v_cache.sizes() != k_cache.sizes())
        refuse("shapes do not match");
    const char *why = "positions are a contiguous int32 vector of T elements, slots int64, weights [d] of q's dtype, inv_freq float64";
    const void *wq = x.none(3) ? nullptr : vector<void>(x.tensor(3), q.scalar_type(), d, why);
    const void *wk = x.none(4) ? nullptr : vector<void>(x.tensor(4), q.scalar_type(), d, why);
    const double *freq = nullptr;
    int rot = 0;
    if (!x.none(6)) {
        const at::Tensor &f = x.tensor(6);
        if (f.dim() != 1 || f.size(0) > d) refuse(why);
        freq = vector<double>(f, at::kDouble, f.size(0), why);
        rot = 2 * (int)f.size(0);
    }
    const int32_t *ps = vector(positions, at::kInt, T, why);
    const int64_t *sl = vector<int64_t>(slots, at::kLong, T, why);
    c10::cuda::OptionalCUDAGuard guard((c10::DeviceIndex)x.device);
    return f_rope(q.data_ptr(), rq.s, k.data_ptr(), rk.s, v.data_ptr(), rv.s, T, Hq, Hkv, (int)d, dt, wq, wk,
                  (float)x.number(5), freq, rot, x.truth(7), ps, sl, q_out.data_ptr(), ro.s, k_cache.data_ptr(),
                  pk.s, v_cache.data_ptr(), pv.s, size32(k_cache, 0), size32(k_cache, 2), x.stream(13));
}

int paged_attn(Args &x)
{
    const at::Tensor &q = x.tensor(0), &k = x.tensor(1), &v = x.tensor(2), &table = x.tensor(3), &q_start = x.tensor(4),
                     &kv_lens = x.tensor(5), &out = x.tensor(6), &ws = x.tensor(7);
    const Rows rq(q), ro(out);
    const Pool pk(k), pv(v);
    const int64_t T = q.size(0), d = q.size(2);
    const think_dtype_t dt = dtype_of(q);
    if (k.scalar_type() != q.scalar_type() || v.scalar_type() != q.scalar_type() || out.scalar_type() != q.scalar_type())
        refuse("q, the caches and out must be of one dtype");
    if (v.sizes() != k.sizes() || k.size(3) != d || out.sizes() != q.sizes()) refuse("shapes do not match");
    if (kv_lens.dim() != 1) refuse("kv_lens is a vector");
    const int B = size32(kv_lens, 0);
    const char *why = "kv_lens and q_start are contiguous int32 vectors of B and B + 1 elements";
    const int32_t *kl = vector(kv_lens, at::kInt, B, why), *qs = vector(q_start, at::kInt, (int64_t)B + 1, why);
    const int64_t ld = table_ld(table, B);
    // scale None: 1 / sqrt(d)
    const float scale = x.none(9) ? (float)(1.0 / std::sqrt((double)d)) : (float)x.number(9);
    c10::cuda::OptionalCUDAGuard guard((c10::DeviceIndex)x.device);
    return f_attn(q.data_ptr(), rq.s, k.data_ptr(), pk.s, v.data_ptr(), pv.s, size32(k, 0), size32(k, 2),
                  static_cast<const int32_t *>(table.data_ptr()), ld, size32(table, 1), qs, kl, B, T, x.int32(10), size32(q, 1),
                  size32(k, 1), (int)d, dt, scale, x.int32(8), out.data_ptr(), ro.s, ws.data_ptr(), bytes_of(ws), x.stream(11));
}

int gather_pages(Args &x)
{
    const at::Tensor &cache = x.tensor(0), &table = x.tensor(1), &kv_lens = x.tensor(2), &out = x.tensor(3);
    const Pool pc(cache);
    const think_dtype_t dt = dtype_of(cache);
    if (kv_lens.dim() != 1) refuse("kv_lens is a vector");
    const int B = size32(kv_lens, 0);
    if (out.scalar_type() != cache.scalar_type() || !out.is_contiguous() || out.dim() != 4 || out.size(0) != B ||
        out.size(1) != cache.size(1) || out.size(3) != cache.size(3))
        refuse("out must be a contiguous [B,Hkv,N,d] tensor of the cache's dtype");
    const int32_t *kl = vector(kv_lens, at::kInt, B, "kv_lens is a contiguous int32 vector");
    const int64_t ld = table_ld(table, B);
    c10::cuda::OptionalCUDAGuard guard((c10::DeviceIndex)x.device);
    return f_gather(cache.data_ptr(), pc.s, size32(cache, 0), size32(cache, 2), static_cast<const int32_t *>(table.data_ptr()), ld,
                    size32(table, 1), kl, B, size32(cache, 1), out.size(2), (int)cache.size(3), dt, out.data_ptr(), x.stream(4));
}

// Returns None, the status code of a call that the library refused, or the
// reason (str) of one that was refused here.  No C++ exception leaves it.
template <int (*F)(Args &), int N>
PyObject *entry(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", N, n);
        return nullptr;
    }
    try {
        Args x{a, n};
        const int rc = F(x);
        if (rc == THINK_OK) Py_RETURN_NONE;
        return PyLong_FromLong(rc);
    } catch (const Refused &r) {
        return PyUnicode_FromString(r.why.c_str());
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

// bind(extend_pages, norm_rope_append, paged_attn, gather_pages): the
// addresses of the library's entry points
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    void *p[4];
    for (int i = 0; i < 4; ++i) {
        p[i] = n == 4 ? PyLong_AsVoidPtr(a[i]) : nullptr;
        if (!p[i]) {
            PyErr_Clear();
            PyErr_SetString(PyExc_TypeError, "bind takes four addresses");
            return nullptr;
        }
    }
    f_extend = reinterpret_cast<decltype(f_extend)>(p[0]);
    f_rope = reinterpret_cast<decltype(f_rope)>(p[1]);
    f_attn = reinterpret_cast<decltype(f_attn)>(p[2]);
    f_gather = reinterpret_cast<decltype(f_gather)>(p[3]);
    Py_RETURN_NONE;
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f))
PyMethodDef methods[] = {
    {"bind", FAST(&bind), METH_FASTCALL, nullptr},
    {"extend_pages", FAST((&entry<extend_pages, 13>)), METH_FASTCALL, nullptr},
    {"norm_rope_append", FAST((&entry<norm_rope_append, 14>)), METH_FASTCALL, nullptr},
    {"paged_attn", FAST((&entry<paged_attn, 12>)), METH_FASTCALL, nullptr},
    {"gather_pages", FAST((&entry<gather_pages, 5>)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// The torch that this was built with: its C++ interface is not stable between
// versions.  (The build looks for the text, so as to build again for another one.)
const char kTorchVersion[] = "torch_version=" THINK_TORCH_VERSION;

PyMODINIT_FUNC PyInit__binding()
{
    PyObject *m = PyModule_Create(&module);
    if (m && PyModule_AddStringConstant(m, "torch_version", std::strchr(kTorchVersion, '=') + 1) < 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
