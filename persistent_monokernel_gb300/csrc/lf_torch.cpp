// lf_torch.cpp -- what the caches (KV4Cache, PagedKVCache, PageTables) do per
// call, for Python: torch tensors to lf_rows, their checks, the outputs' and the
// scratch's memory, the call.
//
// The kernels of a decode step take a few microseconds, and a launch 1.4.  In
// Python the same work (attributes of four tensors, three structures, an
// allocation, the foreign call) costs several times that, most of it in code
// that is cold again after every launch.
//
// A module of the C API: nothing here computes, and the library is reached
// through the addresses of its entry points (bind).
#include <Python.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/core/AutogradState.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/version.h>

#include <climits>
#include <memory>
#include <optional>
#include <sstream>
#include <string>

#include "../../include/lf.h"

namespace {

decltype(&lf_kv4_append) g_append;
decltype(&lf_kv4_read) g_read;
decltype(&lf_kv4_attend) g_attend;
decltype(&lf_kv4_workspace) g_workspace;
decltype(&lf_paged_plan) g_plan;
decltype(&lf_paged_append) g_paged_append;
decltype(&lf_paged_attend) g_paged_attend;
decltype(&lf_paged_workspace) g_paged_workspace;
PyObject *g_fail;   // raises the library's error: fail(status, entry point)

struct Refused : std::runtime_error {
    using std::runtime_error::runtime_error;
};

// These calls form no derivatives: what asks for some is refused, backward ones and forward ones (a tangent).
void no_derivatives(const at::Tensor &t, const char *what)
{
    if (t.requires_grad() && c10::GradMode::is_enabled())
        throw Refused(std::string(what) + " requires a gradient, and these calls form none: detach it, or call under torch.no_grad()");
    if (c10::AutogradState::get_tls_state().get_fw_grad_mode() && t._fw_grad(0).defined())
        throw Refused(std::string(what) + " has a tangent, and these calls form none: pass its primal, or call under torch.inference_mode()");
}

// A call writes t: its version says so to a backward pass that has kept it.  (Tensors made in inference mode have none.)
void written(const at::Tensor &t)
{
    if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}
void written(PyObject *o) { written(THPVariable_Unpack(o)); }

// A cache as the library has it, its tensors (k_codes, k_scales, v_codes, v_scales) and device, and the scratch that
// the last query that needed some did.
struct Cache {
    static constexpr const char *name = "lf_kv4";
    lf_kv4 c;
    at::Tensor parts[4];
    c10::DeviceIndex device;
    int n = -1, heads = -1;
    int64_t scratch = 0;

    // The tensors' addresses as they are now: resize_ or set_ may have moved them, or left something else.
    void locate()
    {
        void **const at[4] = {&c.k_codes, &c.k_scales, &c.v_codes, &c.v_scales};
        for (int i = 0; i < 4; ++i) {
            const at::Tensor &t = parts[i];
            const auto size = t.sizes();
            if (size.size() != 3 || size[0] != c.n_kv_heads || size[1] != c.max_seq || size[2] != c.head_dim / (i % 2 ? 16 : 2) ||
                !t.is_contiguous() || t.scalar_type() != at::kByte || t.get_device() != device)
                throw Refused("a tensor of the cache is no longer what the cache was made with");
            *at[i] = t.mutable_data_ptr();
        }
    }
};

// The pools of a paged cache, and the page tables of a batch.
struct Paged {
    static constexpr const char *name = "lf_paged";
    lf_paged c;
    at::Tensor k, v;
    c10::DeviceIndex device;

    static bool fits(const at::Tensor &t, const lf_paged &c, c10::DeviceIndex device)
    {
        const auto size = t.sizes();
        return t.layout() == at::kStrided && size.size() == 4 && size[0] == c.n_pages && size[1] == c.n_kv_heads &&
               size[2] == c.page && size[3] == c.head_dim && t.stride(3) == 1 && t.is_cuda() && t.get_device() == device &&
               t.scalar_type() == (c.dtype == LF_F16 ? at::kHalf : at::kBFloat16);
    }
    static bool alike(const at::Tensor &a, const at::Tensor &b)   // strides, but those of dimensions of one
    {
        for (int i = 0; i < 3; ++i)
            if (a.size(i) != 1 && a.stride(i) != b.stride(i)) return false;
        return true;
    }
    void locate()
    {
        if (!fits(k, c, device) || !fits(v, c, device) || !alike(k, v))
            throw Refused("a tensor of the cache is no longer what the cache was made with");
        no_derivatives(k, "k of the cache");
        no_derivatives(v, "v of the cache");
        place();
    }
    void place()
    {
        c.page_stride = k.stride(0);
        c.head_stride = k.stride(1);
        c.pos_stride = k.stride(2);
        c.k = k.mutable_data_ptr();
        c.v = v.mutable_data_ptr();
    }
};
struct Tables {
    static constexpr const char *name = "lf_page_tables";
    lf_page_tables c;
    at::Tensor parts[5];   // tables, lens, free_pages, n_free, status
    c10::DeviceIndex device;

    void locate()
    {
        int32_t **const at[5] = {&c.tables, &c.lens, &c.free_pages, &c.n_free, &c.status};
        const int64_t size[5] = {c.n_seqs, c.n_seqs, c.n_pages, 1, 1};
        for (int i = 0; i < 5; ++i) {
            const at::Tensor &t = parts[i];
            const bool two = i == 0;
            if (t.layout() != at::kStrided || t.dim() != (two ? 2 : 1) || t.size(0) != size[i] || (two && t.size(1) != c.max_pages) ||
                (two ? t.size(1) > 1 && t.stride(1) != 1 : !t.is_contiguous()) || t.scalar_type() != at::kInt || !t.is_cuda() ||
                t.get_device() != device)
                throw Refused("a tensor of the page tables is no longer what they were made with");
            *at[i] = t.mutable_data_ptr<int32_t>();
        }
        c.table_stride = c.n_seqs > 1 ? parts[0].stride(0) : c.max_pages;
    }
};

struct NoGil {   // an allocation may wait for another thread
    PyThreadState *s = PyEval_SaveThread();
    ~NoGil() { PyEval_RestoreThread(s); }
};

template <class H>
H *handle_of(PyObject *o) { return static_cast<H *>(PyCapsule_GetPointer(o, H::name)); }

// A Python integer of 32 bits; false with an error set for anything else.
bool int32(PyObject *o, int32_t &x, const char *what)
{
    int over = 0;
    const long long v = PyLong_AsLongLongAndOverflow(o, &over);
    if (v == -1 && !over && PyErr_Occurred()) return false;
    if (over || v < INT_MIN || v > INT_MAX) {
        PyErr_Format(PyExc_ValueError, "%s %S: 32 bits are needed", what, o);
        return false;
    }
    x = (int32_t)v;
    return true;
}

// The rows of tensor o [n, heads, head_dim], or Refused.
template <class H>
lf_rows rows_of(PyObject *o, const H &c, int64_t n, int64_t heads, const char *what)
{
    if (!THPVariable_Check(o)) throw Refused(std::string(what) + " is no tensor");
    const at::Tensor &t = THPVariable_Unpack(o);
    int code = -1;
    if (t.scalar_type() == at::kHalf) code = LF_F16;
    else if (t.scalar_type() == at::kBFloat16) code = LF_BF16;
    else if (t.scalar_type() == at::kFloat) code = LF_F32;
    const int64_t hd = c.c.head_dim;
    if (code < 0 || t.layout() != at::kStrided || t.dim() != 3 || t.size(0) != n || t.size(1) != heads || t.size(2) != hd ||
        !t.is_cuda() || t.get_device() != c.device || t.stride(2) != 1) {
        std::ostringstream s;
        s << what << " is " << t.scalar_type() << ' ' << t.sizes();
        if (t.layout() == at::kStrided) s << ", strides " << t.strides();
        s << ", on " << t.device() << ": [" << n << ", " << heads << ", " << hd
          << "] float16, bfloat16 or float32 with a contiguous last dimension on cuda:" << (int)c.device << " is needed";
        throw Refused(s.str());
    }
    no_derivatives(t, what);
    // the stride of a dimension of one is never used (and may be anything)
    return {const_cast<void *>(t.const_data_ptr()), code, n > 1 ? t.stride(0) : 0, heads > 1 ? t.stride(1) : 0};
}
// Sizes of a tensor of rows: [n, heads, ..] (the rest is rows_of's to check)
void sizes_of(PyObject *o, int32_t &n, int32_t &heads, const char *what)
{
    if (!THPVariable_Check(o)) throw Refused(std::string(what) + " is no tensor");
    const at::Tensor &t = THPVariable_Unpack(o);
    if (t.dim() != 3 || t.size(0) > INT_MAX || t.size(1) > INT_MAX) {
        std::ostringstream s;
        s << what << " is " << t.sizes() << ": three dimensions of 32 bits are needed";
        throw Refused(s.str());
    }
    n = (int32_t)t.size(0);
    heads = (int32_t)t.size(1);
}
at::Tensor empty(at::IntArrayRef size, at::ScalarType type, c10::DeviceIndex device)
{
    return at::Tensor(at::detail::empty_cuda(size, type, at::Device(at::kCUDA, device), std::nullopt));
}
// A new output of n rows, as q says and not its tensor (which another thread may resize meanwhile), and q.out for it.
template <class Q>
at::Tensor output(int64_t n, Q &q, int64_t hd, c10::DeviceIndex device)
{
    const at::ScalarType type = q.q.dtype == LF_F16 ? at::kHalf : q.q.dtype == LF_BF16 ? at::kBFloat16 : at::kFloat;
    at::Tensor t = empty({n, q.n_heads, hd}, type, device);
    q.out = {t.mutable_data_ptr(), q.q.dtype, q.n_heads * hd, hd};
    return t;
}
// A contiguous tensor of n 32-bit integers.
const int32_t *ints_of(PyObject *o, int64_t n, c10::DeviceIndex device, const char *what)
{
    if (!THPVariable_Check(o)) throw Refused(std::string(what) + " is no tensor");
    const at::Tensor &t = THPVariable_Unpack(o);
    if (t.layout() != at::kStrided || t.dim() != 1 || t.size(0) != n || t.scalar_type() != at::kInt || !t.is_contiguous() ||
        !t.is_cuda() || t.get_device() != device) {
        std::ostringstream s;
        s << what << " is " << t.scalar_type() << ' ' << t.sizes() << ", on " << t.device() << ": [" << n
          << "] int32, contiguous, on cuda:" << (int)device << " is needed";
        throw Refused(s.str());
    }
    return static_cast<const int32_t *>(t.const_data_ptr());
}
template <class H>
void *stream_of(const H &c) { return c10::cuda::getCurrentCUDAStream(c.device).stream(); }

// Runs f with C++ errors turned into Python ones; NotImplemented where the cache's device is not the current one.
template <class H = Cache, class F>
PyObject *call(PyObject *const *args, Py_ssize_t n_args, Py_ssize_t want, const char *where, F f)
{
    if (n_args != want) {
        PyErr_Format(PyExc_TypeError, "%s takes %zd arguments", where, want);
        return nullptr;
    }
    H *c = handle_of<H>(args[0]);
    if (!c) return nullptr;
    HANDLE_TH_ERRORS
    try {
        if (c10::cuda::current_device() != c->device) Py_RETURN_NOTIMPLEMENTED;
        c->locate();
        lf_status st = LF_OK;
        PyObject *out = f(*c, st);
        if (st == LF_OK || !out) return out;
        Py_DECREF(out);
        Py_XDECREF(PyObject_CallFunction(g_fail, "is", (int)st, where));
    } catch (const Refused &e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    }
    return nullptr;
    END_HANDLE_TH_ERRORS
}

// append(cache, k, v, pos)
PyObject *append(PyObject *, PyObject *const *args, Py_ssize_t n_args)
{
    return call(args, n_args, 4, "lf_kv4_append", [&](Cache &c, lf_status &st) -> PyObject * {
        int32_t pos, n, heads;
        if (!int32(args[3], pos, "pos")) return nullptr;
        sizes_of(args[1], n, heads, "k");
        const lf_rows k = rows_of(args[1], c, n, c.c.n_kv_heads, "k"), v = rows_of(args[2], c, n, c.c.n_kv_heads, "v");
        st = g_append(&c.c, &k, &v, n, pos, stream_of(c));
        for (const at::Tensor &t : c.parts) written(t);
        Py_RETURN_NONE;
    });
}

// read(cache, pos, n, type, k or None, v or None) -> (k, v)
PyObject *read(PyObject *, PyObject *const *args, Py_ssize_t n_args)
{
    return call(args, n_args, 6, "lf_kv4_read", [&](Cache &c, lf_status &st) -> PyObject * {
        int32_t pos, n, type;
        if (!int32(args[1], pos, "pos") || !int32(args[2], n, "n") || !int32(args[3], type, "type")) return nullptr;
        // (rows that the cache does not have are the library's to refuse, before any memory is asked for)
        const int64_t rows = n > 0 && pos >= 0 && (long long)pos + n <= c.c.max_seq ? n : 0, heads = c.c.n_kv_heads;
        PyObject *k = args[4], *v = args[5];
        if (k == Py_None) {
            const at::ScalarType t = type == LF_F16 ? at::kHalf : type == LF_BF16 ? at::kBFloat16 : at::kFloat;
            at::Tensor x, y;
            {
                NoGil free;
                x = empty({rows, heads, c.c.head_dim}, t, c.device);
                y = empty({rows, heads, c.c.head_dim}, t, c.device);
            }
            k = THPVariable_Wrap(std::move(x));
            v = THPVariable_Wrap(std::move(y));
        } else {
            Py_INCREF(k);
            Py_INCREF(v);
        }
        PyObject *out = k && v ? PyTuple_New(2) : nullptr;
        if (!out) {
            Py_XDECREF(k);
            Py_XDECREF(v);
            return nullptr;
        }
        PyTuple_SET_ITEM(out, 0, k);
        PyTuple_SET_ITEM(out, 1, v);
        try {
            const lf_rows a = rows_of(k, c, rows, heads, "k"), b = rows_of(v, c, rows, heads, "v");
            st = g_read(&c.c, &a, &b, n, pos, stream_of(c));
            written(k);
            written(v);
        } catch (...) {
            Py_DECREF(out);
            throw;
        }
        return out;
    });
}

// attend(cache, q, pos, length or None, window, scale, out or None) -> out
PyObject *attend(PyObject *, PyObject *const *args, Py_ssize_t n_args)
{
    return call(args, n_args, 7, "lf_kv4_attend", [&](Cache &c, lf_status &st) -> PyObject * {
        lf_kv4_query q = {};
        sizes_of(args[1], q.n, q.n_heads, "q");
        if (!int32(args[2], q.pos, "pos") || !int32(args[4], q.window, "window")) return nullptr;
        if (args[3] == Py_None) {
            const long long seen = (long long)q.pos + q.n;
            q.length = (int32_t)(seen < INT_MAX ? seen : INT_MAX);   // (refused as more than the cache holds)
        } else if (!int32(args[3], q.length, "length")) {
            return nullptr;
        }
        const double scale = PyFloat_AsDouble(args[5]);
        if (scale == -1.0 && PyErr_Occurred()) return nullptr;
        q.scale = (float)scale;
        if (q.scale == 0.f && scale != 0.0) throw Refused("scale vanishes in 32 bits, and 0 selects 1 / sqrt(head_dim)");
        q.q = rows_of(args[1], c, q.n, q.n_heads, "q");
        PyObject *out = args[6];
        void *const stream = stream_of(c);
        if (out != Py_None) q.out = rows_of(out, c, q.n, q.n_heads, "out");
        // Scratch (long contexts and large blocks need some) belongs to this call alone: no two streams or captured
        // graphs share it.  Its size is asked for when a call like the last one turns out not to have enough.
        const bool like = c.n == q.n && c.heads == q.n_heads;
        const int64_t had = like ? c.scratch : 0;
        int64_t need = 0;
        at::Tensor made;
        const lf_kv4 cache = c.c;                         // (c is another thread's to change meanwhile)
        {
            NoGil free;
            if (out == Py_None) made = output(q.n, q, cache.head_dim, c.device);
            at::Tensor ws;
            if (had) ws = empty({had}, at::kByte, c.device);
            st = g_attend(&cache, &q, had ? ws.mutable_data_ptr() : nullptr, had, stream);
            if (st == LF_ERR_INVALID_ARG && g_workspace(&cache, &q, &need) == LF_OK && need > had) {
                ws = empty({need}, at::kByte, c.device);
                st = g_attend(&cache, &q, ws.mutable_data_ptr(), need, stream);
            }
        }
        if (need > had) c.n = q.n, c.heads = q.n_heads, c.scratch = need;
        if (out != Py_None) written(out);
        return out == Py_None ? THPVariable_Wrap(std::move(made)) : Py_NewRef(out);
    });
}

template <class H>
void drop(PyObject *o) { delete handle_of<H>(o); }

// cache(n_kv_heads, head_dim, max_seq, device, k_codes, k_scales, v_codes, v_scales)
PyObject *cache(PyObject *, PyObject *args)
{
    int h, hd, s, device;
    PyObject *p[4];
    if (!PyArg_ParseTuple(args, "iiiiOOOO", &h, &hd, &s, &device, &p[0], &p[1], &p[2], &p[3])) return nullptr;
    Cache *c = new (std::nothrow) Cache;
    if (!c) return PyErr_NoMemory();
    c->c = {h, hd, s, nullptr, nullptr, nullptr, nullptr};
    c->device = (c10::DeviceIndex)device;
    for (int i = 0; i < 4; ++i) {
        if (!THPVariable_Check(p[i])) {
            delete c;
            PyErr_SetString(PyExc_ValueError, "a cache is four tensors");
            return nullptr;
        }
        c->parts[i] = THPVariable_Unpack(p[i]);
    }
    PyObject *o = PyCapsule_New(c, Cache::name, drop<Cache>);
    if (!o) delete c;
    return o;
}

// paged(k, v): the pools [n_pages, n_kv_heads, page, head_dim] (their checks are here and in the library)
PyObject *paged(PyObject *, PyObject *args)
{
    PyObject *k, *v;
    if (!PyArg_ParseTuple(args, "OO", &k, &v)) return nullptr;
    HANDLE_TH_ERRORS
    try {
        if (!THPVariable_Check(k) || !THPVariable_Check(v)) throw Refused("a paged cache is two tensors");
        const at::Tensor &a = THPVariable_Unpack(k), &b = THPVariable_Unpack(v);
        std::unique_ptr<Paged> c(new Paged);
        c->c = {};
        bool ok = a.layout() == at::kStrided && a.dim() == 4 && a.is_cuda() && (a.scalar_type() == at::kHalf || a.scalar_type() == at::kBFloat16);
        for (int i = 0; ok && i < 4; ++i) ok = a.size(i) <= INT_MAX;
        if (ok) {
            c->c.n_pages = (int32_t)a.size(0);
            c->c.n_kv_heads = (int32_t)a.size(1);
            c->c.page = (int32_t)a.size(2);
            c->c.head_dim = (int32_t)a.size(3);
            c->c.dtype = a.scalar_type() == at::kHalf ? LF_F16 : LF_BF16;
            c->device = a.get_device();
            c->k = a;
            c->v = b;
            ok = Paged::fits(a, c->c, c->device) && Paged::fits(b, c->c, c->device) && Paged::alike(a, b);
        }
        if (!ok)
            throw Refused("k and v must be CUDA tensors [n_pages, n_kv_heads, page, head_dim] in float16 or bfloat16, alike in type, "
                          "device and strides, with a contiguous last dimension");
        c->place();
        // what else the library refuses, at once: an append of no rows checks the pools and does nothing
        if (const lf_status st = g_paged_append(&c->c, nullptr, nullptr, 0, nullptr, nullptr); st != LF_OK) {
            Py_XDECREF(PyObject_CallFunction(g_fail, "is", (int)st, "lf_paged"));
            return nullptr;
        }
        PyObject *o = PyCapsule_New(c.get(), Paged::name, drop<Paged>);
        if (o) c.release();
        return o;
    } catch (const Refused &e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    }
    return nullptr;
    END_HANDLE_TH_ERRORS
}

// paged_append(cache, k, v, slots)
PyObject *paged_append(PyObject *, PyObject *const *args, Py_ssize_t n_args)
{
    return call<Paged>(args, n_args, 4, "lf_paged_append", [&](Paged &c, lf_status &st) -> PyObject * {
        int32_t n, heads;
        sizes_of(args[1], n, heads, "k");
        const lf_rows k = rows_of(args[1], c, n, c.c.n_kv_heads, "k"), v = rows_of(args[2], c, n, c.c.n_kv_heads, "v");
        st = g_paged_append(&c.c, &k, &v, n, ints_of(args[3], n, c.device, "slots"), stream_of(c));
        written(c.k);
        written(c.v);
        Py_RETURN_NONE;
    });
}

// paged_attend(cache, q, tables, lens, window, scale, out or None) -> out
PyObject *paged_attend(PyObject *, PyObject *const *args, Py_ssize_t n_args)
{
    return call<Paged>(args, n_args, 7, "lf_paged_attend", [&](Paged &c, lf_status &st) -> PyObject * {
        lf_paged_query q = {};
        sizes_of(args[1], q.n_seqs, q.n_heads, "q");
        if (!int32(args[4], q.window, "window")) return nullptr;
        const double scale = PyFloat_AsDouble(args[5]);
        if (scale == -1.0 && PyErr_Occurred()) return nullptr;
        q.scale = (float)scale;
        if (q.scale == 0.f && scale != 0.0) throw Refused("scale vanishes in 32 bits, and 0 selects 1 / sqrt(head_dim)");
        q.q = rows_of(args[1], c, q.n_seqs, q.n_heads, "q");
        if (!THPVariable_Check(args[2])) throw Refused("tables is no tensor");
        const at::Tensor &t = THPVariable_Unpack(args[2]);
        if (t.layout() != at::kStrided || t.dim() != 2 || t.size(0) != q.n_seqs || t.size(1) > INT_MAX || t.scalar_type() != at::kInt ||
            (t.size(1) > 1 && t.stride(1) != 1) || !t.is_cuda() || t.get_device() != c.device) {
            std::ostringstream s;
            s << "tables is " << t.scalar_type() << ' ' << t.sizes() << ", on " << t.device() << ": [" << q.n_seqs
              << ", pages] int32 with a contiguous last dimension on cuda:" << (int)c.device << " is needed";
            throw Refused(s.str());
        }
        q.tables = static_cast<const int32_t *>(t.const_data_ptr());
        q.table_width = (int32_t)t.size(1);
        q.table_stride = q.n_seqs > 1 ? t.stride(0) : 0;
        q.lens = ints_of(args[3], q.n_seqs, c.device, "lens");
        PyObject *out = args[6];
        void *const stream = stream_of(c);
        if (out != Py_None) q.out = rows_of(out, c, q.n_seqs, q.n_heads, "out");
        at::Tensor made;
        const lf_paged cache = c.c;                       // (c is another thread's to change meanwhile)
        {
            NoGil free;
            if (out == Py_None) made = output(q.n_seqs, q, cache.head_dim, c.device);
            // Scratch, where a call needs some (few long sequences do), is that call's alone: no two streams or captured
            // graphs share it.
            st = g_paged_attend(&cache, &q, nullptr, 0, stream);
            int64_t need = 0;
            if (st == LF_ERR_INVALID_ARG && g_paged_workspace(&cache, &q, &need) == LF_OK && need > 0) {
                const at::Tensor ws = empty({need}, at::kByte, c.device);
                st = g_paged_attend(&cache, &q, ws.mutable_data_ptr(), need, stream);
            }
        }
        if (out != Py_None) written(out);
        return out == Py_None ? THPVariable_Wrap(std::move(made)) : Py_NewRef(out);
    });
}

// page_tables(page, tables, lens, free_pages, n_free, status)
PyObject *page_tables(PyObject *, PyObject *args)
{
    int page;
    PyObject *p[5];
    if (!PyArg_ParseTuple(args, "iOOOOO", &page, &p[0], &p[1], &p[2], &p[3], &p[4])) return nullptr;
    HANDLE_TH_ERRORS
    try {
        std::unique_ptr<Tables> c(new Tables);
        c->c = {};
        for (int i = 0; i < 5; ++i) {
            if (!THPVariable_Check(p[i])) throw Refused("page tables are tensors");
            c->parts[i] = THPVariable_Unpack(p[i]);
        }
        const at::Tensor &t = c->parts[0], &f = c->parts[2];
        if (t.dim() != 2 || f.dim() != 1 || t.size(0) > INT_MAX || t.size(1) > INT_MAX || f.size(0) > INT_MAX)
            throw Refused("tables [n_seqs, max_pages] and free [n_pages] of 32 bits are needed");
        c->c.n_seqs = (int32_t)t.size(0);
        c->c.max_pages = (int32_t)t.size(1);
        c->c.n_pages = (int32_t)f.size(0);
        c->c.page = page;
        c->device = t.get_device();
        try {
            c->locate();
        } catch (const Refused &) {
            throw Refused("tables [n_seqs, max_pages], lens [n_seqs], free [n_pages] and n_free [1] must be contiguous CUDA "
                          "torch.int32 tensors on one device (tables in its last dimension)");
        }
        PyObject *o = PyCapsule_New(c.get(), Tables::name, drop<Tables>);
        if (o) c.release();
        return o;
    } catch (const Refused &e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    }
    return nullptr;
    END_HANDLE_TH_ERRORS
}

// plan(tables, n_new, max_tokens, keep or None) -> (slots, positions, offsets)
PyObject *plan(PyObject *, PyObject *const *args, Py_ssize_t n_args)
{
    return call<Tables>(args, n_args, 4, "lf_paged_plan", [&](Tables &c, lf_status &st) -> PyObject * {
        int32_t most;
        if (!int32(args[2], most, "max_tokens")) return nullptr;
        if (most < 0) throw Refused("max_tokens is negative");
        const int32_t *n_new = ints_of(args[1], c.c.n_seqs, c.device, "n_new");
        const int32_t *keep = args[3] == Py_None ? nullptr : ints_of(args[3], c.c.n_seqs, c.device, "keep");
        void *const stream = stream_of(c);
        const lf_page_tables tables = c.c;
        // one allocation for the three (each costs two microseconds where its code is cold)
        const int64_t size[3] = {most, most, (int64_t)tables.n_seqs + 1}, pitch = ((int64_t)most + 3) / 4 * 4;
        at::Tensor all, made[3];
        {
            NoGil free;
            all = empty({2 * pitch + size[2]}, at::kInt, c.device);
            int32_t *const p = all.mutable_data_ptr<int32_t>();
            st = g_plan(&tables, n_new, keep, p, p + pitch, p + 2 * pitch, most, stream);
        }
        for (const at::Tensor &t : c.parts) written(t);
        for (int i = 0; i < 3; ++i) {
            made[i] = at::detail::make_tensor<at::TensorImpl>(c10::Storage(all.storage()), all.key_set(), all.dtype());
            made[i].unsafeGetTensorImpl()->set_sizes_contiguous(size[i]);
            made[i].unsafeGetTensorImpl()->set_storage_offset(i * pitch);
        }
        PyObject *out = PyTuple_New(3);
        for (int i = 0; out && i < 3; ++i) {
            PyObject *x = THPVariable_Wrap(std::move(made[i]));
            if (!x) {
                Py_DECREF(out);
                return nullptr;
            }
            PyTuple_SET_ITEM(out, i, x);
        }
        return out;
    });
}

// bind(append, read, attend, workspace, plan, paged append, attend, workspace, fail): the library's entry points, by
// address
PyObject *bind(PyObject *, PyObject *args)
{
    unsigned long long a, r, t, w, p, pa, pt, pw;
    PyObject *fail;
    if (!PyArg_ParseTuple(args, "KKKKKKKKO", &a, &r, &t, &w, &p, &pa, &pt, &pw, &fail)) return nullptr;
    g_append = reinterpret_cast<decltype(g_append)>(a);
    g_read = reinterpret_cast<decltype(g_read)>(r);
    g_attend = reinterpret_cast<decltype(g_attend)>(t);
    g_workspace = reinterpret_cast<decltype(g_workspace)>(w);
    g_plan = reinterpret_cast<decltype(g_plan)>(p);
    g_paged_append = reinterpret_cast<decltype(g_paged_append)>(pa);
    g_paged_attend = reinterpret_cast<decltype(g_paged_attend)>(pt);
    g_paged_workspace = reinterpret_cast<decltype(g_paged_workspace)>(pw);
    Py_INCREF(fail);
    Py_XSETREF(g_fail, fail);
    Py_RETURN_NONE;
}

#define FAST(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(append),
                         FAST(read),
                         FAST(attend),
                         FAST(paged_append),
                         FAST(paged_attend),
                         FAST(plan),
                         {"cache", cache, METH_VARARGS, nullptr},
                         {"paged", paged, METH_VARARGS, nullptr},
                         {"page_tables", page_tables, METH_VARARGS, nullptr},
                         {"bind", bind, METH_VARARGS, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
#undef FAST
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_lft", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// made_for: the release of torch and the version of Python (sys.hexversion >> 16) that this module fits
PyMODINIT_FUNC PyInit__lft()
{
    PyObject *m = PyModule_Create(&module);
    PyObject *made = m ? Py_BuildValue("(si)", TORCH_VERSION, (int)(PY_VERSION_HEX >> 16)) : nullptr;
    if (!made || PyModule_AddObjectRef(m, "made_for", made) < 0) Py_CLEAR(m);
    Py_XDECREF(made);
    return m;
}
