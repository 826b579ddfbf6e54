// lf_torch.cpp -- what KV4Cache does per call, for Python: torch tensors to
// lf_rows, their checks, the output's and the scratch's memory, the call.
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
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/version.h>

#include <climits>
#include <optional>
#include <sstream>
#include <string>

#include "../../include/lf.h"

namespace {

decltype(&lf_kv4_append) g_append;
decltype(&lf_kv4_read) g_read;
decltype(&lf_kv4_attend) g_attend;
decltype(&lf_kv4_workspace) g_workspace;
PyObject *g_fail;   // raises the library's error: fail(status, entry point)

struct Refused : std::runtime_error {
    using std::runtime_error::runtime_error;
};

// A cache as the library has it, its tensors (k_codes, k_scales, v_codes, v_scales) and device, and the scratch that
// the last query that needed some did.
struct Cache {
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

struct NoGil {   // an allocation may wait for another thread
    PyThreadState *s = PyEval_SaveThread();
    ~NoGil() { PyEval_RestoreThread(s); }
};

Cache *cache_of(PyObject *o) { return static_cast<Cache *>(PyCapsule_GetPointer(o, "lf_kv4")); }

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
lf_rows rows_of(PyObject *o, const Cache &c, int64_t n, int64_t heads, const char *what)
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
    if (t.requires_grad() && c10::GradMode::is_enabled())
        throw Refused(std::string(what) + " requires a gradient, and these calls form none: detach it, or call under torch.no_grad()");
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
void *stream_of(const Cache &c) { return c10::cuda::getCurrentCUDAStream(c.device).stream(); }

// Runs f with C++ errors turned into Python ones; NotImplemented where the cache's device is not the current one.
template <class F>
PyObject *call(PyObject *const *args, Py_ssize_t n_args, Py_ssize_t want, const char *where, F f)
{
    if (n_args != want) {
        PyErr_Format(PyExc_TypeError, "%s takes %zd arguments", where, want);
        return nullptr;
    }
    Cache *c = cache_of(args[0]);
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
            if (out == Py_None) {
                const at::Tensor &t = THPVariable_Unpack(args[1]);
                made = empty(t.sizes(), t.scalar_type(), c.device);
                q.out = {made.mutable_data_ptr(), q.q.dtype, q.n_heads * (int64_t)c.c.head_dim, c.c.head_dim};
            }
            at::Tensor ws;
            if (had) ws = empty({had}, at::kByte, c.device);
            st = g_attend(&cache, &q, had ? ws.mutable_data_ptr() : nullptr, had, stream);
            if (st == LF_ERR_INVALID_ARG && g_workspace(&cache, &q, &need) == LF_OK && need > had) {
                ws = empty({need}, at::kByte, c.device);
                st = g_attend(&cache, &q, ws.mutable_data_ptr(), need, stream);
            }
        }
        if (need > had) c.n = q.n, c.heads = q.n_heads, c.scratch = need;
        return out == Py_None ? THPVariable_Wrap(std::move(made)) : Py_NewRef(out);
    });
}

void drop(PyObject *o) { delete cache_of(o); }

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
    PyObject *o = PyCapsule_New(c, "lf_kv4", drop);
    if (!o) delete c;
    return o;
}

// bind(append, read, attend, workspace, fail): the library's entry points, by address
PyObject *bind(PyObject *, PyObject *args)
{
    unsigned long long a, r, t, w;
    PyObject *fail;
    if (!PyArg_ParseTuple(args, "KKKKO", &a, &r, &t, &w, &fail)) return nullptr;
    g_append = reinterpret_cast<decltype(g_append)>(a);
    g_read = reinterpret_cast<decltype(g_read)>(r);
    g_attend = reinterpret_cast<decltype(g_attend)>(t);
    g_workspace = reinterpret_cast<decltype(g_workspace)>(w);
    Py_INCREF(fail);
    Py_XSETREF(g_fail, fail);
    Py_RETURN_NONE;
}

PyMethodDef methods[] = {{"append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(append)), METH_FASTCALL, nullptr},
                         {"read", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(read)), METH_FASTCALL, nullptr},
                         {"attend", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(attend)), METH_FASTCALL, nullptr},
                         {"cache", cache, METH_VARARGS, nullptr},
                         {"bind", bind, METH_VARARGS, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
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
