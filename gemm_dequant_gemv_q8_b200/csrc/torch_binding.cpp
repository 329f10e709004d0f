// torch_binding.cpp -- argument marshalling of the calls that a decode step makes once a layer: the same checks and the
// same C ABI as a ctypes call, on torch tensors without the Python objects in between (a call is 5 to 6 us on the host
// instead of 13 to 17).  No computation happens here; the library's entry points come in by address (bind).
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/qlin.h"

namespace {

decltype(&qlin_qk_norm_rope) f_qk_norm_rope = nullptr;
decltype(&qlin_kv_append) f_kv_append = nullptr;
decltype(&qlin_kv_gather) f_kv_gather = nullptr;
decltype(&qlin_attn_kv4) f_attn_kv4 = nullptr;
PyObject* error_type = nullptr;  // QlinError

struct Fail {};  // a Python error is set

[[noreturn]] void fail(PyObject* type, const char* fmt, const char* name) {
    PyErr_Format(type, fmt, name);
    throw Fail();
}
void check_status(const char* fn, qlin_status_t st) {
    if (st == QLIN_OK) return;
    PyObject* e = PyObject_CallFunction(error_type, "si", fn, (int)st);
    if (e) {
        PyErr_SetObject(error_type, e);
        Py_DECREF(e);
    }
    throw Fail();
}
int64_t integer(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Fail();
    return v;
}
int small(PyObject* o) {
    const int64_t v = integer(o);
    if (v < INT32_MIN || v > INT32_MAX) fail(PyExc_OverflowError, "%s does not fit 32 bits", "an argument");
    return (int)v;
}
float real(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Fail();
    return (float)v;
}
const at::Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) fail(PyExc_TypeError, "%s must be a tensor", name);
    return THPVariable_Unpack(o);
}
const at::Tensor& on_device(PyObject* o, const char* name, at::ScalarType dt, int dev) {
    const at::Tensor& t = tensor(o, name);
    if (!t.is_cuda() || t.get_device() != dev || t.scalar_type() != dt)
        fail(PyExc_TypeError, "%s must be of the right type and on the call's CUDA device", name);
    return t;
}
// Address of a contiguous vector of n values (n < 0: any), NULL for None.
template <typename T>
T* vec(PyObject* o, const char* name, at::ScalarType dt, int dev, int64_t n) {
    if (o == Py_None) return nullptr;
    const at::Tensor& t = on_device(o, name, dt, dev);
    if (t.dim() != 1 || (n >= 0 && t.size(0) != n)) fail(PyExc_ValueError, "%s must be 1-d and of the right length", name);
    if (!t.is_contiguous()) fail(PyExc_ValueError, "%s must be contiguous", name);
    return static_cast<T*>(t.data_ptr());
}
at::ScalarType dtype_of(int ydt) {
    if (ydt != QLIN_F32 && ydt != QLIN_BF16) fail(PyExc_ValueError, "%s must be QLIN_F32 or QLIN_BF16", "ydt");
    return ydt == QLIN_F32 ? at::kFloat : at::kBFloat16;
}

// T rows of heads * D contiguous values, (T, heads, D) or (T, heads * D): given, or new ones.
struct Rows {
    PyObject* obj;  // a new reference
    void* p;
    int64_t ld;
};
Rows rows(PyObject* o, const char* name, at::ScalarType dt, const at::Tensor& like, int64_t T, int64_t heads, int64_t D) {
    Rows r;
    if (o == Py_None) {
        at::Tensor t = at::empty({T, heads, D}, like.options().dtype(dt));
        r.p = t.data_ptr(), r.ld = heads * D;
        r.obj = THPVariable_Wrap(std::move(t));
        if (!r.obj) throw Fail();
        return r;
    }
    const at::Tensor& t = on_device(o, name, dt, like.get_device());
    const bool three = t.dim() == 3;
    if (!(three && t.size(0) == T && t.size(1) == heads && t.size(2) == D) &&
        !(t.dim() == 2 && t.size(0) == T && t.size(1) == heads * D))
        fail(PyExc_ValueError, "%s must be (rows, heads, D) or (rows, heads * D)", name);
    if ((t.size(t.dim() - 1) > 1 && t.stride(t.dim() - 1) != 1) || (three && heads > 1 && t.stride(1) != D))
        fail(PyExc_ValueError, "%s's rows must be contiguous", name);
    r.p = t.data_ptr(), r.ld = T > 1 ? t.stride(0) : heads * D;
    Py_INCREF(o);
    r.obj = o;
    return r;
}

struct Input {
    const at::Tensor* t;
    qlin_dtype_t dt;
    int dev;
    int64_t T, ld;
};
Input projections(PyObject* o, int64_t width, bool exact) {
    const at::Tensor& t = tensor(o, "x");
    const at::ScalarType s = t.scalar_type();
    if (!t.is_cuda() || t.dim() != 2 || (s != at::kFloat && s != at::kBFloat16))
        fail(PyExc_TypeError, "%s must be a 2-d float32 or bfloat16 CUDA tensor", "x");
    if (exact ? t.size(1) != width : t.size(1) < width) fail(PyExc_ValueError, "%s has the wrong number of columns", "x");
    if (t.stride(1) != 1) fail(PyExc_ValueError, "%s's rows must be contiguous", "x");
    return {&t, s == at::kFloat ? QLIN_F32 : QLIN_BF16, (int)t.get_device(), t.size(0), t.size(0) > 1 ? t.stride(0) : t.size(1)};
}
struct Scratch {
    void* p;
    size_t n;
};
Scratch scratch(PyObject* o, int dev) {
    const at::Tensor& t = tensor(o, "ws");
    if (!t.is_cuda() || t.get_device() != dev || !t.is_contiguous()) fail(PyExc_TypeError, "%s must be contiguous and on the call's CUDA device", "ws");
    return {t.data_ptr(), t.nbytes()};
}
// The call's device, made current (the library works on the current one), and its current stream.
struct Where {
    c10::cuda::OptionalCUDAGuard guard;
    qlin_stream_t stream;
    explicit Where(int dev) {
        if (c10::cuda::current_device() != dev) guard.set_index((c10::DeviceIndex)dev);
        stream = (qlin_stream_t)c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream();
    }
};
// cos_sin, q_weight, k_weight, eps, rot, flags
qlin_qk_params params(PyObject* const* a, int D, int dev) {
    qlin_qk_params p = {};
    if (a[4] != Py_None) p.rot = small(a[4]);  // without a table the library refuses what is not 0
    if (a[0] != Py_None) {
        const at::Tensor& t = on_device(a[0], "cos_sin", at::kFloat, dev);
        if (t.dim() != 2 || !t.is_contiguous()) fail(PyExc_ValueError, "%s must be a contiguous (positions, rot) tensor", "cos_sin");
        if (t.size(1) > INT32_MAX) fail(PyExc_ValueError, "%s is too large", "cos_sin");
        if (a[4] == Py_None) p.rot = (int)t.size(1);
        if (p.rot && t.size(1) != p.rot) fail(PyExc_ValueError, "%s must be (positions, rot)", "cos_sin");
        p.cos_sin = static_cast<const float*>(t.data_ptr());
        p.n_pos = t.size(0);
    }
    p.q_weight = vec<const float>(a[1], "q_weight", at::kFloat, dev, D);
    p.k_weight = vec<const float>(a[2], "k_weight", at::kFloat, dev, D);
    p.eps = real(a[3]);
    p.flags = small(a[5]);
    return p;
}
const qlin_kv_cache* cache_of(PyObject* o) { return reinterpret_cast<const qlin_kv_cache*>((uintptr_t)integer(o)); }

PyObject* pair(PyObject* a, PyObject* b) {
    PyObject* t = PyTuple_Pack(2, a, b);
    Py_DECREF(a);
    Py_DECREF(b);
    return t;
}
struct Held {  // drops its reference if the call fails
    PyObject* o;
    ~Held() { Py_XDECREF(o); }
    PyObject* release() {
        PyObject* r = o;
        o = nullptr;
        return r;
    }
};

#define CALL(name, nargs)                                                              \
    PyObject* name##_(PyObject* const* a);                                             \
    PyObject* name(PyObject*, PyObject* const* a, Py_ssize_t n) {                      \
        HANDLE_TH_ERRORS                                                               \
        if (n != nargs || !f_##name) {                                                 \
            PyErr_SetString(PyExc_TypeError, #name ": wrong number of arguments");     \
            return nullptr;                                                            \
        }                                                                              \
        try {                                                                          \
            return name##_(a);                                                         \
        } catch (const Fail&) {                                                        \
            return nullptr;                                                            \
        }                                                                              \
        END_HANDLE_TH_ERRORS                                                           \
    }                                                                                  \
    PyObject* name##_(PyObject* const* a)

// x, Hq, Hkv, D, positions, (cos_sin, q_weight, k_weight, eps, rot, flags), q, k, ydt, ws
CALL(qk_norm_rope, 15) {
    const int Hq = small(a[1]), Hkv = small(a[2]), D = small(a[3]), ydt = small(a[13]);
    const Input x = projections(a[0], (int64_t)(Hq + Hkv) * D, false);
    const qlin_qk_params p = params(a + 5, D, x.dev);
    const int32_t* pos = vec<const int32_t>(a[4], "positions", at::kInt, x.dev, x.T);
    const Rows q = rows(a[11], "q", dtype_of(ydt), *x.t, x.T, Hq, D);
    Held hq{q.obj};
    const Rows k = rows(a[12], "k", dtype_of(ydt), *x.t, x.T, Hkv, D);
    Held hk{k.obj};
    const Scratch ws = scratch(a[14], x.dev);
    const Where w(x.dev);
    check_status("qlin_qk_norm_rope", f_qk_norm_rope(x.t->data_ptr(), x.dt, x.T, x.ld, Hq, Hkv, D, &p, pos, q.p, q.ld, k.p, k.ld,
                                                     (qlin_dtype_t)ydt, 0, ws.p, ws.n, w.stream));
    return pair(hq.release(), hk.release());
}

// cache, device, x, Hq, Hkv, D, positions, slots, (cos_sin, q_weight, k_weight, eps, rot, flags), q, ws
CALL(kv_append, 16) {
    const qlin_kv_cache* c = cache_of(a[0]);
    const int dev = small(a[1]), Hq = small(a[3]), Hkv = small(a[4]), D = small(a[5]);
    const Input x = projections(a[2], (int64_t)(Hq + 2 * Hkv) * D, true);
    if (x.dev != dev) fail(PyExc_ValueError, "%s must be on x's device", "the cache");
    const qlin_qk_params p = params(a + 8, D, dev);
    const int32_t* pos = vec<const int32_t>(a[6], "positions", at::kInt, dev, x.T);
    const int32_t* slots = vec<const int32_t>(a[7], "slots", at::kInt, dev, x.T);
    const Rows q = rows(a[14], "q", at::kBFloat16, *x.t, x.T, Hq, D);
    Held hq{q.obj};
    const Scratch ws = scratch(a[15], dev);
    const Where w(dev);
    check_status("qlin_kv_append", f_kv_append(c, x.t->data_ptr(), x.dt, x.T, x.ld, Hq, &p, pos, slots, Hq ? q.p : nullptr, q.ld, 0,
                                               ws.p, ws.n, w.stream));
    return hq.release();
}

// cache, device, slots, Hkv, D, k, v, ydt, ws
CALL(kv_gather, 9) {
    const qlin_kv_cache* c = cache_of(a[0]);
    const int dev = small(a[1]), Hkv = small(a[3]), D = small(a[4]), ydt = small(a[7]);
    const at::Tensor& s = on_device(a[2], "slots", at::kInt, dev);
    const int32_t* slots = vec<const int32_t>(a[2], "slots", at::kInt, dev, -1);
    const int64_t T = s.size(0);
    const Rows k = rows(a[5], "k", dtype_of(ydt), s, T, Hkv, D);
    Held hk{k.obj};
    const Rows v = rows(a[6], "v", dtype_of(ydt), s, T, Hkv, D);
    Held hv{v.obj};
    if (k.ld != (int64_t)Hkv * D || v.ld != (int64_t)Hkv * D) fail(PyExc_ValueError, "%s must be contiguous", "k and v");
    const Scratch ws = scratch(a[8], dev);
    const Where w(dev);
    check_status("qlin_kv_gather", f_kv_gather(c, T, slots, k.p, v.p, (qlin_dtype_t)ydt, ws.p, ws.n, w.stream));
    return pair(hk.release(), hv.release());
}

// cache, device, D, q, block_table, seq_lens, cu_q, max_q, scale, window, out, ws
CALL(attn_kv4, 12) {
    const qlin_kv_cache* c = cache_of(a[0]);
    const int dev = small(a[1]), D = small(a[2]), max_q = small(a[7]), window = small(a[9]);
    const at::Tensor& qt = on_device(a[3], "q", at::kBFloat16, dev);
    if (qt.dim() != 3 || qt.size(2) != D) fail(PyExc_ValueError, "%s must be (total_q, Hq, D)", "q");
    const int64_t total = qt.size(0), Hq = qt.size(1);
    const Rows q = rows(a[3], "q", at::kBFloat16, qt, total, Hq, D);
    Held hq{q.obj};
    const at::Tensor& lens = on_device(a[5], "seq_lens", at::kInt, dev);
    const int32_t* plens = vec<const int32_t>(a[5], "seq_lens", at::kInt, dev, -1);
    const int64_t B = lens.size(0);
    const int32_t* cu = vec<const int32_t>(a[6], "cu_q", at::kInt, dev, B + 1);
    const at::Tensor& table = on_device(a[4], "block_table", at::kInt, dev);
    if (table.dim() != 2 || table.size(0) != B || (table.size(1) > 1 && table.stride(1) != 1))
        fail(PyExc_ValueError, "%s must be (B, pages) with contiguous rows", "block_table");
    if (Hq > INT32_MAX || B > INT32_MAX || table.size(1) > INT32_MAX) fail(PyExc_ValueError, "%s is too large", "an argument");
    const Rows out = rows(a[10], "out", at::kBFloat16, qt, total, Hq, D);
    Held ho{out.obj};
    const Scratch ws = scratch(a[11], dev);
    const Where w(dev);
    check_status("qlin_attn_kv4",
                 f_attn_kv4(c, q.p, q.ld, static_cast<const int32_t*>(table.data_ptr()), B > 1 ? table.stride(0) : table.size(1),
                            (int)table.size(1), plens, cu, (int)B, max_q, total, (int)Hq, real(a[8]), window, out.p, out.ld, 0,
                            ws.p, ws.n, w.stream));
    return ho.release();
}

// bind(QlinError, addresses of qlin_qk_norm_rope, qlin_kv_append, qlin_kv_gather, qlin_attn_kv4)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 5) {
        PyErr_SetString(PyExc_TypeError, "bind: five arguments");
        return nullptr;
    }
    void* p[4];
    for (int i = 0; i < 4; ++i) {
        p[i] = PyLong_AsVoidPtr(a[i + 1]);
        if (!p[i] && PyErr_Occurred()) return nullptr;
    }
    Py_INCREF(a[0]);
    Py_XDECREF(error_type);
    error_type = a[0];
    f_qk_norm_rope = (decltype(f_qk_norm_rope))p[0];
    f_kv_append = (decltype(f_kv_append))p[1];
    f_kv_gather = (decltype(f_kv_gather))p[2];
    f_attn_kv4 = (decltype(f_attn_kv4))p[3];
    Py_RETURN_NONE;
}

#define METHOD(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(bind), METHOD(qk_norm_rope), METHOD(kv_append), METHOD(kv_gather), METHOD(attn_kv4),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_qlin_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__qlin_torch() { return PyModule_Create(&module); }
