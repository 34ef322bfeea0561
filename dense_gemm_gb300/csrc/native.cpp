// Argument marshalling for ops.py as a CPython extension: tensors' attributes
// -> gemm_matrix_t, outputs and workspaces from torch.empty, one C call. No
// arithmetic. The same steps through ctypes took 20 us a call on the GB300's host
// (three times a small kernel's time); here about 7.
//
// Every function works on the current device and its current stream; ops.py
// makes another device or stream current first. The library's entry points
// and the torch objects arrive through setup().
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <cstdint>
#include <initializer_list>

#include "gemm_ops.h"

namespace {

// ------------------------------------------------------------------ what setup() stores
enum Entry { kLinear, kLinearSize, kBackward, kBackwardSize, kNorm, kNormBackward, kNormBackwardSize, kEntries };
const char *const kEntryNames[kEntries] = {"gemm_linear", "gemm_linear_workspace_size", "gemm_linear_backward",
                                           "gemm_linear_backward_workspace_size", "gemm_rms_norm",
                                           "gemm_rms_norm_backward", "gemm_rms_norm_backward_workspace_size"};
void *g_entry[kEntries];

template <typename F>
F *entry(Entry e, F *) { return reinterpret_cast<F *>(g_entry[e]); }
#define CALL(e, fn) (entry(e, &fn))

PyObject *g_empty, *g_raw_stream, *g_error, *g_dtype[4], *g_uint8, *g_device_of;  // owned
PyObject *s_dtype, *s_shape, *s_stride, *s_data_ptr, *s_get_device, *s_t;          // interned names
PyObject *g_kw_empty;  // ("dtype", "device")

const char *const kTypeNames[4] = {"float32", "float16", "bfloat16", "float8_e4m3fn"};

// ------------------------------------------------------------------ tensors
struct Tensor {
    PyObject *obj = nullptr;  // borrowed; nullptr: absent
    void *data = nullptr;
    int64_t n[2] = {0, 0}, s[2] = {1, 1};
    int dims = 0;
    int type = -1;  // GEMM_TYPE_*, -1: another one
    int device = -1;
    explicit operator bool() const { return obj != nullptr; }
};

bool small_ints(PyObject *tuple, int64_t *v, int dims) {
    for (int i = 0; i < dims; ++i) {
        v[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(tuple, i));
        if (v[i] == -1 && PyErr_Occurred()) return false;
    }
    return true;
}

int type_code(PyObject *dtype) {
    for (int i = 0; i < 4; ++i)
        if (dtype == g_dtype[i]) return i;
    return -1;
}

// False with a Python error set. None is an absent tensor.
bool read_tensor(PyObject *o, Tensor *t, const char *what) {
    if (o == Py_None) return true;
    t->obj = o;
    PyObject *shape = PyObject_GetAttr(o, s_shape);
    if (shape == nullptr || !PyTuple_Check(shape)) {
        Py_XDECREF(shape);
        PyErr_Format(PyExc_TypeError, "%s must be a torch.Tensor", what);
        return false;
    }
    t->dims = int(PyTuple_GET_SIZE(shape));
    const int d = t->dims < 2 ? t->dims : 2;
    bool ok = small_ints(shape, t->n, d);
    Py_DECREF(shape);
    PyObject *stride = ok ? PyObject_CallMethodNoArgs(o, s_stride) : nullptr;
    ok = stride != nullptr && PyTuple_Check(stride) && small_ints(stride, t->s, d);
    Py_XDECREF(stride);
    PyObject *dtype = ok ? PyObject_GetAttr(o, s_dtype) : nullptr;
    ok = dtype != nullptr;
    if (ok) t->type = type_code(dtype);
    Py_XDECREF(dtype);
    PyObject *dev = ok ? PyObject_CallMethodNoArgs(o, s_get_device) : nullptr;
    if (dev != nullptr) t->device = int(PyLong_AsLong(dev));
    Py_XDECREF(dev);
    PyObject *ptr = dev != nullptr ? PyObject_CallMethodNoArgs(o, s_data_ptr) : nullptr;
    if (ptr != nullptr) t->data = PyLong_AsVoidPtr(ptr);
    Py_XDECREF(ptr);
    return !PyErr_Occurred();
}

// Dimensions of one element may have any stride in torch, also 0; a stride of 0
// elsewhere (an expanded tensor) goes through and is refused by the library.
gemm_matrix_t matrix(const Tensor &t) {
    if (!t) return gemm_matrix_t{nullptr, 1, 1, 0};
    return gemm_matrix_t{t.data, t.s[0] == 0 && t.n[0] <= 1 ? 1 : t.s[0], t.s[1] == 0 && t.n[1] <= 1 ? 1 : t.s[1], t.type};
}

bool same_device(const Tensor &first, std::initializer_list<const Tensor *> others) {
    if (first.device < 0) {
        PyErr_SetString(PyExc_ValueError, "the operators take CUDA tensors");
        return false;
    }
    for (const Tensor *t : others)
        if (*t && t->device != first.device) {
            PyErr_Format(PyExc_ValueError, "all tensors must be on one CUDA device, got device %d and %d", first.device,
                         t->device);
            return false;
        }
    return true;
}

bool is_matrix(const Tensor &t, int64_t rows, int64_t cols, int type, const char *what) {
    if (!t || (t.dims == 2 && t.n[0] == rows && t.n[1] == cols && t.type == type)) return true;
    PyErr_Format(PyExc_ValueError, "%s must be %s of shape [%lld, %lld]", what, kTypeNames[type], (long long)rows,
                 (long long)cols);
    return false;
}

bool is_vector(const Tensor &t, int64_t n, int type, int or_type, const char *what) {
    if (!t) return true;
    if (t.type < 0 || (t.type != type && t.type != or_type)) {
        PyErr_Format(PyExc_TypeError, "%s must be %s%s%s", what, kTypeNames[type], type == or_type ? "" : " or ",
                     type == or_type ? "" : kTypeNames[or_type]);
        return false;
    }
    if (t.dims == 1 && t.n[0] == n && (t.s[0] == 1 || n <= 1)) return true;
    PyErr_Format(PyExc_ValueError, "%s must be a contiguous vector of %lld elements", what, (long long)n);
    return false;
}

// New reference: torch.empty(shape, dtype=, device=) on the tensors' device, and its data.
PyObject *empty(std::initializer_list<int64_t> shape, PyObject *dtype, PyObject *device, void **data) {
    PyObject *size = PyTuple_New(Py_ssize_t(shape.size()));
    if (size == nullptr) return nullptr;
    Py_ssize_t i = 0;
    for (int64_t n : shape) PyTuple_SET_ITEM(size, i++, PyLong_FromLongLong(n));
    PyObject *args[3] = {size, dtype, device};
    PyObject *t = PyObject_Vectorcall(g_empty, args, 1, g_kw_empty);
    Py_DECREF(size);
    if (t == nullptr) return nullptr;
    PyObject *ptr = PyObject_CallMethodNoArgs(t, s_data_ptr);
    if (ptr == nullptr) {
        Py_DECREF(t);
        return nullptr;
    }
    *data = PyLong_AsVoidPtr(ptr);
    Py_DECREF(ptr);
    return t;
}

// An owned reference that may stay empty.
struct Ref {
    PyObject *p = nullptr;
    Ref() = default;
    Ref(const Ref &) = delete;
    Ref &operator=(const Ref &) = delete;
    ~Ref() { Py_XDECREF(p); }
    PyObject *give() {
        PyObject *r = p != nullptr ? p : Py_NewRef(Py_None);
        p = nullptr;
        return r;
    }
};

// The matrix of an output: the given tensor, or a new one stored by rows or (turned) by columns.
bool output(const Tensor &given, int64_t rows, int64_t cols, int type, bool turned, PyObject *device, Ref *keep,
            gemm_matrix_t *m) {
    if (given) {
        keep->p = Py_NewRef(given.obj);
        *m = matrix(given);
        return true;
    }
    void *data = nullptr;
    PyObject *t = turned ? empty({cols, rows}, g_dtype[type], device, &data) : empty({rows, cols}, g_dtype[type], device, &data);
    if (t == nullptr) return false;
    if (turned) {
        keep->p = PyObject_CallMethodNoArgs(t, s_t);
        Py_DECREF(t);
        if (keep->p == nullptr) return false;
        *m = gemm_matrix_t{data, 1, rows > 0 ? rows : 1, type};
    } else {
        keep->p = t;
        *m = gemm_matrix_t{data, cols > 0 ? cols : 1, 1, type};
    }
    return true;
}

// Raises for a status other than 0.
bool passed(int status, const char *what) {
    if (status == 0) return true;
    PyObject *e = PyObject_CallFunction(g_error, "is", status, what);
    if (e != nullptr) {
        PyErr_SetObject(reinterpret_cast<PyObject *>(Py_TYPE(e)), e);
        Py_DECREF(e);
    }
    return false;
}

bool current_stream(int device, gemm_stream_t *stream) {
    PyObject *d = PyLong_FromLong(device);
    PyObject *s = PyObject_CallOneArg(g_raw_stream, d);
    Py_DECREF(d);
    if (s == nullptr) return false;
    *stream = static_cast<gemm_stream_t>(PyLong_AsVoidPtr(s));
    Py_DECREF(s);
    return !PyErr_Occurred();
}

// The caller's workspace (any CUDA tensor) or one of `need` bytes.
bool workspace(PyObject *given, uint64_t need, int device_index, PyObject *device, Ref *keep, void **data, uint64_t *bytes) {
    *data = nullptr;
    *bytes = 0;
    if (given == Py_None) {
        if (need == 0) return true;
        *bytes = need;
        keep->p = empty({int64_t(need)}, g_uint8, device, data);
        return keep->p != nullptr;
    }
    Tensor t;
    if (!read_tensor(given, &t, "workspace")) return false;
    if (t.device != device_index) {
        PyErr_SetString(PyExc_ValueError, "the workspace is on another device than the tensors");
        return false;
    }
    PyObject *nbytes = PyObject_GetAttrString(given, "nbytes");
    if (nbytes == nullptr) return false;
    *bytes = PyLong_AsUnsignedLongLong(nbytes);
    Py_DECREF(nbytes);
    *data = t.data;
    return !PyErr_Occurred();
}

// The torch.device of a tensor (new reference).
PyObject *device_of(const Tensor &t) { return PyObject_GetAttr(t.obj, g_device_of); }

bool arguments(Py_ssize_t got, Py_ssize_t want) {
    if (got == want) return true;
    PyErr_Format(PyExc_TypeError, "%zd arguments, got %zd", want, got);
    return false;
}

bool operands(const Tensor &A, const Tensor &B) {
    if (!A || !B || A.type < GEMM_TYPE_F16 || A.type != B.type) {
        PyErr_SetString(PyExc_TypeError, "A and B must both be float16, bfloat16 or float8_e4m3fn");
        return false;
    }
    if (A.dims != 2 || B.dims != 2 || A.n[1] != B.n[0]) {
        PyErr_SetString(PyExc_ValueError, "A and B must be matrices whose shapes chain ([M, K] and [K, N])");
        return false;
    }
    return true;
}

bool c_dtype(PyObject *given, int otherwise, int *type, const char *what) {
    *type = given == Py_None ? otherwise : type_code(given);
    if (*type >= GEMM_TYPE_F32 && *type <= GEMM_TYPE_BF16) return true;
    PyErr_Format(PyExc_TypeError, "%s must be float32, float16 or bfloat16", what);
    return false;
}

PyObject *pair_or_first(Ref *first, Ref *second) {
    if (second->p == nullptr) return first->give();
    PyObject *t = PyTuple_New(2);
    if (t == nullptr) return nullptr;
    PyTuple_SET_ITEM(t, 0, first->give());
    PyTuple_SET_ITEM(t, 1, second->give());
    return t;
}

// ------------------------------------------------------------------ entry points
PyObject *py_linear_workspace_size(PyObject *, PyObject *const *a, Py_ssize_t n) {
    Tensor A, B;
    if (!arguments(n, 2) || !read_tensor(a[0], &A, "A") || !read_tensor(a[1], &B, "B") || !operands(A, B)) return nullptr;
    const gemm_matrix_t ma = matrix(A), mb = matrix(B);
    uint64_t need = 0;
    if (!passed(CALL(kLinearSize, gemm_linear_workspace_size)(&ma, &mb, A.n[0], B.n[1], A.n[1], &need), kEntryNames[kLinear]))
        return nullptr;
    return PyLong_FromUnsignedLongLong(need);
}

// (A, B, bias, activation, residual, scale_a, scale_b, out, out_dtype, pre, return_pre, flags, workspace)
PyObject *py_linear(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (!arguments(n, 13)) return nullptr;
    Tensor A, B, bias, res, sa, sb, out, pre;
    if (!read_tensor(a[0], &A, "A") || !read_tensor(a[1], &B, "B") || !operands(A, B) || !read_tensor(a[2], &bias, "bias") ||
        !read_tensor(a[4], &res, "residual") || !read_tensor(a[5], &sa, "scale_a") || !read_tensor(a[6], &sb, "scale_b") ||
        !read_tensor(a[7], &out, "out") || !read_tensor(a[9], &pre, "pre"))
        return nullptr;
    const int64_t M = A.n[0], K = A.n[1], N = B.n[1];
    const bool eight = A.type == GEMM_TYPE_E4M3;
    if (eight != bool(sa) || eight != bool(sb)) {
        PyErr_SetString(PyExc_ValueError, "scale_a and scale_b go with float8_e4m3fn operands, and only with them");
        return nullptr;
    }
    int type = out ? out.type : -1;
    if (out ? !c_dtype(Py_None, type, &type, "C")
            : !c_dtype(a[8], res ? res.type : eight ? GEMM_TYPE_BF16 : A.type, &type, "C"))
        return nullptr;
    if (!same_device(A, {&B, &bias, &res, &sa, &sb, &out, &pre}) || !is_matrix(out, M, N, type, "out") ||
        !is_matrix(res, M, N, type, "residual") || !is_matrix(pre, M, N, type, "pre") ||
        !is_vector(bias, N, GEMM_TYPE_F32, type, "bias") || !is_vector(sa, M, GEMM_TYPE_F32, GEMM_TYPE_F32, "scale_a") ||
        !is_vector(sb, N, GEMM_TYPE_F32, GEMM_TYPE_F32, "scale_b"))
        return nullptr;
    const gemm_matrix_t ma = matrix(A), mb = matrix(B);
    uint64_t need = 0, bytes = 0;
    if (!passed(CALL(kLinearSize, gemm_linear_workspace_size)(&ma, &mb, M, N, K, &need), kEntryNames[kLinear])) return nullptr;
    Ref device, c_ref, pre_ref, ws_ref;
    device.p = device_of(A);
    gemm_matrix_t mc, mp = {nullptr, 1, 1, 0};
    void *ws = nullptr;
    gemm_stream_t stream;
    const bool want_pre = pre || a[10] == Py_True;
    if (device.p == nullptr || !output(out, M, N, type, false, device.p, &c_ref, &mc) ||
        (want_pre && !output(pre, M, N, type, false, device.p, &pre_ref, &mp)) ||
        !workspace(a[12], need, A.device, device.p, &ws_ref, &ws, &bytes) || !current_stream(A.device, &stream))
        return nullptr;
    gemm_epilogue_t ep = {};
    ep.bias = bias.data;
    ep.bias_type = bias ? bias.type : 0;
    ep.activation = int32_t(PyLong_AsLong(a[3]));
    ep.scale_a = static_cast<const float *>(sa.data);
    ep.scale_b = static_cast<const float *>(sb.data);
    ep.residual = matrix(res);
    ep.pre = mp;
    if (!passed(CALL(kLinear, gemm_linear)(&ma, &mb, &mc, &ep, M, N, K, uint32_t(PyLong_AsLong(a[11])), ws, bytes, stream),
                kEntryNames[kLinear]))
        return nullptr;
    return pair_or_first(&c_ref, &pre_ref);
}

// (grad, A, B, pre, activation, need_a, need_b, need_bias, grad_dtype, flags, workspace)
PyObject *py_linear_backward(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (!arguments(n, 11)) return nullptr;
    Tensor G, A, B, pre;
    if (!read_tensor(a[0], &G, "grad") || !read_tensor(a[1], &A, "A") || !read_tensor(a[2], &B, "B") || !operands(A, B) ||
        !read_tensor(a[3], &pre, "pre"))
        return nullptr;
    if (A.type == GEMM_TYPE_E4M3) {
        PyErr_SetString(PyExc_TypeError, "linear_backward takes float16 or bfloat16 operands");
        return nullptr;
    }
    const int64_t M = A.n[0], K = A.n[1], N = B.n[1];
    const int32_t act = int32_t(PyLong_AsLong(a[4]));
    if (act != GEMM_ACT_NONE && !pre) {
        PyErr_SetString(PyExc_ValueError, "with an activation, linear_backward needs pre (linear(..., return_pre=True))");
        return nullptr;
    }
    if (act == GEMM_ACT_NONE) pre = Tensor();
    int type;
    if (!c_dtype(a[8], A.type, &type, "gradients") || !same_device(A, {&B, &G, &pre}) || !is_matrix(G, M, N, A.type, "grad") ||
        !is_matrix(pre, M, N, A.type, "pre"))
        return nullptr;
    if (!G) {
        PyErr_SetString(PyExc_TypeError, "grad must be a torch.Tensor");
        return nullptr;
    }
    const bool need_a = a[5] == Py_True, need_b = a[6] == Py_True, need_bias = a[7] == Py_True;
    const gemm_matrix_t mg = matrix(G), ma = matrix(A), mb = matrix(B), mp = matrix(pre);
    uint64_t need = 0, bytes = 0;
    if (!passed(CALL(kBackwardSize, gemm_linear_backward_workspace_size)(&mg, &ma, &mb, act, need_bias, M, N, K, &need),
                kEntryNames[kBackward]))
        return nullptr;
    Ref device, da_ref, db_ref, bias_ref, ws_ref;
    device.p = device_of(A);
    gemm_matrix_t mda = {nullptr, 1, 1, 0}, mdb = mda;
    void *ws = nullptr, *dbias = nullptr;
    gemm_stream_t stream;
    const Tensor none;
    // gradients are stored as their operands are: by columns where those are
    auto turned = [](const Tensor &t) { return t.s[0] == 1 && t.s[1] != 1 && t.n[0] > 1 && t.n[1] > 1; };
    if (device.p == nullptr || (need_a && !output(none, M, K, type, turned(A), device.p, &da_ref, &mda)) ||
        (need_b && !output(none, K, N, type, turned(B), device.p, &db_ref, &mdb)) ||
        (need_bias && (bias_ref.p = empty({N}, g_dtype[GEMM_TYPE_F32], device.p, &dbias)) == nullptr) ||
        !workspace(a[10], need, A.device, device.p, &ws_ref, &ws, &bytes) || !current_stream(A.device, &stream))
        return nullptr;
    if (!passed(CALL(kBackward, gemm_linear_backward)(&mg, &ma, &mb, &mp, act, &mda, &mdb, static_cast<float *>(dbias), M, N, K,
                                                      uint32_t(PyLong_AsLong(a[9])), ws, bytes, stream),
                kEntryNames[kBackward]))
        return nullptr;
    PyObject *t = PyTuple_New(3);
    if (t == nullptr) return nullptr;
    PyTuple_SET_ITEM(t, 0, da_ref.give());
    PyTuple_SET_ITEM(t, 1, db_ref.give());
    PyTuple_SET_ITEM(t, 2, bias_ref.give());
    return t;
}

// (x, weight, residual, eps, out_dtype, return_rstd, out, h_out) -> (y, h, scale, rstd)
PyObject *py_rms_norm(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (!arguments(n, 8)) return nullptr;
    Tensor x, w, r, out, h;
    if (!read_tensor(a[0], &x, "x") || !read_tensor(a[1], &w, "weight") || !read_tensor(a[2], &r, "residual") ||
        !read_tensor(a[6], &out, "out") || !read_tensor(a[7], &h, "h_out"))
        return nullptr;
    if (!x || !w || x.dims != 2 || x.type < GEMM_TYPE_F32 || x.type > GEMM_TYPE_BF16) {
        PyErr_SetString(PyExc_TypeError, "x must be a float32, float16 or bfloat16 matrix, weight a vector");
        return nullptr;
    }
    const int64_t rows = x.n[0], width = x.n[1];
    const int type = out ? out.type : a[4] == Py_None ? x.type : type_code(a[4]);
    if (type != x.type && type != GEMM_TYPE_E4M3) {
        PyErr_SetString(PyExc_TypeError, "y has x's type or float8_e4m3fn");
        return nullptr;
    }
    const double eps = PyFloat_AsDouble(a[3]);
    if (eps == -1.0 && PyErr_Occurred()) return nullptr;
    if (h && !r) {
        PyErr_SetString(PyExc_ValueError, "h_out goes with a residual: without one h is x");
        return nullptr;
    }
    if (!same_device(x, {&w, &r, &out, &h}) || !is_vector(w, width, GEMM_TYPE_F32, x.type, "weight") ||
        !is_matrix(r, rows, width, x.type, "residual") || !is_matrix(out, rows, width, type, "out") ||
        !is_matrix(h, rows, width, x.type, "h_out"))
        return nullptr;
    Ref device, y_ref, h_ref, scale_ref, rstd_ref;
    device.p = device_of(x);
    gemm_matrix_t my, mh = {nullptr, 1, 1, 0};
    void *scale = nullptr, *rstd = nullptr;
    gemm_stream_t stream;
    if (device.p == nullptr || !output(out, rows, width, type, false, device.p, &y_ref, &my) ||
        (r && !output(h, rows, width, x.type, false, device.p, &h_ref, &mh)) ||
        (type == GEMM_TYPE_E4M3 && (scale_ref.p = empty({rows}, g_dtype[GEMM_TYPE_F32], device.p, &scale)) == nullptr) ||
        (a[5] == Py_True && (rstd_ref.p = empty({rows}, g_dtype[GEMM_TYPE_F32], device.p, &rstd)) == nullptr) ||
        !current_stream(x.device, &stream))
        return nullptr;
    const gemm_matrix_t mx = matrix(x), mr = matrix(r);
    if (!passed(CALL(kNorm, gemm_rms_norm)(&mx, &mr, w.data, w.type, &my, &mh, static_cast<float *>(scale),
                                           static_cast<float *>(rstd), rows, width, float(eps), stream),
                kEntryNames[kNorm]))
        return nullptr;
    PyObject *t = PyTuple_New(4);
    if (t == nullptr) return nullptr;
    PyTuple_SET_ITEM(t, 0, y_ref.give());
    PyTuple_SET_ITEM(t, 1, h_ref.give());
    PyTuple_SET_ITEM(t, 2, scale_ref.give());
    PyTuple_SET_ITEM(t, 3, rstd_ref.give());
    return t;
}

// (grad, h, weight, rstd, grad_h, need_weight, out, workspace) -> (dx, dweight)
PyObject *py_rms_norm_backward(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (!arguments(n, 8)) return nullptr;
    Tensor g, h, w, rstd, gh, out;
    if (!read_tensor(a[0], &g, "grad") || !read_tensor(a[1], &h, "h") || !read_tensor(a[2], &w, "weight") ||
        !read_tensor(a[3], &rstd, "rstd") || !read_tensor(a[4], &gh, "grad_h") || !read_tensor(a[6], &out, "out"))
        return nullptr;
    if (!h || !g || !w || !rstd || h.dims != 2 || h.type < GEMM_TYPE_F32 || h.type > GEMM_TYPE_BF16) {
        PyErr_SetString(PyExc_TypeError, "h must be a float32, float16 or bfloat16 matrix; grad, weight and rstd are needed");
        return nullptr;
    }
    const int64_t rows = h.n[0], width = h.n[1];
    if (!same_device(h, {&g, &w, &rstd, &gh, &out}) || !is_matrix(g, rows, width, h.type, "grad") ||
        !is_matrix(gh, rows, width, h.type, "grad_h") || !is_matrix(out, rows, width, h.type, "out") ||
        !is_vector(w, width, GEMM_TYPE_F32, h.type, "weight") || !is_vector(rstd, rows, GEMM_TYPE_F32, GEMM_TYPE_F32, "rstd"))
        return nullptr;
    const bool need_weight = a[5] == Py_True;
    uint64_t need = 0, bytes = 0;
    if (need_weight &&
        !passed(CALL(kNormBackwardSize, gemm_rms_norm_backward_workspace_size)(rows, width, &need), kEntryNames[kNormBackward]))
        return nullptr;
    Ref device, dx_ref, dw_ref, ws_ref;
    device.p = device_of(h);
    gemm_matrix_t mdx;
    void *ws = nullptr, *dw = nullptr;
    gemm_stream_t stream;
    if (device.p == nullptr || !output(out, rows, width, h.type, false, device.p, &dx_ref, &mdx) ||
        (need_weight && (dw_ref.p = empty({width}, g_dtype[GEMM_TYPE_F32], device.p, &dw)) == nullptr) ||
        !workspace(a[7], need, h.device, device.p, &ws_ref, &ws, &bytes) || !current_stream(h.device, &stream))
        return nullptr;
    const gemm_matrix_t mg = matrix(g), mh = matrix(h), mgh = matrix(gh);
    if (!passed(CALL(kNormBackward, gemm_rms_norm_backward)(&mg, &mh, w.data, w.type, static_cast<const float *>(rstd.data), &mgh,
                                                            &mdx, static_cast<float *>(dw), rows, width, ws, bytes, stream),
                kEntryNames[kNormBackward]))
        return nullptr;
    PyObject *t = PyTuple_New(2);
    if (t == nullptr) return nullptr;
    PyTuple_SET_ITEM(t, 0, dx_ref.give());
    PyTuple_SET_ITEM(t, 1, dw_ref.give());
    return t;
}

// setup({entry name: address}, (float32, float16, bfloat16, float8_e4m3fn), uint8, empty, raw_stream, error)
PyObject *py_setup(PyObject *, PyObject *args) {
    PyObject *entries, *types, *uint8, *empty_fn, *raw, *error;
    if (!PyArg_ParseTuple(args, "O!O!OOOO", &PyDict_Type, &entries, &PyTuple_Type, &types, &uint8, &empty_fn, &raw, &error))
        return nullptr;
    for (int i = 0; i < kEntries; ++i) {
        PyObject *p = PyDict_GetItemString(entries, kEntryNames[i]);
        if (p == nullptr) {
            PyErr_Format(PyExc_KeyError, "%s", kEntryNames[i]);
            return nullptr;
        }
        g_entry[i] = PyLong_AsVoidPtr(p);
        if (PyErr_Occurred()) return nullptr;
    }
    if (PyTuple_GET_SIZE(types) != 4) {
        PyErr_SetString(PyExc_ValueError, "four element types");
        return nullptr;
    }
    for (int i = 0; i < 4; ++i) Py_XSETREF(g_dtype[i], Py_NewRef(PyTuple_GET_ITEM(types, i)));
    Py_XSETREF(g_uint8, Py_NewRef(uint8));
    Py_XSETREF(g_empty, Py_NewRef(empty_fn));
    Py_XSETREF(g_raw_stream, Py_NewRef(raw));
    Py_XSETREF(g_error, Py_NewRef(error));
    Py_RETURN_NONE;
}

template <typename F>
PyCFunction as_function(F *f) { return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)); }

PyMethodDef kMethods[] = {
    {"setup", py_setup, METH_VARARGS, nullptr},
    {"linear_workspace_size", as_function(&py_linear_workspace_size), METH_FASTCALL, nullptr},
    {"linear", as_function(&py_linear), METH_FASTCALL, nullptr},
    {"linear_backward", as_function(&py_linear_backward), METH_FASTCALL, nullptr},
    {"rms_norm", as_function(&py_rms_norm), METH_FASTCALL, nullptr},
    {"rms_norm_backward", as_function(&py_rms_norm_backward), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_native", "Argument marshalling of ops.py.", -1, kMethods, nullptr, nullptr,
                       nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native() {
    s_dtype = PyUnicode_InternFromString("dtype");
    s_shape = PyUnicode_InternFromString("shape");
    s_stride = PyUnicode_InternFromString("stride");
    s_data_ptr = PyUnicode_InternFromString("data_ptr");
    s_get_device = PyUnicode_InternFromString("get_device");
    s_t = PyUnicode_InternFromString("t");
    g_device_of = PyUnicode_InternFromString("device");
    g_kw_empty = Py_BuildValue("(ss)", "dtype", "device");
    if (!s_dtype || !s_shape || !s_stride || !s_data_ptr || !s_get_device || !s_t || !g_device_of || !g_kw_empty) return nullptr;
    return PyModule_Create(&kModule);
}
