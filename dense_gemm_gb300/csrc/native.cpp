// Argument marshalling for ops.py as a CPython extension on PyTorch's C++ API:
// tensors -> gemm_matrix_t, outputs and workspaces allocated, one C call. No
// arithmetic. The smallest kernels take 2 us on the GPU; through ctypes the same
// steps took 20 us a call on the GB300's host, through the tensors' Python
// attributes 7 to 10.
//
// Every function makes the tensors' device and, where one is given, the stream
// current for its call, so that what it allocates belongs to the stream it is
// written on. The library's entry points arrive through setup().
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/Stream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <initializer_list>
#include <optional>

#include "gemm_ops.h"

namespace {

// ------------------------------------------------------------------ what setup() stores
enum Entry {
    kLinear, kLinearSize, kBackward, kBackwardSize, kNorm, kNormBackward, kNormBackwardSize,
    kLayerNorm, kLayerNormBackward, kLayerNormBackwardSize, kQuantize, kSaved, kSavedSize, kEntries
};
const char *const kEntryNames[kEntries] = {"gemm_linear", "gemm_linear_workspace_size", "gemm_linear_backward",
                                           "gemm_linear_backward_workspace_size", "gemm_rms_norm",
                                           "gemm_rms_norm_backward", "gemm_rms_norm_backward_workspace_size",
                                           "gemm_layer_norm", "gemm_layer_norm_backward",
                                           "gemm_layer_norm_backward_workspace_size", "gemm_quantize_rows",
                                           "gemm_saved_backward", "gemm_saved_backward_workspace_size"};
void *g_entry[kEntries];

template <typename F>
F *entry(Entry e, F *) { return reinterpret_cast<F *>(g_entry[e]); }
#define CALL(e, fn) (entry(e, &fn))

PyObject *g_error, *g_norm_result, *g_layer_norm_result;  // GemmError, RmsNormResult, LayerNormResult (owned)

constexpr int kTypeCount = 5;
const char *const kTypeNames[kTypeCount] = {"float32", "float16", "bfloat16", "float8_e4m3fn", "int8"};
const at::ScalarType kTypes[kTypeCount] = {at::kFloat, at::kHalf, at::kBFloat16, at::kFloat8_e4m3fn, at::kChar};

int type_code(at::ScalarType t) {
    for (int i = 0; i < kTypeCount; ++i)
        if (t == kTypes[i]) return i;
    return -1;
}

bool is_eight(int type) { return type == GEMM_TYPE_E4M3 || type == GEMM_TYPE_I8; }

// ------------------------------------------------------------------ tensors
struct Tensor {
    PyObject *obj = nullptr;  // borrowed; nullptr: absent
    void *data = nullptr;
    int64_t n[2] = {0, 0}, s[2] = {1, 1};
    int64_t nbytes = 0;
    int dims = 0;
    int type = -1;  // GEMM_TYPE_*, -1: another one
    int device = -1;
    explicit operator bool() const { return obj != nullptr; }
};

// False with a Python error set. None is an absent tensor.
bool read_tensor(PyObject *o, Tensor *t, const char *what) {
    if (o == Py_None) return true;
    if (!THPVariable_Check(o)) {
        PyErr_Format(PyExc_TypeError, "%s must be a torch.Tensor", what);
        return false;
    }
    const at::Tensor &v = THPVariable_Unpack(o);
    t->obj = o;
    t->dims = int(v.dim());
    for (int i = 0; i < t->dims && i < 2; ++i) {
        t->n[i] = v.size(i);
        t->s[i] = v.stride(i);
    }
    t->type = type_code(v.scalar_type());
    t->device = v.is_cuda() ? int(v.get_device()) : -1;
    if (t->device >= 0) {
        t->data = v.data_ptr();
        t->nbytes = int64_t(v.nbytes());
    }
    return true;
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

// ------------------------------------------------------------------ where a call runs
// The tensors' device and, where one is given, the stream made current.
struct Place {
    std::optional<c10::cuda::CUDAGuard> device;
    std::optional<c10::cuda::CUDAStreamGuard> guard;
    gemm_stream_t stream = nullptr;
    at::TensorOptions options;

    // False with a Python error set.
    bool enter(int index, PyObject *given) {
        options = at::TensorOptions().device(at::Device(at::kCUDA, at::DeviceIndex(index)));
        if (given == Py_None) {
            device.emplace(at::DeviceIndex(index));
            stream = c10::cuda::getCurrentCUDAStream(at::DeviceIndex(index)).stream();
            return true;
        }
        if (!THPStream_Check(given)) {
            PyErr_SetString(PyExc_TypeError, "stream must be a torch.cuda.Stream");
            return false;
        }
        const auto *s = reinterpret_cast<const THPStream *>(given);
        if (s->device_type != int64_t(at::kCUDA) || s->device_index != index) {
            PyErr_Format(PyExc_ValueError, "stream is on device %lld, the tensors on %d", (long long)s->device_index, index);
            return false;
        }
        const auto cs = c10::cuda::CUDAStream::unpack3(s->stream_id, at::DeviceIndex(index), at::kCUDA);
        guard.emplace(cs);
        stream = cs.stream();
        return true;
    }

    // torch.empty on the call's device and stream.
    at::Tensor empty(at::IntArrayRef shape, at::ScalarType type) const { return at::empty(shape, options.dtype(type)); }
};

// The matrix of an output: the given tensor, or a new one stored by rows or (turned) by columns.
struct Output {
    PyObject *given = nullptr;  // borrowed
    at::Tensor made;
    gemm_matrix_t m = {nullptr, 1, 1, 0};

    void set(const Tensor &t, int64_t rows, int64_t cols, int type, bool turned, const Place &place) {
        if (t) {
            given = t.obj;
            m = matrix(t);
            return;
        }
        made = turned ? place.empty({cols, rows}, kTypes[type]).t() : place.empty({rows, cols}, kTypes[type]);
        m = turned ? gemm_matrix_t{made.data_ptr(), 1, rows > 0 ? rows : 1, type}
                   : gemm_matrix_t{made.data_ptr(), cols > 0 ? cols : 1, 1, type};
    }
    void set_vector(int64_t n, const Place &place) {
        made = place.empty({n}, at::kFloat);
        m.data = made.data_ptr();
    }
    float *floats() const { return static_cast<float *>(m.data); }
    // New reference. A tensor that was given has been written: autograd is told, so that a graph that saved
    // its old values refuses them instead of using the new ones.
    PyObject *give() {
        if (given != nullptr) {
            const at::Tensor &t = THPVariable_Unpack(given);
            if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
            return Py_NewRef(given);
        }
        return made.defined() ? THPVariable_Wrap(std::move(made)) : Py_NewRef(Py_None);
    }
};

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

// The caller's workspace (any contiguous CUDA tensor: the bytes of one with strides, or
// expanded, are not all its own) or one of `need` bytes.
struct Workspace {
    at::Tensor made;
    void *data = nullptr;
    uint64_t bytes = 0;

    bool set(PyObject *given, uint64_t need, int device, const Place &place) {
        if (given == Py_None) {
            if (need == 0) return true;
            made = place.empty({int64_t(need)}, at::kByte);
            data = made.data_ptr();
            bytes = need;
            return true;
        }
        Tensor t;
        if (!read_tensor(given, &t, "workspace")) return false;
        if (t.device != device) {
            PyErr_SetString(PyExc_ValueError, "the workspace is on another device than the tensors");
            return false;
        }
        if (!THPVariable_Unpack(given).is_contiguous()) {
            PyErr_SetString(PyExc_ValueError, "the workspace must be a contiguous tensor");
            return false;
        }
        data = t.data;
        bytes = uint64_t(t.nbytes);
        return true;
    }
};

bool arguments(Py_ssize_t got, Py_ssize_t want) {
    if (got == want) return true;
    PyErr_Format(PyExc_TypeError, "%zd arguments, got %zd", want, got);
    return false;
}

bool operands(const Tensor &A, const Tensor &B) {
    if (!A || !B || A.type < GEMM_TYPE_F16 || A.type != B.type) {
        PyErr_SetString(PyExc_TypeError, "A and B must both be float16, bfloat16, float8_e4m3fn or int8");
        return false;
    }
    if (A.dims != 2 || B.dims != 2 || A.n[1] != B.n[0]) {
        PyErr_SetString(PyExc_ValueError, "A and B must be matrices whose shapes chain ([M, K] and [K, N])");
        return false;
    }
    return true;
}

// The type code of a torch.dtype argument; None: `otherwise`. -1: not one of the five.
int dtype_code(PyObject *o, int otherwise) {
    if (o == Py_None) return otherwise;
    return THPDtype_Check(o) ? type_code(reinterpret_cast<const THPDtype *>(o)->scalar_type) : -1;
}

bool is_c_type(int type, const char *what) {
    if (type >= GEMM_TYPE_F32 && type <= GEMM_TYPE_BF16) return true;
    PyErr_Format(PyExc_TypeError, "%s must be float32, float16 or bfloat16", what);
    return false;
}

// A tuple of new references (each taken, also on failure).
PyObject *tuple_of(std::initializer_list<PyObject *> items) {
    PyObject *t = PyTuple_New(Py_ssize_t(items.size()));
    Py_ssize_t i = 0;
    for (PyObject *o : items) {
        if (t == nullptr) Py_XDECREF(o);
        else PyTuple_SET_ITEM(t, i++, o);
    }
    return t;
}

// ------------------------------------------------------------------ entry points
PyObject *py_linear_workspace_size(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    Tensor A, B;
    if (!arguments(n, 2) || !read_tensor(a[0], &A, "A") || !read_tensor(a[1], &B, "B") || !operands(A, B)) return nullptr;
    const gemm_matrix_t ma = matrix(A), mb = matrix(B);
    uint64_t need = 0;
    if (!passed(CALL(kLinearSize, gemm_linear_workspace_size)(&ma, &mb, A.n[0], B.n[1], A.n[1], &need), kEntryNames[kLinear]))
        return nullptr;
    return PyLong_FromUnsignedLongLong(need);
    END_HANDLE_TH_ERRORS
}

// (A, B, bias, activation, residual, scale_a, scale_b, out, out_dtype, pre, return_pre, flags, workspace, stream)
PyObject *py_linear(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!arguments(n, 14)) return nullptr;
    Tensor A, B, bias, res, sa, sb, out, pre;
    if (!read_tensor(a[0], &A, "A") || !read_tensor(a[1], &B, "B") || !operands(A, B) || !read_tensor(a[2], &bias, "bias") ||
        !read_tensor(a[4], &res, "residual") || !read_tensor(a[5], &sa, "scale_a") || !read_tensor(a[6], &sb, "scale_b") ||
        !read_tensor(a[7], &out, "out") || !read_tensor(a[9], &pre, "pre"))
        return nullptr;
    const int64_t M = A.n[0], K = A.n[1], N = B.n[1];
    const bool eight = is_eight(A.type);
    if (eight != bool(sa) || eight != bool(sb)) {
        PyErr_SetString(PyExc_ValueError, "scale_a and scale_b go with float8_e4m3fn and int8 operands, and only with them");
        return nullptr;
    }
    const int type = out ? out.type : dtype_code(a[8], res ? res.type : eight ? GEMM_TYPE_BF16 : A.type);
    if (!is_c_type(type, "C") || !same_device(A, {&B, &bias, &res, &sa, &sb, &out, &pre}) ||
        !is_matrix(out, M, N, type, "out") || !is_matrix(res, M, N, type, "residual") || !is_matrix(pre, M, N, type, "pre") ||
        !is_vector(bias, N, GEMM_TYPE_F32, type, "bias") || !is_vector(sa, M, GEMM_TYPE_F32, GEMM_TYPE_F32, "scale_a") ||
        !is_vector(sb, N, GEMM_TYPE_F32, GEMM_TYPE_F32, "scale_b"))
        return nullptr;
    const gemm_matrix_t ma = matrix(A), mb = matrix(B);
    uint64_t need = 0;
    if (!passed(CALL(kLinearSize, gemm_linear_workspace_size)(&ma, &mb, M, N, K, &need), kEntryNames[kLinear])) return nullptr;
    Place place;
    Workspace ws;
    if (!place.enter(A.device, a[13]) || !ws.set(a[12], need, A.device, place)) return nullptr;
    Output c, p;
    const bool want_pre = pre || a[10] == Py_True;
    c.set(out, M, N, type, false, place);
    if (want_pre) p.set(pre, M, N, type, false, place);
    gemm_epilogue_t ep = {};
    ep.bias = bias.data;
    ep.bias_type = bias ? bias.type : 0;
    ep.activation = int32_t(PyLong_AsLong(a[3]));
    ep.scale_a = static_cast<const float *>(sa.data);
    ep.scale_b = static_cast<const float *>(sb.data);
    ep.residual = matrix(res);
    ep.pre = p.m;
    if (!passed(CALL(kLinear, gemm_linear)(&ma, &mb, &c.m, &ep, M, N, K, uint32_t(PyLong_AsLong(a[11])), ws.data, ws.bytes,
                                           place.stream),
                kEntryNames[kLinear]))
        return nullptr;
    return want_pre ? tuple_of({c.give(), p.give()}) : c.give();
    END_HANDLE_TH_ERRORS
}

// (grad, A, B, pre, activation, need_a, need_b, need_bias, grad_dtype, flags, workspace, stream)
PyObject *py_linear_backward(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!arguments(n, 12)) return nullptr;
    Tensor G, A, B, pre;
    if (!read_tensor(a[0], &G, "grad") || !read_tensor(a[1], &A, "A") || !read_tensor(a[2], &B, "B") || !operands(A, B) ||
        !read_tensor(a[3], &pre, "pre"))
        return nullptr;
    if (is_eight(A.type) || !G) {
        PyErr_SetString(PyExc_TypeError, "linear_backward takes a gradient and float16 or bfloat16 operands (8-bit ones with scale_a)");
        return nullptr;
    }
    const int64_t M = A.n[0], K = A.n[1], N = B.n[1];
    const int32_t act = int32_t(PyLong_AsLong(a[4]));
    if (act != GEMM_ACT_NONE && !pre) {
        PyErr_SetString(PyExc_ValueError, "with an activation, linear_backward needs pre (linear(..., return_pre=True))");
        return nullptr;
    }
    if (act == GEMM_ACT_NONE) pre = Tensor();
    const int type = dtype_code(a[8], A.type);
    if (!is_c_type(type, "gradients") || !same_device(A, {&B, &G, &pre}) || !is_matrix(G, M, N, A.type, "grad") ||
        !is_matrix(pre, M, N, A.type, "pre"))
        return nullptr;
    const bool need_a = a[5] == Py_True, need_b = a[6] == Py_True, need_bias = a[7] == Py_True;
    const gemm_matrix_t mg = matrix(G), ma = matrix(A), mb = matrix(B), mp = matrix(pre);
    uint64_t need = 0;
    if (!passed(CALL(kBackwardSize, gemm_linear_backward_workspace_size)(&mg, &ma, &mb, act, need_bias, M, N, K, &need),
                kEntryNames[kBackward]))
        return nullptr;
    Place place;
    Workspace ws;
    if (!place.enter(A.device, a[11]) || !ws.set(a[10], need, A.device, place)) return nullptr;
    Output da, db, dbias;
    // gradients are stored as their operands are: by columns where those are
    auto turned = [](const Tensor &t) { return t.s[0] == 1 && t.s[1] != 1 && t.n[0] > 1 && t.n[1] > 1; };
    if (need_a) da.set(Tensor(), M, K, type, turned(A), place);
    if (need_b) db.set(Tensor(), K, N, type, turned(B), place);
    if (need_bias) dbias.set_vector(N, place);
    if (!passed(CALL(kBackward, gemm_linear_backward)(&mg, &ma, &mb, &mp, act, &da.m, &db.m, dbias.floats(), M, N, K,
                                                      uint32_t(PyLong_AsLong(a[9])), ws.data, ws.bytes, place.stream),
                kEntryNames[kBackward]))
        return nullptr;
    return tuple_of({da.give(), db.give(), dbias.give()});
    END_HANDLE_TH_ERRORS
}

// Values kept in 8 bits, with a scale for each row.
bool is_kept(const Tensor &t, const Tensor &scale, int64_t rows, const char *what) {
    if (is_eight(t.type) == bool(scale)) return is_vector(scale, rows, GEMM_TYPE_F32, GEMM_TYPE_F32, what);
    PyErr_Format(PyExc_ValueError, "%s goes with float8_e4m3fn or int8 values, and only with them", what);
    return false;
}

// (grad, A, scale_a, activation_a, B, pre, scale_pre, activation, need_a, need_b, need_bias, grad_dtype, flags, workspace, stream)
PyObject *py_saved_backward(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!arguments(n, 15)) return nullptr;
    Tensor G, A, sa, B, pre, sp;
    if (!read_tensor(a[0], &G, "grad") || !read_tensor(a[1], &A, "A") || !read_tensor(a[2], &sa, "scale_a") ||
        !read_tensor(a[4], &B, "B") || !read_tensor(a[5], &pre, "pre") || !read_tensor(a[6], &sp, "scale_pre"))
        return nullptr;
    if (!G || !A || !B || (B.type != GEMM_TYPE_F16 && B.type != GEMM_TYPE_BF16) || (A.type != B.type && !is_eight(A.type))) {
        PyErr_SetString(PyExc_TypeError,
                        "linear_backward takes a gradient, a float16 or bfloat16 B, and an A of B's type, float8_e4m3fn or int8");
        return nullptr;
    }
    if (A.dims != 2 || B.dims != 2 || A.n[1] != B.n[0]) {
        PyErr_SetString(PyExc_ValueError, "A and B must be matrices whose shapes chain ([M, K] and [K, N])");
        return nullptr;
    }
    const int64_t M = A.n[0], K = A.n[1], N = B.n[1];
    const int32_t act_a = int32_t(PyLong_AsLong(a[3])), act = int32_t(PyLong_AsLong(a[7]));
    if (act != GEMM_ACT_NONE && !pre) {
        PyErr_SetString(PyExc_ValueError, "with an activation, linear_backward needs pre (linear(..., return_pre=True), or kept in 8 bits)");
        return nullptr;
    }
    if (act_a != GEMM_ACT_NONE && !sa) {
        PyErr_SetString(PyExc_ValueError, "activation_a goes with an A kept in 8 bits (scale_a)");
        return nullptr;
    }
    if (!is_kept(A, sa, M, "scale_a") || !is_kept(pre, sp, M, "scale_pre")) return nullptr;
    if (act == GEMM_ACT_NONE) pre = sp = Tensor();
    const int type = dtype_code(a[11], B.type);
    if (!is_c_type(type, "gradients") || !same_device(A, {&B, &G, &pre, &sa, &sp}) || !is_matrix(G, M, N, B.type, "grad") ||
        !is_matrix(pre, M, N, sp ? pre.type : B.type, "pre"))
        return nullptr;
    const bool need_a = a[8] == Py_True, need_b = a[9] == Py_True, need_bias = a[10] == Py_True;
    const gemm_matrix_t mg = matrix(G), ma = matrix(A), mb = matrix(B), mp = matrix(pre);
    uint64_t need = 0;
    if (!passed(CALL(kSavedSize, gemm_saved_backward_workspace_size)(&mg, &ma, &mb, act, need_bias, M, N, K, &need), kEntryNames[kSaved]))
        return nullptr;
    Place place;
    Workspace ws;
    if (!place.enter(A.device, a[14]) || !ws.set(a[13], need, A.device, place)) return nullptr;
    Output da, db, dbias;
    // gradients are stored as their operands are: by columns where those are
    auto turned = [](const Tensor &t) { return t.s[0] == 1 && t.s[1] != 1 && t.n[0] > 1 && t.n[1] > 1; };
    if (need_a) da.set(Tensor(), M, K, type, turned(A), place);
    if (need_b) db.set(Tensor(), K, N, type, turned(B), place);
    if (need_bias) dbias.set_vector(N, place);
    if (!passed(CALL(kSaved, gemm_saved_backward)(&mg, &ma, static_cast<const float *>(sa.data), act_a, &mb, &mp,
                                                  static_cast<const float *>(sp.data), act, &da.m, &db.m, dbias.floats(), M, N, K,
                                                  uint32_t(PyLong_AsLong(a[12])), ws.data, ws.bytes, place.stream),
                kEntryNames[kSaved]))
        return nullptr;
    return tuple_of({da.give(), db.give(), dbias.give()});
    END_HANDLE_TH_ERRORS
}

// A named tuple's type filled from new references (each taken, also on failure), as its _make.
PyObject *named_tuple(PyObject *type, std::initializer_list<PyObject *> items) {
    PyObject *t = tuple_of(items);
    if (t == nullptr) return nullptr;
    PyObject *args = tuple_of({t});
    if (args == nullptr) return nullptr;
    PyObject *result = PyTuple_Type.tp_new(reinterpret_cast<PyTypeObject *>(type), args, nullptr);
    Py_DECREF(args);
    return result;
}

// (x, weight, bias, residual, eps, out_dtype, return_stats, out, h_out, stream) -> LayerNormResult
PyObject *py_layer_norm(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!arguments(n, 10)) return nullptr;
    Tensor x, w, b, r, out, h;
    if (!read_tensor(a[0], &x, "x") || !read_tensor(a[1], &w, "weight") || !read_tensor(a[2], &b, "bias") ||
        !read_tensor(a[3], &r, "residual") || !read_tensor(a[7], &out, "out") || !read_tensor(a[8], &h, "h_out"))
        return nullptr;
    if (!x || !w || x.dims != 2 || x.type < GEMM_TYPE_F32 || x.type > GEMM_TYPE_BF16) {
        PyErr_SetString(PyExc_TypeError, "x must be a float32, float16 or bfloat16 matrix, weight a vector");
        return nullptr;
    }
    const int64_t rows = x.n[0], width = x.n[1];
    const int type = out ? out.type : dtype_code(a[5], x.type);
    if (type != x.type && !is_eight(type)) {
        PyErr_SetString(PyExc_TypeError, "y has x's type, float8_e4m3fn or int8");
        return nullptr;
    }
    const double eps = PyFloat_AsDouble(a[4]);
    if (eps == -1.0 && PyErr_Occurred()) return nullptr;
    if (h && !r) {
        PyErr_SetString(PyExc_ValueError, "h_out goes with a residual: without one h is x");
        return nullptr;
    }
    if (!same_device(x, {&w, &b, &r, &out, &h}) || !is_vector(w, width, GEMM_TYPE_F32, x.type, "weight") ||
        !is_vector(b, width, w.type, w.type, "bias") || !is_matrix(r, rows, width, x.type, "residual") ||
        !is_matrix(out, rows, width, type, "out") || !is_matrix(h, rows, width, x.type, "h_out"))
        return nullptr;
    Place place;
    if (!place.enter(x.device, a[9])) return nullptr;
    Output y, sum, scale, mean, rstd;
    y.set(out, rows, width, type, false, place);
    if (r) sum.set(h, rows, width, x.type, false, place);
    if (is_eight(type)) scale.set_vector(rows, place);
    if (a[6] == Py_True) {
        mean.set_vector(rows, place);
        rstd.set_vector(rows, place);
    }
    const gemm_matrix_t mx = matrix(x), mr = matrix(r);
    if (!passed(CALL(kLayerNorm, gemm_layer_norm)(&mx, &mr, w.data, b.data, w.type, &y.m, &sum.m, scale.floats(), mean.floats(),
                                                  rstd.floats(), rows, width, float(eps), place.stream),
                kEntryNames[kLayerNorm]))
        return nullptr;
    return named_tuple(g_layer_norm_result, {y.give(), sum.give(), scale.give(), mean.give(), rstd.give()});
    END_HANDLE_TH_ERRORS
}

// (grad, h, weight, mean, rstd, grad_h, need_weight, need_bias, out, workspace, stream) -> (dx, dweight, dbias)
PyObject *py_layer_norm_backward(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!arguments(n, 11)) return nullptr;
    Tensor g, h, w, mean, rstd, gh, out;
    if (!read_tensor(a[0], &g, "grad") || !read_tensor(a[1], &h, "h") || !read_tensor(a[2], &w, "weight") ||
        !read_tensor(a[3], &mean, "mean") || !read_tensor(a[4], &rstd, "rstd") || !read_tensor(a[5], &gh, "grad_h") ||
        !read_tensor(a[8], &out, "out"))
        return nullptr;
    if (!h || !g || !w || !mean || !rstd || h.dims != 2 || h.type < GEMM_TYPE_F32 || h.type > GEMM_TYPE_BF16) {
        PyErr_SetString(PyExc_TypeError, "h must be a float32, float16 or bfloat16 matrix; grad, weight, mean and rstd are needed");
        return nullptr;
    }
    const int64_t rows = h.n[0], width = h.n[1];
    if (!same_device(h, {&g, &w, &mean, &rstd, &gh, &out}) || !is_matrix(g, rows, width, h.type, "grad") ||
        !is_matrix(gh, rows, width, h.type, "grad_h") || !is_matrix(out, rows, width, h.type, "out") ||
        !is_vector(w, width, GEMM_TYPE_F32, h.type, "weight") || !is_vector(mean, rows, GEMM_TYPE_F32, GEMM_TYPE_F32, "mean") ||
        !is_vector(rstd, rows, GEMM_TYPE_F32, GEMM_TYPE_F32, "rstd"))
        return nullptr;
    const bool need_weight = a[6] == Py_True, need_bias = a[7] == Py_True;
    uint64_t need = 0;
    if ((need_weight || need_bias) &&
        !passed(CALL(kLayerNormBackwardSize, gemm_layer_norm_backward_workspace_size)(rows, width, &need), kEntryNames[kLayerNormBackward]))
        return nullptr;
    Place place;
    Workspace ws;
    if (!place.enter(h.device, a[10]) || !ws.set(a[9], need, h.device, place)) return nullptr;
    Output dx, dw, db;
    dx.set(out, rows, width, h.type, false, place);
    if (need_weight) dw.set_vector(width, place);
    if (need_bias) db.set_vector(width, place);
    const gemm_matrix_t mg = matrix(g), mh = matrix(h), mgh = matrix(gh);
    if (!passed(CALL(kLayerNormBackward, gemm_layer_norm_backward)(&mg, &mh, w.data, w.type, static_cast<const float *>(mean.data),
                                                                   static_cast<const float *>(rstd.data), &mgh, &dx.m, dw.floats(),
                                                                   db.floats(), rows, width, ws.data, ws.bytes, place.stream),
                kEntryNames[kLayerNormBackward]))
        return nullptr;
    return tuple_of({dx.give(), dw.give(), db.give()});
    END_HANDLE_TH_ERRORS
}

// (x, dtype, out, stream) -> (values, scale)
PyObject *py_quantize_rows(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!arguments(n, 4)) return nullptr;
    Tensor x, out;
    if (!read_tensor(a[0], &x, "x") || !read_tensor(a[2], &out, "out")) return nullptr;
    if (!x || x.dims != 2 || x.type < GEMM_TYPE_F32 || x.type > GEMM_TYPE_BF16) {
        PyErr_SetString(PyExc_TypeError, "x must be a float32, float16 or bfloat16 matrix");
        return nullptr;
    }
    const int64_t rows = x.n[0], width = x.n[1];
    const int type = out ? out.type : dtype_code(a[1], GEMM_TYPE_E4M3);
    if (!is_eight(type)) {
        PyErr_SetString(PyExc_TypeError, "rows are quantized to float8_e4m3fn or int8");
        return nullptr;
    }
    if (!same_device(x, {&out}) || !is_matrix(out, rows, width, type, "out")) return nullptr;
    Place place;
    if (!place.enter(x.device, a[3])) return nullptr;
    Output q, scale;
    q.set(out, rows, width, type, false, place);
    scale.set_vector(rows, place);
    const gemm_matrix_t mx = matrix(x);
    if (!passed(CALL(kQuantize, gemm_quantize_rows)(&mx, &q.m, scale.floats(), rows, width, place.stream), kEntryNames[kQuantize]))
        return nullptr;
    return tuple_of({q.give(), scale.give()});
    END_HANDLE_TH_ERRORS
}

// (x, weight, residual, eps, out_dtype, return_rstd, out, h_out, stream) -> RmsNormResult
PyObject *py_rms_norm(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!arguments(n, 9)) return nullptr;
    Tensor x, w, r, out, h;
    if (!read_tensor(a[0], &x, "x") || !read_tensor(a[1], &w, "weight") || !read_tensor(a[2], &r, "residual") ||
        !read_tensor(a[6], &out, "out") || !read_tensor(a[7], &h, "h_out"))
        return nullptr;
    if (!x || !w || x.dims != 2 || x.type < GEMM_TYPE_F32 || x.type > GEMM_TYPE_BF16) {
        PyErr_SetString(PyExc_TypeError, "x must be a float32, float16 or bfloat16 matrix, weight a vector");
        return nullptr;
    }
    const int64_t rows = x.n[0], width = x.n[1];
    const int type = out ? out.type : dtype_code(a[4], x.type);
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
    Place place;
    if (!place.enter(x.device, a[8])) return nullptr;
    Output y, sum, scale, rstd;
    y.set(out, rows, width, type, false, place);
    if (r) sum.set(h, rows, width, x.type, false, place);
    if (type == GEMM_TYPE_E4M3) scale.set_vector(rows, place);
    if (a[5] == Py_True) rstd.set_vector(rows, place);
    const gemm_matrix_t mx = matrix(x), mr = matrix(r);
    if (!passed(CALL(kNorm, gemm_rms_norm)(&mx, &mr, w.data, w.type, &y.m, &sum.m, scale.floats(), rstd.floats(), rows, width,
                                           float(eps), place.stream),
                kEntryNames[kNorm]))
        return nullptr;
    return named_tuple(g_norm_result, {y.give(), sum.give(), scale.give(), rstd.give()});
    END_HANDLE_TH_ERRORS
}

// (grad, h, weight, rstd, grad_h, need_weight, out, workspace, stream) -> (dx, dweight)
PyObject *py_rms_norm_backward(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!arguments(n, 9)) return nullptr;
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
    uint64_t need = 0;
    if (need_weight &&
        !passed(CALL(kNormBackwardSize, gemm_rms_norm_backward_workspace_size)(rows, width, &need), kEntryNames[kNormBackward]))
        return nullptr;
    Place place;
    Workspace ws;
    if (!place.enter(h.device, a[8]) || !ws.set(a[7], need, h.device, place)) return nullptr;
    Output dx, dw;
    dx.set(out, rows, width, h.type, false, place);
    if (need_weight) dw.set_vector(width, place);
    const gemm_matrix_t mg = matrix(g), mh = matrix(h), mgh = matrix(gh);
    if (!passed(CALL(kNormBackward, gemm_rms_norm_backward)(&mg, &mh, w.data, w.type, static_cast<const float *>(rstd.data), &mgh,
                                                            &dx.m, dw.floats(), rows, width, ws.data, ws.bytes, place.stream),
                kEntryNames[kNormBackward]))
        return nullptr;
    return tuple_of({dx.give(), dw.give()});
    END_HANDLE_TH_ERRORS
}

// setup({entry name: address}, GemmError, RmsNormResult, LayerNormResult)
PyObject *py_setup(PyObject *, PyObject *args) {
    PyObject *entries, *error, *norm_result, *layer_norm_result;
    if (!PyArg_ParseTuple(args, "O!OOO", &PyDict_Type, &entries, &error, &norm_result, &layer_norm_result)) return nullptr;
    for (int i = 0; i < kEntries; ++i) {
        PyObject *p = PyDict_GetItemString(entries, kEntryNames[i]);
        if (p == nullptr) {
            PyErr_Format(PyExc_KeyError, "%s", kEntryNames[i]);
            return nullptr;
        }
        g_entry[i] = PyLong_AsVoidPtr(p);
        if (PyErr_Occurred()) return nullptr;
    }
    Py_XSETREF(g_error, Py_NewRef(error));
    Py_XSETREF(g_norm_result, Py_NewRef(norm_result));
    Py_XSETREF(g_layer_norm_result, Py_NewRef(layer_norm_result));
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
    {"layer_norm", as_function(&py_layer_norm), METH_FASTCALL, nullptr},
    {"layer_norm_backward", as_function(&py_layer_norm_backward), METH_FASTCALL, nullptr},
    {"quantize_rows", as_function(&py_quantize_rows), METH_FASTCALL, nullptr},
    {"saved_backward", as_function(&py_saved_backward), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_native", "Argument marshalling of ops.py.", -1, kMethods, nullptr, nullptr,
                       nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native() { return PyModule_Create(&kModule); }
