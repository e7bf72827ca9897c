// Python entry points of the operators that run in a few microseconds
// (k3moe_gate, k3moe_linear, k3moe_layer_routed).  Argument marshalling only,
// like the ctypes wrappers of the other calls, but read from the tensors
// without a Python call each: through ctypes a call cost 10 to 13 us of host
// time, more than most of its kernels take.
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "k3moe.h"

namespace {

decltype(k3moe_gate) *g_gate;
decltype(k3moe_linear) *g_linear;
decltype(k3moe_layer_routed) *g_routed;

const at::Tensor *tensor_of(PyObject *o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

// An address: a tensor's, an integer, or none.
bool address(PyObject *o, void **out) {
    if (o == Py_None) {
        *out = nullptr;
    } else if (const at::Tensor *t = tensor_of(o)) {
        *out = t->data_ptr();
    } else {
        *out = PyLong_AsVoidPtr(o);
        if (PyErr_Occurred()) return false;
    }
    return true;
}

// What an operand's elements are.  bf16 tensors may also be integer ones that
// hold the bits.
enum Kind { kBf16, kFp32, kInt32, kPointer };
bool is(const at::Tensor *t, Kind kind) {
    const at::ScalarType s = t->scalar_type();
    switch (kind) {
        case kBf16: return s == at::kBFloat16 || s == at::kShort || s == at::kUInt16;
        case kFp32: return s == at::kFloat;
        case kInt32: return s == at::kInt;
        default: return s == at::kLong || s == at::kUInt64;
    }
}

// Row distance of a 2-D operand given as a tensor (0: an address or none,
// rows without gaps); -1, which means an invalid argument, when the tensor is
// not `cols` wide with consecutive elements of this kind, or has fewer than
// `n` rows.
int64_t rows(PyObject *o, Kind kind, int64_t n, int64_t cols) {
    const at::Tensor *t = tensor_of(o);
    if (!t) return 0;
    const int64_t dim = t->dim();
    if (dim < 1 || dim > 2 || !is(t, kind) || t->size(dim - 1) != cols || (cols > 1 && t->stride(dim - 1) != 1)) return -1;
    const int64_t have = dim == 1 ? 1 : t->size(0);
    if (have < n) return -1;
    if (have <= 1) return cols;
    return t->stride(0) >= cols ? t->stride(0) : -1;
}

// Whether an operand (a tensor; an address is taken as it is) is contiguous
// with at least n elements of this kind.
bool flat(PyObject *o, Kind kind, int64_t n) {
    const at::Tensor *t = tensor_of(o);
    return !t || (is(t, kind) && t->is_contiguous() && t->numel() >= n);
}

// Whether every tensor among the arguments is in the current device's memory
// (the library runs on that device and takes the addresses as they are).
bool on_device(PyObject *const *a, Py_ssize_t n) {
    int device = -1;
    for (Py_ssize_t i = 0; i < n; ++i)
        if (const at::Tensor *t = tensor_of(a[i])) {
            if (!t->is_cuda()) return false;
            if (device < 0) device = c10::cuda::current_device();
            if (t->device().index() != device) return false;
        }
    return true;
}

bool stream_of(PyObject *o, void **out) {
    if (o == Py_None) {
        *out = c10::cuda::getCurrentCUDAStream().stream();
        return true;
    }
    if (PyLong_Check(o)) {
        *out = PyLong_AsVoidPtr(o);
        return !PyErr_Occurred();
    }
    PyObject *s = PyObject_GetAttrString(o, "cuda_stream");
    if (!s) return false;
    *out = PyLong_AsVoidPtr(s);
    Py_DECREF(s);
    return !PyErr_Occurred();
}

// A descriptor (a ctypes structure); the caller's reference keeps it in place.
template <typename T>
bool descriptor(PyObject *o, const T **out) {
    Py_buffer b;
    if (PyObject_GetBuffer(o, &b, PyBUF_SIMPLE) != 0) return false;
    const bool ok = b.len == (Py_ssize_t)sizeof(T);
    *out = static_cast<const T *>(b.buf);
    PyBuffer_Release(&b);
    if (!ok) PyErr_SetString(PyExc_TypeError, "descriptor of another type");
    return ok;
}

bool int32_of(PyObject *o, int32_t *out) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) return false;
    if (v < INT32_MIN || v > INT32_MAX) {
        PyErr_SetString(PyExc_OverflowError, "T does not fit 32 bits");
        return false;
    }
    *out = (int32_t)v;
    return true;
}

// The workspace's size: as given, or the tensor's.
bool bytes_of(PyObject *ws, PyObject *given, size_t *out) {
    if (given != Py_None) {
        *out = PyLong_AsSize_t(given);
        return !PyErr_Occurred();
    }
    const at::Tensor *t = tensor_of(ws);
    if (!t) {
        PyErr_SetString(PyExc_TypeError, "ws_bytes is needed with a workspace that is not a tensor");
        return false;
    }
    *out = t->nbytes();
    return true;
}
bool holds(PyObject *ws, size_t bytes) {
    const at::Tensor *t = tensor_of(ws);
    return !t || (t->is_contiguous() && t->nbytes() >= bytes);
}

bool count(Py_ssize_t n, Py_ssize_t want) {
    if (n == want) return true;
    PyErr_Format(PyExc_TypeError, "%zd arguments, not %zd", want, n);
    return false;
}

PyObject *status(k3moe_status s) { return PyLong_FromLong(s); }

// The call itself, without the interpreter lock (as ctypes makes it).
template <typename F, typename... A>
PyObject *call(F *f, A... args) {
    k3moe_status s;
    Py_BEGIN_ALLOW_THREADS
    s = f(args...);
    Py_END_ALLOW_THREADS
    return status(s);
}

// (logits, T, bias, gate, idx, weight, stream)
PyObject *gate(PyObject *, PyObject *const *a, Py_ssize_t n) {
    void *logits, *bias, *idx, *weight, *stream;
    const k3moe_gate_desc *d;
    int32_t T;
    if (!count(n, 7) || !address(a[0], &logits) || !int32_of(a[1], &T) || !address(a[2], &bias) || !descriptor(a[3], &d) ||
        !address(a[4], &idx) || !address(a[5], &weight) || !stream_of(a[6], &stream))
        return nullptr;
    const int64_t ld = rows(a[0], d->flags & K3MOE_LOGITS_BF16 ? kBf16 : kFp32, T, d->n_experts), picks = (int64_t)T * d->top_k;
    if (!on_device(a, 6) || ld < 0 || !flat(a[2], kFp32, d->n_experts) || !flat(a[4], kInt32, picks) ||
        !flat(a[5], kFp32, picks))
        return status(K3MOE_ERR_INVALID_ARGUMENT);
    return call(g_gate, logits, ld, T, static_cast<const float *>(bias), d, static_cast<int32_t *>(idx),
                static_cast<float *>(weight), stream);
}

// (x, T, w, w_gate, bias, bias_gate, residual, lin, out, ws, ws_bytes, stream)
PyObject *linear(PyObject *, PyObject *const *a, Py_ssize_t n) {
    void *x, *w, *wg, *b, *bg, *r, *out, *ws, *stream;
    const k3moe_linear_desc *d;
    int32_t T;
    size_t bytes;
    if (!count(n, 12) || !address(a[0], &x) || !int32_of(a[1], &T) || !address(a[2], &w) || !address(a[3], &wg) ||
        !address(a[4], &b) || !address(a[5], &bg) || !address(a[6], &r) || !descriptor(a[7], &d) || !address(a[8], &out) ||
        !address(a[9], &ws) || !bytes_of(a[9], a[10], &bytes) || !stream_of(a[11], &stream))
        return nullptr;
    const Kind kind = d->flags & K3MOE_OUT_FP32 ? kFp32 : kBf16;
    const int64_t ldx = rows(a[0], kBf16, T, d->k), ldw = rows(a[2], kBf16, d->n, d->k), ldr = rows(a[6], kind, T, d->n),
                  ldo = rows(a[8], kind, T, d->n);
    if (!on_device(a, 10) || ldx < 0 || ldw < 0 || ldr < 0 || ldo < 0 || !flat(a[4], kFp32, d->n) ||
        !flat(a[5], kFp32, d->n) || (a[3] != Py_None && rows(a[3], kBf16, d->n, d->k) != ldw) || !holds(a[9], bytes))
        return status(K3MOE_ERR_INVALID_ARGUMENT);
    return call(g_linear, x, ldx, T, w, wg, ldw, static_cast<const float *>(b), static_cast<const float *>(bg), r, ldr, d, out,
                ldo, ws, bytes, stream);
}

// (x, T, idx, weight, expert_blobs, shared_wg, shared_wu, shared_wd, dims, y, ws, ws_bytes, stream)
PyObject *layer_routed(PyObject *, PyObject *const *a, Py_ssize_t n) {
    void *x, *idx, *weight, *blobs, *sg, *su, *sd, *y, *ws, *stream;
    const k3moe_dims *d;
    int32_t T;
    size_t bytes;
    if (!count(n, 13) || !address(a[0], &x) || !int32_of(a[1], &T) || !address(a[2], &idx) || !address(a[3], &weight) ||
        !address(a[4], &blobs) || !address(a[5], &sg) || !address(a[6], &su) || !address(a[7], &sd) ||
        !descriptor(a[8], &d) || !address(a[9], &y) || !address(a[10], &ws) || !bytes_of(a[10], a[11], &bytes) ||
        !stream_of(a[12], &stream))
        return nullptr;
    // The library takes x, y and the shared matrices as dense: a slice of wider
    // rows is refused, not misread.
    const int64_t td = (int64_t)T * d->d, picks = (int64_t)T * d->top_k, mat = (int64_t)d->ff_shared * d->d;
    const bool shared = !(d->flags & K3MOE_NO_SHARED);
    if (!on_device(a, 11) || !flat(a[0], kBf16, td) || !flat(a[2], kInt32, picks) || !flat(a[3], kFp32, picks) ||
        !flat(a[4], kPointer, d->n_experts) ||
        (shared && (!flat(a[5], kBf16, mat) || !flat(a[6], kBf16, mat) || !flat(a[7], kBf16, mat))) ||
        !flat(a[9], d->flags & K3MOE_OUT_FP32 ? kFp32 : kBf16, td) || !holds(a[10], bytes))
        return status(K3MOE_ERR_INVALID_ARGUMENT);
    return call(g_routed, x, T, static_cast<const int32_t *>(idx), static_cast<const float *>(weight),
                static_cast<const uint8_t *const *>(blobs), sg, su, sd, d, y, ws, bytes, stream);
}

// The library's functions, as the package loaded them.
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (!count(n, 3)) return nullptr;
    g_gate = reinterpret_cast<decltype(g_gate)>(PyLong_AsVoidPtr(a[0]));
    g_linear = reinterpret_cast<decltype(g_linear)>(PyLong_AsVoidPtr(a[1]));
    g_routed = reinterpret_cast<decltype(g_routed)>(PyLong_AsVoidPtr(a[2]));
    if (PyErr_Occurred()) return nullptr;
    Py_RETURN_NONE;
}

template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t)>
PyObject *guarded(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    try {
        return F(self, a, n);
    } catch (const std::exception &e) {  // no C++ exception passes into the interpreter
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

PyMethodDef methods[] = {
    {"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(guarded<bind>)), METH_FASTCALL, nullptr},
    {"gate", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(guarded<gate>)), METH_FASTCALL, nullptr},
    {"linear", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(guarded<linear>)), METH_FASTCALL, nullptr},
    {"layer_routed", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(guarded<layer_routed>)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
