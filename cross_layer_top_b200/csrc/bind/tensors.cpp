// What the binding (indexcache.py) does to tensor arguments before a call of
// the drafted-token operators and of ic_qk_norm_rope: checks, pointers, and the
// latter's descriptors.  Through Python's tensor methods that took as long as
// the small calls' kernels, or longer (the descriptors of five tensors 15 us
// there, 1.2 us here; eight arguments' checks 4 us there, 1.5 us here).
//
// Each function handles what is in order and returns None for anything else:
// the binding's Python code then says what is wrong.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <cstring>

#include "indexcache.h"

namespace {

enum { K_X, K_NORM, K_WEIGHT, K_BIAS, K_EPS, K_ROPE, K_INTER, K_OUT, K_OUT8, K_SCALE, K_SLOT, K_N };
const char *const key_names[K_N] = {"x",           "norm", "weight", "bias",      "eps", "rope",
                                           "interleaved", "out",  "out8",   "out_scale", "slot"};
PyObject *keys[K_N];

// The tensor if it has this type and lies on this GPU (contiguous unless
// `strided`), else null.
const at::Tensor *on(PyObject *o, at::ScalarType type, int64_t dev, bool strided = false) {
    if (!THPVariable_Check(o)) return nullptr;
    const at::Tensor &t = THPVariable_Unpack(o);
    const bool ok = t.scalar_type() == type && t.get_device() == dev && !t.is_meta() &&
                    (strided || t.is_contiguous());
    return ok ? &t : nullptr;
}

// Data pointer of a vector of heads[i]; false if it is not in order.
template <class T>
bool vector(PyObject *o, at::ScalarType type, int64_t dev, int64_t numel, const T **out) {
    const at::Tensor *t = on(o, type, dev);
    if (!t || t->numel() != numel) return false;
    *out = static_cast<const T *>(t->data_ptr());
    return true;
}

bool pack_one(PyObject *hd, int64_t dev, ic_head_io *io, int64_t *rows, int64_t *n_pos) {
    PyObject *v[K_N];
    Py_ssize_t known = 0;
    if (!PyDict_CheckExact(hd)) return false;
    for (int k = 0; k < K_N; ++k) {
        v[k] = PyDict_GetItemWithError(hd, keys[k]);
        if (v[k]) ++known;
        else if (PyErr_Occurred()) {
            PyErr_Clear();
            return false;
        }
        if (v[k] == Py_None) v[k] = nullptr;
    }
    if (known != PyDict_GET_SIZE(hd) || !v[K_X] || !v[K_OUT] == !v[K_OUT8]) return false;

    const at::Tensor *x = on(v[K_X], at::kBFloat16, dev, true);
    if (!x || x->dim() != 3) return false;
    const int64_t n = x->size(0), H = x->size(1), d = x->size(2), row = H * d, sr = x->stride(0);
    if (H < 1 || d < 1 || H > INT_MAX || d > INT_MAX || n > INT_MAX) return false;
    if (x->stride(2) != 1 || (x->stride(1) != d && H > 1) || (*rows >= 0 && n != *rows)) return false;
    *rows = n;
    io->x = x->data_ptr();
    io->x_stride = n <= 1 && sr < row ? row : sr;
    io->H = static_cast<int>(H);
    io->d = static_cast<int>(d);

    io->norm = IC_NORM_NONE;
    if (v[K_NORM]) {
        if (!PyUnicode_Check(v[K_NORM])) return false;
        if (PyUnicode_CompareWithASCIIString(v[K_NORM], "rms") == 0) io->norm = IC_NORM_RMS;
        else if (PyUnicode_CompareWithASCIIString(v[K_NORM], "layer") == 0) io->norm = IC_NORM_LAYER;
        else return false;
    }
    io->eps = 1e-6f;
    if (v[K_EPS]) {
        if (!PyFloat_CheckExact(v[K_EPS])) return false;
        io->eps = (float)PyFloat_AS_DOUBLE(v[K_EPS]);
    } else if (PyDict_GetItem(hd, keys[K_EPS])) {
        return false;  // None
    }
    io->interleaved = 0;
    if (v[K_INTER]) {
        if (!PyBool_Check(v[K_INTER])) return false;
        io->interleaved = v[K_INTER] == Py_True;
    }
    if (v[K_WEIGHT] && !vector(v[K_WEIGHT], at::kFloat, dev, d, &io->weight)) return false;
    if (v[K_BIAS] && !vector(v[K_BIAS], at::kFloat, dev, d, &io->bias)) return false;
    if (v[K_ROPE]) {
        const at::Tensor *t = on(v[K_ROPE], at::kFloat, dev);
        if (!t || t->dim() != 2 || t->size(0) > INT_MAX || t->size(1) > INT_MAX ||
            (*n_pos >= 0 && t->size(0) != *n_pos))
            return false;
        *n_pos = t->size(0);
        io->rope = static_cast<const float *>(t->data_ptr());
        io->d_rot = static_cast<int>(t->size(1));
    }
    const at::Tensor *o = v[K_OUT] ? on(v[K_OUT], at::kBFloat16, dev) : on(v[K_OUT8], at::kByte, dev);
    if (!o || o->numel() % row || (!v[K_SLOT] && o->numel() != n * row)) return false;
    if (v[K_OUT])
        io->out = o->data_ptr();
    else
        io->out8 = static_cast<uint8_t *>(o->data_ptr());
    io->out_rows = o->numel() / row;
    const float *scale = nullptr;
    if (v[K_SCALE] && !vector(v[K_SCALE], at::kFloat, dev, o->numel() / d, &scale)) return false;
    io->out_scale = const_cast<float *>(scale);
    return !v[K_SLOT] || vector(v[K_SLOT], at::kLong, dev, n, &io->slot);
}

// pack(heads, device) -> (descriptors as bytes, rows, n_pos), or None
PyObject *pack(PyObject *, PyObject *const *args, Py_ssize_t nargs) {
    if (nargs != 2) {
        PyErr_SetString(PyExc_TypeError, "pack(heads, device)");
        return nullptr;
    }
    const long long dev = PyLong_AsLongLong(args[1]);
    if (dev == -1 && PyErr_Occurred()) return nullptr;
    if (!PyList_CheckExact(args[0])) Py_RETURN_NONE;
    const Py_ssize_t n = PyList_GET_SIZE(args[0]);
    if (n < 1 || n > IC_MAX_HEAD_IO) Py_RETURN_NONE;
    ic_head_io io[IC_MAX_HEAD_IO];
    std::memset(static_cast<void *>(io), 0, sizeof(io));  // padding bytes too
    int64_t rows = -1, n_pos = -1;
    try {
        for (Py_ssize_t i = 0; i < n; ++i)
            if (!pack_one(PyList_GET_ITEM(args[0], i), dev, &io[i], &rows, &n_pos)) Py_RETURN_NONE;
    } catch (...) {  // a tensor without storage, say
        PyErr_Clear();
        Py_RETURN_NONE;
    }
    PyObject *bytes =
        PyBytes_FromStringAndSize(reinterpret_cast<const char *>(io), n * static_cast<Py_ssize_t>(sizeof(io[0])));
    if (!bytes) return nullptr;
    return Py_BuildValue("(Nii)", bytes, static_cast<int>(rows), static_cast<int>(n_pos < 0 ? 0 : n_pos));
}

// ptr(tensor, dtype, device, shape or None) -> data pointer of a contiguous tensor, or None
PyObject *ptr(PyObject *, PyObject *const *args, Py_ssize_t nargs) {
    if (nargs != 4) {
        PyErr_SetString(PyExc_TypeError, "ptr(tensor, dtype, device, shape)");
        return nullptr;
    }
    const long long dev = PyLong_AsLongLong(args[2]);
    if (dev == -1 && PyErr_Occurred()) return nullptr;
    if (!THPDtype_Check(args[1])) Py_RETURN_NONE;
    try {
        const at::Tensor *t = on(args[0], reinterpret_cast<THPDtype *>(args[1])->scalar_type, dev);
        if (!t) Py_RETURN_NONE;
        PyObject *shape = args[3];
        if (shape != Py_None) {
            if (!PyTuple_Check(shape) || PyTuple_GET_SIZE(shape) != t->dim()) Py_RETURN_NONE;
            for (int64_t i = 0; i < t->dim(); ++i) {
                const long long want = PyLong_AsLongLong(PyTuple_GET_ITEM(shape, i));
                if (want == -1 && PyErr_Occurred()) {
                    PyErr_Clear();
                    Py_RETURN_NONE;
                }
                if (want != t->size(i)) Py_RETURN_NONE;
            }
        }
        return PyLong_FromVoidPtr(t->data_ptr());
    } catch (...) {
        PyErr_Clear();
        Py_RETURN_NONE;
    }
}

// cache(tensor, device, B, kv_len, d) -> (data pointer, sequence stride) of a
// cache [B, kv_len, d] whose sequences' rows are contiguous, or None
PyObject *cache(PyObject *, PyObject *const *args, Py_ssize_t nargs) {
    long long v[4];
    if (nargs != 5) {
        PyErr_SetString(PyExc_TypeError, "cache(tensor, device, B, kv_len, d)");
        return nullptr;
    }
    for (int i = 0; i < 4; ++i) {
        v[i] = PyLong_AsLongLong(args[i + 1]);
        if (v[i] == -1 && PyErr_Occurred()) return nullptr;
    }
    const long long B = v[1], n = v[2], d = v[3];
    try {
        const at::Tensor *t = on(args[0], at::kBFloat16, v[0], true);
        if (!t || t->dim() != 3 || t->size(0) != B || t->size(1) != n || t->size(2) != d ||
            t->stride(2) != 1 || (n > 1 && t->stride(1) != d))
            Py_RETURN_NONE;
        return Py_BuildValue("(NL)", PyLong_FromVoidPtr(t->data_ptr()),
                             static_cast<long long>(B > 1 ? t->stride(0) : n * d));
    } catch (...) {
        PyErr_Clear();
        Py_RETURN_NONE;
    }
}

PyMethodDef methods[] = {
    {"ptr", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(ptr)), METH_FASTCALL,
     "data pointer of a contiguous tensor"},
    {"cache", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(cache)), METH_FASTCALL,
     "data pointer and sequence stride of a cache"},
    {"pack", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(pack)), METH_FASTCALL,
     "descriptors of ic_qk_norm_rope"},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensors", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensors(void) {
    for (int k = 0; k < K_N; ++k)
        if (!(keys[k] = PyUnicode_InternFromString(key_names[k]))) return nullptr;
    PyObject *m = PyModule_Create(&module);
    // the torch it was built for: another one's tensors may be laid out differently
    if (m && PyModule_AddStringConstant(m, "torch_version", IC_TORCH_VERSION) < 0) Py_CLEAR(m);
    return m;
}
