// binding.cpp -- the Python binding's look at a call's tensors, natively.
//
// A call that is over on the GPU in three microseconds takes up to thirteen tensors, and asking each for its
// type, shape, device, layout and pointer from Python costs half a microsecond. The functions here
// answer for all tensors of a call at once, or with None where something is not as it has to be; the caller
// then asks one by one and says what. They keep nothing, touch no data and launch nothing.
#include <Python.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

namespace {

// A tensor of this type on this device, or null.
const at::Tensor* tensor_of(PyObject* o, PyObject* dtype, long dev) {
    if (!THPVariable_Check(o)) return nullptr;
    const at::Tensor& t = THPVariable_Unpack(o);
    if (t.layout() != at::kStrided || t.scalar_type() != reinterpret_cast<THPDtype*>(dtype)->scalar_type || t.get_device() != dev) return nullptr;
    return &t;
}

// pointers(spec, dev, dims, tensor, ...): the device pointers of contiguous tensors (None for None). spec holds
// (name, dtype, axes) for each; axis i has dims[i] entries.
PyObject* pointers(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (n < 3 || !PyTuple_Check(args[0]) || !PyTuple_Check(args[2]) || PyTuple_GET_SIZE(args[0]) != n - 3) {
        PyErr_SetString(PyExc_TypeError, "pointers(spec, dev, dims, tensor, ...)");
        return nullptr;
    }
    const long dev = PyLong_AsLong(args[1]);
    const Py_ssize_t n_dims = PyTuple_GET_SIZE(args[2]);
    int64_t dims[16];
    if (n_dims > 16) Py_RETURN_NONE;
    for (Py_ssize_t i = 0; i < n_dims; ++i) dims[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(args[2], i));
    if (PyErr_Occurred()) return nullptr;
    PyObject* out = PyTuple_New(n - 3);
    if (!out) return nullptr;
    for (Py_ssize_t i = 0; i < n - 3; ++i) {
        PyObject* o = args[3 + i];
        PyObject* p = nullptr;
        if (o == Py_None) {
            Py_INCREF(o);
            p = o;
        } else {
            PyObject* want = PyTuple_GET_ITEM(args[0], i);
            PyObject* axes = PyTuple_GET_ITEM(want, 2);
            const at::Tensor* t = tensor_of(o, PyTuple_GET_ITEM(want, 1), dev);
            bool fits = t && t->dim() == PyTuple_GET_SIZE(axes) && t->is_contiguous();
            for (Py_ssize_t k = 0; fits && k < t->dim(); ++k) fits = t->size(k) == dims[PyLong_AsLong(PyTuple_GET_ITEM(axes, k))];
            if (!fits) {
                Py_DECREF(out);
                Py_RETURN_NONE;
            }
            p = PyLong_FromVoidPtr(t->data_ptr());
            if (!p) {
                Py_DECREF(out);
                return nullptr;
            }
        }
        PyTuple_SET_ITEM(out, i, p);
    }
    return out;
}

// caches(k_cache, v_cache, dtype, dev, heads, d): (page size, pages, the three strides, k's and v's pointer).
PyObject* caches(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (n != 6) {
        PyErr_SetString(PyExc_TypeError, "caches(k_cache, v_cache, dtype, dev, heads, d)");
        return nullptr;
    }
    const long dev = PyLong_AsLong(args[3]), heads = PyLong_AsLong(args[4]), d = PyLong_AsLong(args[5]);
    if (PyErr_Occurred()) return nullptr;
    const at::Tensor* k = tensor_of(args[0], args[2], dev);
    const at::Tensor* v = tensor_of(args[1], args[2], dev);
    if (!k || !v || k->dim() != 4 || k->sizes() != v->sizes() || k->strides() != v->strides() || k->size(2) != heads ||
        k->size(3) != d || k->stride(3) != 1)
        Py_RETURN_NONE;
    return Py_BuildValue("LLLLLKK", (long long)k->size(1), (long long)k->size(0), (long long)k->stride(0), (long long)k->stride(1),
                         (long long)k->stride(2), (unsigned long long)k->data_ptr(), (unsigned long long)v->data_ptr());
}

// tokens(dtype, dev, B, T, d, tensor, heads, ...): for each [B, T, heads, d] its stride from token to token (its heads
// contiguous within one) and its pointer.
PyObject* tokens(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (n < 5 || (n - 5) % 2) {
        PyErr_SetString(PyExc_TypeError, "tokens(dtype, dev, B, T, d, tensor, heads, ...)");
        return nullptr;
    }
    const long dev = PyLong_AsLong(args[1]);
    const int64_t B = PyLong_AsLongLong(args[2]), T = PyLong_AsLongLong(args[3]), d = PyLong_AsLongLong(args[4]);
    if (PyErr_Occurred()) return nullptr;
    PyObject* out = PyTuple_New(n - 5);
    if (!out) return nullptr;
    for (Py_ssize_t i = 5; i < n; i += 2) {
        const int64_t H = PyLong_AsLongLong(args[i + 1]);
        const at::Tensor* t = tensor_of(args[i], args[0], dev);
        int64_t st = 0;
        bool fits = t && t->dim() == 4 && t->size(0) == B && t->size(1) == T && t->size(2) == H && t->size(3) == d;
        if (fits) {
            st = T != 1 ? t->stride(1) : B > 1 ? t->stride(0) : H * d;
            fits = t->stride(3) == 1 && (H <= 1 || t->stride(2) == d) && (B <= 1 || t->stride(0) == T * st);
        }
        PyObject* a = fits ? PyLong_FromLongLong(st) : nullptr;
        PyObject* b = a ? PyLong_FromVoidPtr(t->data_ptr()) : nullptr;
        if (!b) {
            Py_XDECREF(a);
            Py_DECREF(out);
            if (PyErr_Occurred()) return nullptr;
            Py_RETURN_NONE;
        }
        PyTuple_SET_ITEM(out, i - 5, a);
        PyTuple_SET_ITEM(out, i - 4, b);
    }
    return out;
}

// No exception of libtorch's leaves this file: whatever it did not like is looked at again, one by one.
template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject* self, PyObject* const* args, Py_ssize_t n) {
    try {
        return F(self, args, n);
    } catch (...) {
        PyErr_Clear();
        Py_RETURN_NONE;
    }
}

PyMethodDef kMethods[] = {
    {"pointers", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(guarded<pointers>)), METH_FASTCALL, nullptr},
    {"caches", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(guarded<caches>)), METH_FASTCALL, nullptr},
    {"tokens", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(guarded<tokens>)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// built_for: the versions of PyTorch and Python whose headers this was compiled with; the importer compares them.
PyMODINIT_FUNC PyInit__binding() {
    PyObject* m = PyModule_Create(&kModule);
    if (m && PyModule_AddStringConstant(m, "built_for", GDN_BUILT_FOR) < 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
