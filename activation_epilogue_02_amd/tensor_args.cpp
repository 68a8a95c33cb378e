// tensor_args.cpp -- checks of the tensors that a call of the operators is given, as a Python module
// (_tensor_args).  The kernels see addresses, sizes and row strides only, so a tensor that does not hold what the
// plan says would be read or written out of place.  In Python an attribute of a tensor takes about 0.1 us, and the
// checks of a one-token product's seven operands made its 6.2 us of host time 7.6; here an attribute is a field and the
// call takes 5.6 (the norm of one token: 5.7 without the checks, 6.7 in Python, 5.1).
//
//   matrix(t, rows, cols, ld, dtype, device, what)   a matrix of at least rows x cols values with row stride ld
//   vector(t, count, dtype, device, what)            at least `count` packed values
//   scale_rows(t, rows, ld, device, what)            block scales: rows of ld bytes, packed
//   workspace(t, device, what)                       a packed tensor of any type: (address, bytes)
//   set_error(cls)                                   the exception: cls(status, what)
//
// Each returns the address, and raises cls with the ABI's status for another type (GE_ERR_DTYPE), a tensor that does
// not hold the values (GE_ERR_SHAPE), or one on another device (GE_ERR_HIP).
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../include/gemm_epilog.h"

namespace {

PyObject* g_error;   // GemmEpilogError

PyObject* fail(int status, PyObject* what, const char* more = "") {
    PyObject* text = PyUnicode_FromFormat("%U%s", what, more);
    PyObject* e = text && g_error ? PyObject_CallFunction(g_error, "iO", status, text) : nullptr;
    if (e) PyErr_SetObject(g_error, e);
    else if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, "set_error was not called");
    Py_XDECREF(e);
    Py_XDECREF(text);
    return nullptr;
}

PyObject* address(const at::Tensor& t) { return PyLong_FromVoidPtr(t.data_ptr()); }

// Tensor `arg`, or NULL with a TypeError.
const at::Tensor* tensor(PyObject* arg) {
    if (THPVariable_Check(arg)) return &THPVariable_Unpack(arg);
    PyErr_SetString(PyExc_TypeError, "a torch.Tensor is expected");
    return nullptr;
}

bool count_is(Py_ssize_t n, Py_ssize_t want) {
    if (n == want) return true;
    PyErr_Format(PyExc_TypeError, "%zd arguments are expected", want);
    return false;
}

bool number(PyObject* o, int64_t* v) {
    *v = PyLong_AsLongLong(o);
    return *v != -1 || !PyErr_Occurred();
}

bool dtype(PyObject* o, at::ScalarType* v) {
    if (!THPDtype_Check(o)) {
        PyErr_SetString(PyExc_TypeError, "a torch.dtype is expected");
        return false;
    }
    *v = reinterpret_cast<THPDtype*>(o)->scalar_type;
    return true;
}

bool text(PyObject* o) {
    if (PyUnicode_Check(o)) return true;
    PyErr_SetString(PyExc_TypeError, "a str is expected");
    return false;
}

bool on_device(const at::Tensor& t, int64_t device) {
    return (t.device().is_cpu() ? -1 : t.get_device()) == device;
}

// rows x cols values at row stride ld: a matrix, rows along the first of several dimensions, or packed storage.
bool holds(const at::Tensor& t, int64_t rows, int64_t cols, int64_t ld) {
    if (rows <= 0 || cols <= 0) return true;
    const auto size = t.sizes(), stride = t.strides();
    const int64_t dims = t.dim();
    if (dims == 2)
        return size[0] >= rows && size[1] >= cols && (rows == 1 || stride[0] == ld) && (cols == 1 || stride[1] == 1);
    if (dims > 2 && size[0] >= rows && (rows == 1 || stride[0] == ld)) {
        int64_t inner = 1;   // values of one entry of the first dimension, packed
        for (int64_t i = dims - 1; i > 0; --i) {
            if (size[i] != 1 && stride[i] != inner) return false;
            inner *= size[i];
        }
        return inner >= cols;
    }
    if (!t.is_contiguous() || t.numel() < (rows - 1) * ld + cols) return false;
    if (rows == 1 || dims < 2) return true;
    for (const int64_t s : stride)
        if (s == ld) return true;
    return false;
}

PyObject* vector_of(const at::Tensor& t, int64_t count, int64_t device, PyObject* what) {
    if (t.numel() < count || !t.is_contiguous()) return fail(GE_ERR_SHAPE, what);
    if (!on_device(t, device)) return fail(GE_ERR_HIP, what, " is on another device");
    return address(t);
}

PyObject* matrix(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    int64_t rows, cols, ld, device;
    at::ScalarType type;
    const at::Tensor* t;
    if (!count_is(n, 7) || !(t = tensor(a[0])) || !number(a[1], &rows) || !number(a[2], &cols) || !number(a[3], &ld) ||
        !dtype(a[4], &type) || !number(a[5], &device) || !text(a[6]))
        return nullptr;
    const at::ScalarType got = t->scalar_type();
    // (8-bit codes may come as bytes)
    if (got != type && !(got == at::kByte && type == at::kFloat8_e4m3fn)) return fail(GE_ERR_DTYPE, a[6]);
    if (!holds(*t, rows, cols, ld)) return fail(GE_ERR_SHAPE, a[6]);
    if (!on_device(*t, device)) return fail(GE_ERR_HIP, a[6], " is on another device");
    return address(*t);
    END_HANDLE_TH_ERRORS
}

PyObject* vector(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    int64_t count, device;
    at::ScalarType type;
    const at::Tensor* t;
    if (!count_is(n, 5) || !(t = tensor(a[0])) || !number(a[1], &count) || !dtype(a[2], &type) ||
        !number(a[3], &device) || !text(a[4]))
        return nullptr;
    if (t->scalar_type() != type) return fail(GE_ERR_DTYPE, a[4]);
    return vector_of(*t, count, device, a[4]);
    END_HANDLE_TH_ERRORS
}

PyObject* scale_rows(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    int64_t rows, ld, device;
    const at::Tensor* t;
    if (!count_is(n, 5) || !(t = tensor(a[0])) || !number(a[1], &rows) || !number(a[2], &ld) ||
        !number(a[3], &device) || !text(a[4]))
        return nullptr;
    if (t->scalar_type() != at::kByte && t->scalar_type() != at::kFloat8_e8m0fnu) return fail(GE_ERR_DTYPE, a[4]);
    return vector_of(*t, rows * ld, device, a[4]);
    END_HANDLE_TH_ERRORS
}

PyObject* workspace(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    int64_t device;
    const at::Tensor* t;
    if (!count_is(n, 3) || !(t = tensor(a[0])) || !number(a[1], &device) || !text(a[2])) return nullptr;
    if (!t->is_contiguous()) return fail(GE_ERR_SHAPE, a[2]);
    if (!on_device(*t, device)) return fail(GE_ERR_HIP, a[2], " is on another device");
    return Py_BuildValue("NL", address(*t), (long long)t->nbytes());
    END_HANDLE_TH_ERRORS
}

PyObject* set_error(PyObject*, PyObject* cls) {
    Py_INCREF(cls);
    Py_XDECREF(g_error);
    g_error = cls;
    Py_RETURN_NONE;
}

PyCFunction fast(PyObject* (*f)(PyObject*, PyObject* const*, Py_ssize_t)) { return (PyCFunction)(void (*)(void))f; }

PyMethodDef methods[] = {{"matrix", fast(matrix), METH_FASTCALL, nullptr},
                         {"vector", fast(vector), METH_FASTCALL, nullptr},
                         {"scale_rows", fast(scale_rows), METH_FASTCALL, nullptr},
                         {"workspace", fast(workspace), METH_FASTCALL, nullptr},
                         {"set_error", set_error, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensor_args", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensor_args(void) { return PyModule_Create(&module); }
