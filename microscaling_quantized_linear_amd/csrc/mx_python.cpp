// mx_python.cpp -- the Python binding's compiled call path: one function for each entry
// point that a decoding step calls every few microseconds and that takes up to 27
// arguments (ctypes needs about 0.1 us for each).  It marshals arguments only: numbers
// by the C prototype, tensors to device pointers after the check that they lie on the
// current GPU, stream None to torch's current stream.
//
// The entry point's address comes with each call (the library that is loaded holds
// it), so this module is linked against nothing of the library's; include/mx.h gives the
// prototypes.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <climits>
#include <cstdint>
#include <tuple>
#include <type_traits>
#include <utility>

#include "../../include/mx.h"

namespace {

PyObject *s_get_device, *s_data_ptr, *s_device, *s_cuda_stream;   // interned names
PyObject *torch_device, *torch_stream;       // torch._C's functions, when first needed

bool torch_functions() {
    if (torch_stream) return true;
    PyObject *m = PyImport_ImportModule("torch._C");
    if (!m) return false;
    PyObject *d = PyObject_GetAttrString(m, "_cuda_getDevice");
    PyObject *s = d ? PyObject_GetAttrString(m, "_cuda_getCurrentRawStream") : nullptr;
    Py_DECREF(m);
    if (!s) {
        Py_XDECREF(d);
        return false;
    }
    torch_device = d;
    torch_stream = s;
    return true;
}

// a number that Python holds as a new reference, taken and released
bool take(PyObject *v, long long &out) {
    if (!v) return false;
    out = PyLong_AsLongLong(v);
    Py_DECREF(v);
    return !(out == -1 && PyErr_Occurred());
}
bool take(PyObject *v, uintptr_t &out) {
    if (!v) return false;
    out = (uintptr_t)PyLong_AsUnsignedLongLong(v);
    Py_DECREF(v);
    return !(out == (uintptr_t)-1 && PyErr_Occurred());
}

struct Args {
    long long device = -1;                   // the current one, when it was asked for

    bool current() {
        return device >= 0 || (torch_functions() && take(PyObject_CallNoArgs(torch_device), device));
    }

    bool get(PyObject *o, int &out) {
        const long v = PyLong_AsLong(o);
        if (v == -1 && PyErr_Occurred()) return false;
        if (v < INT_MIN || v > INT_MAX) {
            PyErr_SetString(PyExc_OverflowError, "an argument does not fit a C int");
            return false;
        }
        out = (int)v;
        return true;
    }
    bool get(PyObject *o, int64_t &out) {
        out = PyLong_AsLongLong(o);
        return !(out == -1 && PyErr_Occurred());
    }
    bool get(PyObject *o, size_t &out) {
        out = PyLong_AsSize_t(o);
        return !(out == (size_t)-1 && PyErr_Occurred());
    }
    bool get(PyObject *o, float &out) {
        const double v = PyFloat_AsDouble(o);
        if (v == -1.0 && PyErr_Occurred()) return false;
        out = (float)v;
        return true;
    }
    // None, an address, or a tensor of the current GPU
    bool address(PyObject *o, uintptr_t &out) {
        out = 0;
        if (o == Py_None) return true;
        if (PyLong_Check(o)) {
            out = (uintptr_t)PyLong_AsUnsignedLongLong(o);
            return !(out == (uintptr_t)-1 && PyErr_Occurred());
        }
        long long at;
        if (!take(PyObject_CallMethodNoArgs(o, s_get_device), at)) return false;
        if (at >= 0 && !current()) return false;
        if (at < 0 || at != device) {
            if (PyObject *d = PyObject_GetAttr(o, s_device)) {
                PyErr_Format(PyExc_ValueError, "a tensor is on %S, not on the current GPU", d);
                Py_DECREF(d);
            }
            return false;
        }
        return take(PyObject_CallMethodNoArgs(o, s_data_ptr), out);
    }
    template <class T>
    bool get(PyObject *o, T *&out) {
        uintptr_t v;
        if (!address(o, v)) return false;
        out = reinterpret_cast<T *>(v);
        return true;
    }
    // None: torch's current stream; an address; or an object with cuda_stream
    bool get(PyObject *o, mx_stream_t &out) {
        uintptr_t v = 0;
        if (o == Py_None) {
            if (!current()) return false;
            PyObject *d = PyLong_FromLongLong(device);
            const bool ok = d && take(PyObject_CallOneArg(torch_stream, d), v);
            Py_XDECREF(d);
            if (!ok) return false;
        } else if (PyLong_Check(o)) {
            v = (uintptr_t)PyLong_AsUnsignedLongLong(o);
            if (v == (uintptr_t)-1 && PyErr_Occurred()) return false;
        } else if (!take(PyObject_GetAttr(o, s_cuda_stream), v)) {
            return false;
        }
        out = reinterpret_cast<mx_stream_t>(v);
        return true;
    }
};

// f(address of the entry point, its arguments ...) -> status
template <class F>
struct Entry;
template <class... A>
struct Entry<mx_status (*)(A...)> {
    static PyObject *call(PyObject *, PyObject *const *args, Py_ssize_t n) {
        if (n != (Py_ssize_t)sizeof...(A) + 1) {
            PyErr_Format(PyExc_TypeError, "%d arguments expected", (int)sizeof...(A) + 1);
            return nullptr;
        }
        const uintptr_t f = (uintptr_t)PyLong_AsUnsignedLongLong(args[0]);
        if (f == 0 || PyErr_Occurred()) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "no entry point");
            return nullptr;
        }
        return go(reinterpret_cast<mx_status (*)(A...)>(f), args + 1, std::index_sequence_for<A...>{});
    }
    template <size_t... I>
    static PyObject *go(mx_status (*f)(A...), PyObject *const *args, std::index_sequence<I...>) {
        std::tuple<std::remove_const_t<A>...> v;
        Args a;
        if (!(a.get(args[I], std::get<I>(v)) && ...)) return nullptr;
        mx_status st;
        Py_BEGIN_ALLOW_THREADS
        st = f(std::get<I>(v)...);
        Py_END_ALLOW_THREADS
        return PyLong_FromLong((long)st);
    }
};

#define ENTRY(name)                                                                         \
    {#name,                                                                                 \
     reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&Entry<decltype(&name)>::call)), \
     METH_FASTCALL, nullptr}
PyMethodDef methods[] = {ENTRY(mx_linear_epilogue), ENTRY(mx_moe_route), ENTRY(mx_block_norm),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_mxcall", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__mxcall() {
    s_get_device = PyUnicode_InternFromString("get_device");
    s_data_ptr = PyUnicode_InternFromString("data_ptr");
    s_device = PyUnicode_InternFromString("device");
    s_cuda_stream = PyUnicode_InternFromString("cuda_stream");
    if (!s_get_device || !s_data_ptr || !s_device || !s_cuda_stream) return nullptr;
    return PyModule_Create(&module);
}
