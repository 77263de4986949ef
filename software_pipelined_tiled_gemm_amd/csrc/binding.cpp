// Call path of the Python wrappers for torch tensors: checks the tensors and calls a C entry
// point of libspgemm in one step.
//
// The wrappers' checks in Python read five attributes of every tensor, 2.5 to 3 us a call:
// as much as the launch itself (about 3.3 us), and for one token more than the kernel hides
// behind.  Here the tensors are read through the DLPack C exchange API that torch exposes
// (torch.Tensor.__dlpack_c_exchange_api__), a table of C functions with a stable layout; no
// torch library is linked.  A tensor that is not what the plan expects, a raw pointer or a
// tensor subclass makes the call return -1 before anything is launched, and the wrapper then
// takes its Python path, which raises the error or makes the call.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/dlpack.h>

#include <stdint.h>

namespace {

const DLPackExchangeAPI* g_api = nullptr;
PyTypeObject* g_types[2] = {nullptr, nullptr};   // torch.Tensor, torch.nn.Parameter

// What a plan expects of one tensor (packed by the wrapper with struct "4i2q")
struct Spec {
    int32_t code, bits, ndim, unused;
    int64_t dim[2];
};

// The tensor behind `o`; false with no Python error set if it is not one that can be read here
bool view(PyObject* o, DLTensor* t) {
    if (Py_TYPE(o) != g_types[0] && Py_TYPE(o) != g_types[1]) return false;
    if (g_api->dltensor_from_py_object_no_sync(o, t) != 0) {
        PyErr_Clear();
        return false;
    }
    return t->device.device_type == kDLROCM || t->device.device_type == kDLCUDA;
}

bool dense(const DLTensor& t) {
    if (!t.strides) return true;
    int64_t want = 1;
    for (int i = t.ndim - 1; i >= 0; --i) {
        if (t.shape[i] == 0) return true;
        if (t.shape[i] != 1 && t.strides[i] != want) return false;
        want *= t.shape[i];
    }
    return true;
}

void* data_of(const DLTensor& t) { return (char*)t.data + t.byte_offset; }

bool typed(const DLTensor& t, int code, int bits) {
    return t.dtype.code == code && t.dtype.bits == bits && t.dtype.lanes == 1;
}

// The caller's stream (an int) or, for None, torch's current one
bool stream_of(PyObject* o, const DLDevice& d, void** s) {
    if (o == Py_None) {
        if (g_api->current_work_stream(d.device_type, d.device_id, s) == 0) return true;
        PyErr_Clear();
        return false;
    }
    if (!PyLong_CheckExact(o)) return false;
    *s = PyLong_AsVoidPtr(o);
    return !PyErr_Occurred() || (PyErr_Clear(), false);
}

typedef int (*Fn6)(void*, void*, void*, void*, void*, void*, void*, void*, int64_t, void*);
typedef int (*Fn7)(void*, void*, void*, void*, void*, void*, void*, void*, void*, int64_t, void*);
typedef int (*Fn9)(void*, void*, void*, void*, void*, void*, void*, void*, void*, void*, void*, int64_t, void*);

// run(fn, handle, specs, tensors, workspace, stream) -> status, or -1: nothing called
PyObject* run(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 6) {
        PyErr_SetString(PyExc_TypeError, "run takes 6 arguments");
        return nullptr;
    }
    void* fn = PyLong_AsVoidPtr(a[0]);
    void* h = PyLong_AsVoidPtr(a[1]);
    if (PyErr_Occurred()) return nullptr;
    const Py_ssize_t m = PyTuple_CheckExact(a[3]) ? PyTuple_GET_SIZE(a[3]) : -1;
    if (!PyBytes_CheckExact(a[2]) || (m != 6 && m != 7 && m != 9) ||
        PyBytes_GET_SIZE(a[2]) != m * (Py_ssize_t)sizeof(Spec)) {
        PyErr_SetString(PyExc_TypeError, "run: 6, 7 or 9 tensors and a spec for each");
        return nullptr;
    }
    const Spec* spec = (const Spec*)PyBytes_AS_STRING(a[2]);
    void* p[9];
    DLDevice dev{kDLCPU, -1};
    DLTensor t;
    for (Py_ssize_t i = 0; i < m; ++i) {
        PyObject* o = PyTuple_GET_ITEM(a[3], i);
        if (o == Py_None) {
            p[i] = nullptr;
            continue;
        }
        const Spec& s = spec[i];
        if (!view(o, &t) || !typed(t, s.code, s.bits) || t.ndim != s.ndim) return PyLong_FromLong(-1);
        for (int d = 0; d < s.ndim; ++d)
            if (t.shape[d] != s.dim[d]) return PyLong_FromLong(-1);
        if (!dense(t)) return PyLong_FromLong(-1);
        if (dev.device_id < 0) dev = t.device;
        else if (dev.device_id != t.device.device_id) return PyLong_FromLong(-1);
        p[i] = data_of(t);
    }
    if (dev.device_id < 0) return PyLong_FromLong(-1);
    void* ws = nullptr;
    int64_t bytes = 0;
    if (a[4] != Py_None) {
        if (!view(a[4], &t) || !dense(t) || t.device.device_id != dev.device_id) return PyLong_FromLong(-1);
        ws = data_of(t);
        bytes = (t.dtype.bits * t.dtype.lanes) / 8;
        for (int d = 0; d < t.ndim; ++d) bytes *= t.shape[d];
    }
    void* st = nullptr;
    if (!stream_of(a[5], dev, &st)) return PyLong_FromLong(-1);
    int r;
    if (m == 6) r = ((Fn6)fn)(h, p[0], p[1], p[2], p[3], p[4], p[5], ws, bytes, st);
    else if (m == 7) r = ((Fn7)fn)(h, p[0], p[1], p[2], p[3], p[4], p[5], p[6], ws, bytes, st);
    else r = ((Fn9)fn)(h, p[0], p[1], p[2], p[3], p[4], p[5], p[6], p[7], p[8], ws, bytes, st);
    return PyLong_FromLong(r);
}

typedef int (*FnRows)(const void*, int, int64_t, int64_t, void*, void*, void*);

// rows(fn, X, A, scale, stream) -> status of gemm_quantize_rows, or -1: nothing called
PyObject* rows(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 5) {
        PyErr_SetString(PyExc_TypeError, "rows takes 5 arguments");
        return nullptr;
    }
    void* fn = PyLong_AsVoidPtr(a[0]);
    if (PyErr_Occurred()) return nullptr;
    DLTensor x, q, s;
    if (!view(a[1], &x) || !view(a[2], &q) || !view(a[3], &s)) return PyLong_FromLong(-1);
    const int type = typed(x, kDLFloat, 16) ? 0 : typed(x, kDLBfloat, 16) ? 1 : typed(x, kDLFloat, 32) ? 2 : -1;
    if (type < 0 || x.ndim < 1 || !dense(x) || !typed(q, kDLInt, 8) || q.ndim != x.ndim || !dense(q) ||
        !typed(s, kDLFloat, 32) || s.ndim != x.ndim - 1 || !dense(s) || q.device.device_id != x.device.device_id ||
        s.device.device_id != x.device.device_id)
        return PyLong_FromLong(-1);
    int64_t m = 1;
    for (int d = 0; d < x.ndim; ++d) {
        if (q.shape[d] != x.shape[d] || (d < s.ndim && s.shape[d] != x.shape[d])) return PyLong_FromLong(-1);
        if (d < s.ndim) m *= x.shape[d];
    }
    void* st = nullptr;
    if (!stream_of(a[4], x.device, &st)) return PyLong_FromLong(-1);
    return PyLong_FromLong(((FnRows)fn)(data_of(x), type, m, x.shape[x.ndim - 1], data_of(q), data_of(s), st));
}

// setup(exchange API capsule, Tensor, Parameter) -> whether the table can be used
PyObject* setup(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 3 || !PyType_Check(a[1]) || !PyType_Check(a[2])) {
        PyErr_SetString(PyExc_TypeError, "setup(capsule, Tensor, Parameter)");
        return nullptr;
    }
    const DLPackExchangeAPI* api = (const DLPackExchangeAPI*)PyCapsule_GetPointer(a[0], "dlpack_exchange_api");
    if (!api) {   // not the interface this file knows
        PyErr_Clear();
        Py_RETURN_FALSE;
    }
    if (api->header.version.major != DLPACK_MAJOR_VERSION || !api->dltensor_from_py_object_no_sync ||
        !api->current_work_stream)
        Py_RETURN_FALSE;
    Py_INCREF(a[1]);   // kept for the life of the process, as the module is
    Py_INCREF(a[2]);
    g_types[0] = (PyTypeObject*)a[1];
    g_types[1] = (PyTypeObject*)a[2];
    g_api = api;
    Py_RETURN_TRUE;
}

PyMethodDef g_methods[] = {
    {"setup", (PyCFunction)(void (*)(void))setup, METH_FASTCALL, nullptr},
    {"run", (PyCFunction)(void (*)(void))run, METH_FASTCALL, nullptr},
    {"rows", (PyCFunction)(void (*)(void))rows, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls(void) { return PyModule_Create(&g_module); }
