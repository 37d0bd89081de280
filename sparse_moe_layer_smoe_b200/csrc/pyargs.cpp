// The Python binding's argument check, natively: arguments(fn, T, ws, ws_bytes, stream, name, tensor, dtype, n,
// ...) returns the tensors' device pointers, then the workspace's pointer and bytes and the stream, as the
// function of the same name in __init__.py does at 0.5 us a tensor. It decides only the regular case (a
// contiguous CUDA tensor of the named type with at least n elements on the current device, an integer, or
// None; a workspace tensor or None, its own size, the current stream); everything else goes to the Python
// function, which refuses or accepts it and explains.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

namespace {

PyObject* g_slow = nullptr;   // the Python function

bool regular(PyObject* t, PyObject* dtype, int64_t n, int device, PyObject** out) {
    if (t == Py_None || PyLong_CheckExact(t)) {
        Py_INCREF(t);
        *out = t;
        return true;
    }
    if (!THPVariable_CheckExact(t) || !PyUnicode_Check(dtype) || PyUnicode_GET_LENGTH(dtype) == 0) return false;
    const at::Tensor& v = THPVariable_Unpack(t);
    c10::ScalarType want;
    switch (PyUnicode_READ_CHAR(dtype, 0)) {   // "bfloat16", "float32", "int32", "uint8"
        case 'b': want = c10::ScalarType::BFloat16; break;
        case 'f': want = c10::ScalarType::Float; break;
        case 'i': want = c10::ScalarType::Int; break;
        case 'u': want = c10::ScalarType::Byte; break;
        default: return false;
    }
    if (v.scalar_type() != want || v.layout() != c10::kStrided || v.numel() < n || !v.is_contiguous() || v.is_neg() ||
        !v.is_cuda() || v.get_device() != device)
        return false;
    *out = PyLong_FromVoidPtr(v.data_ptr());
    return *out != nullptr;
}

constexpr Py_ssize_t kHead = 5;   // fn, T, ws, ws_bytes, stream

PyObject* arguments(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
    try {
        if (nargs >= kHead && (nargs - kHead) % 4 == 0 && args[3] == Py_None && args[4] == Py_None) {
            const int64_t T = PyLong_AsLongLong(args[1]);
            if (T > 0) {
                const int device = (int)c10::cuda::current_device();
                const Py_ssize_t count = (nargs - kHead) / 4;
                PyObject* list = PyList_New(count + 3);
                if (list == nullptr) return nullptr;
                bool ok = true;
                for (Py_ssize_t i = 0; ok && i < count; ++i) {
                    PyObject* const* a = args + kHead + 4 * i;   // name, tensor, dtype, n
                    const int64_t n = PyLong_AsLongLong(a[3]);
                    PyObject* p = nullptr;
                    ok = !(n == -1 && PyErr_Occurred()) && regular(a[1], a[2], n, device, &p);
                    if (ok) PyList_SET_ITEM(list, i, p);
                }
                int64_t bytes = 0;
                if (ok && args[2] != Py_None) {
                    ok = THPVariable_CheckExact(args[2]);
                    if (ok) {
                        const at::Tensor& w = THPVariable_Unpack(args[2]);
                        ok = w.layout() == c10::kStrided && w.is_contiguous() && w.is_cuda() && w.get_device() == device;
                        if (ok) {
                            bytes = w.numel() * (int64_t)w.element_size();
                            PyList_SET_ITEM(list, count, PyLong_FromVoidPtr(w.data_ptr()));
                        }
                    }
                } else if (ok) {
                    PyList_SET_ITEM(list, count, Py_NewRef(Py_None));
                }
                if (ok) {
                    void* stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream();
                    PyList_SET_ITEM(list, count + 1, PyLong_FromLongLong(bytes));
                    PyList_SET_ITEM(list, count + 2, stream ? PyLong_FromVoidPtr(stream) : Py_NewRef(Py_None));
                    return list;
                }
                Py_DECREF(list);
            }
            PyErr_Clear();
        }
    } catch (...) {   // no exception crosses into the interpreter
    }
    return PyObject_Vectorcall(g_slow, args, (size_t)nargs, nullptr);
}

PyObject* use(PyObject*, PyObject* slow) {
    Py_INCREF(slow);
    Py_XSETREF(g_slow, slow);
    Py_RETURN_NONE;
}

PyMethodDef g_methods[] = {
    {"arguments", (PyCFunction)(void (*)(void))arguments, METH_FASTCALL,
     "arguments(fn, T, ws, ws_bytes, stream, name, tensor, dtype, n, ...) -> list"},
    {"use", use, METH_O, "use(function): what decides irregular arguments"},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_pyargs", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__pyargs(void) { return PyModule_Create(&g_module); }
