// The training calls of the Python binding, natively: checking the tensors and calling libstepmoe here takes
// about 0.5 us where the Python functions of the same names (__init__.py) and ctypes take 3. As with ctypes
// the interpreter lock is released meanwhile: a launch may block (a full queue, a host callback). Only the
// regular case is decided here: contiguous CUDA tensors of the right types with at least the elements the
// call touches, on the current device (or integers and None in their places), T > 0, a workspace tensor of
// its own size, the current stream. Everything else returns None, and the Python function checks, explains
// and calls. A regular call returns the library's status.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/stepmoe.h"

namespace {

constexpr auto BF16 = c10::ScalarType::BFloat16;
constexpr auto F32 = c10::ScalarType::Float;
constexpr auto I32 = c10::ScalarType::Int;
constexpr auto U8 = c10::ScalarType::Byte;

// The library's functions, as Python loaded it.
decltype(&smoe_expert_ffn_save) g_expert_ffn_save;
decltype(&smoe_checkpoint_values) g_checkpoint_values;
decltype(&smoe_combine_backward) g_combine_backward;
decltype(&smoe_route_backward) g_route_backward;
decltype(&smoe_expert_ffn_backward) g_expert_ffn_backward;
decltype(&smoe_permute_backward) g_permute_backward;

// One call's arguments; `ok` turns false at the first that is not regular.
struct Call {
    bool ok = false;
    Py_buffer buffer{};
    const smoe_config_t* cfg = nullptr;
    int64_t T = 0, H = 0, E = 0, I = 0, R = 0;   // R = T * top_k
    int device = 0;
    void* ws = nullptr;
    size_t ws_bytes = 0;
    void* stream = nullptr;

    Call(PyObject* c, PyObject* tokens, PyObject* workspace, PyObject* bytes, PyObject* given_stream) {
        if (given_stream != Py_None || bytes != Py_None || !PyLong_CheckExact(tokens)) return;
        T = PyLong_AsLongLong(tokens);
        if (T <= 0 || T > INT32_MAX) return;   // with PyErr_Occurred() cleared by the caller
        if (PyObject_GetBuffer(c, &buffer, PyBUF_SIMPLE) != 0) return;
        if (buffer.len != (Py_ssize_t)sizeof(smoe_config_t)) return;
        cfg = static_cast<const smoe_config_t*>(buffer.buf);
        if (cfg->hidden <= 0 || cfg->n_experts <= 0 || cfg->top_k <= 0 || cfg->top_k > 32 || cfg->inter <= 0) return;
        H = cfg->hidden;
        E = cfg->n_experts;
        I = cfg->inter;
        R = T * cfg->top_k;
        device = (int)c10::cuda::current_device();
        stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream();
        ok = true;
        if (workspace != Py_None) {
            const at::Tensor* w = tensor(workspace);
            if (w == nullptr) return;
            ws = w->data_ptr();
            ws_bytes = (size_t)w->numel() * w->element_size();
        }
    }
    ~Call() {
        if (buffer.obj != nullptr) PyBuffer_Release(&buffer);
    }
    // A contiguous tensor on this device.
    const at::Tensor* tensor(PyObject* o) {
        ok = ok && THPVariable_CheckExact(o);
        if (!ok) return nullptr;
        const at::Tensor& v = THPVariable_Unpack(o);
        ok = v.layout() == c10::kStrided && v.is_cuda() && v.get_device() == device && v.is_contiguous() && !v.is_neg();
        return ok ? &v : nullptr;
    }
    // The pointer of argument o: n elements of the given type.
    template <class P>
    P* at(PyObject* o, c10::ScalarType type, int64_t n) {
        return pointer<P>(o, [&](const at::Tensor& v) { return v.scalar_type() == type && v.numel() >= n; });
    }
    // The packed weights, of any type: the tensor maps span all of smoe_packed_weight_bytes.
    const void* packed(PyObject* o) {
        return pointer<void>(o, [&](const at::Tensor& v) {
            return v.numel() * (int64_t)v.element_size() >= (E + 1) * 3 * I * H * 2;
        });
    }
    template <class P, class Fits>
    P* pointer(PyObject* o, Fits fits) {
        if (!ok || o == Py_None) return nullptr;
        if (PyLong_CheckExact(o)) {
            void* p = PyLong_AsVoidPtr(o);
            ok = PyErr_Occurred() == nullptr;
            return static_cast<P*>(p);
        }
        const at::Tensor* v = tensor(o);
        if (v == nullptr) return nullptr;
        ok = fits(*v);
        return ok ? static_cast<P*>(v->data_ptr()) : nullptr;
    }
    smoe_bf16_t* bf16(PyObject* o, int64_t n) { return at<smoe_bf16_t>(o, BF16, n); }
    float* f32(PyObject* o, int64_t n) { return at<float>(o, F32, n); }
    int32_t* i32(PyObject* o, int64_t n) { return at<int32_t>(o, I32, n); }
    uint8_t* u8(PyObject* o, int64_t n) { return at<uint8_t>(o, U8, n); }
};

// Calls the library for a regular call, without the interpreter lock; -1 for any other.
template <class F>
int call(const Call& c, F library) {
    if (!c.ok) return -1;
    struct Unlocked {
        PyThreadState* state = PyEval_SaveThread();
        ~Unlocked() { PyEval_RestoreThread(state); }
    } unlocked;
    return (int)library();
}

// Runs f, which returns the status of a regular call or -1.
template <class F>
PyObject* guarded(Py_ssize_t nargs, Py_ssize_t want, F f) {
    int status = -1;
    try {
        if (nargs == want) status = f();
    } catch (...) {   // no exception crosses into the interpreter
    }
    PyErr_Clear();
    if (status < 0) Py_RETURN_NONE;
    return PyLong_FromLong(status);
}

#define ARGS PyObject *, PyObject *const *a, Py_ssize_t n

// cfg, x, x_perm, row_token, offsets, T, packed, y, gu_q, gu_scale, ws, ws_bytes, stream
PyObject* expert_ffn_save(ARGS) {
    return guarded(n, 13, [&] {
        Call c(a[0], a[5], a[10], a[11], a[12]);
        const auto *x = c.bf16(a[1], c.T * c.H), *x_perm = c.bf16(a[2], c.R * c.H);
        const int32_t *row_token = c.i32(a[3], c.R), *offsets = c.i32(a[4], c.E + 1);
        const void* packed = c.packed(a[6]);
        smoe_bf16_t* y = c.bf16(a[7], (c.R + c.T) * c.H);
        uint8_t *q = c.u8(a[8], (c.R + c.T) * 2 * c.I), *s = c.u8(a[9], 2 * c.I / 32 * (c.R + c.T));
        return call(c, [&] {
            return g_expert_ffn_save(c.cfg, x, x_perm, row_token, offsets, c.T, packed, y, q, s, c.ws, c.ws_bytes, c.stream);
        });
    });
}

// cfg, gu_q, gu_scale, T, gu, stream
PyObject* checkpoint_values(ARGS) {
    return guarded(n, 6, [&] {
        Call c(a[0], a[3], Py_None, Py_None, a[5]);
        const int64_t rows = c.R + c.T;
        const uint8_t *q = c.u8(a[1], rows * 2 * c.I), *s = c.u8(a[2], 2 * c.I / 32 * rows);
        smoe_bf16_t* gu = c.bf16(a[4], rows * 2 * c.I);
        return call(c, [&] { return g_checkpoint_values(c.cfg, q, s, c.T, gu, c.stream); });
    });
}

// cfg, dout, y, perm_row, topk_w, T, dy, dtopk_w, ws, ws_bytes, stream
PyObject* combine_backward(ARGS) {
    return guarded(n, 11, [&] {
        Call c(a[0], a[5], a[8], a[9], a[10]);
        const auto *dout = c.bf16(a[1], c.T * c.H), *y = c.bf16(a[2], (c.R + c.T) * c.H);
        const int32_t* perm_row = c.i32(a[3], c.R);
        const float* w = c.f32(a[4], c.R);
        smoe_bf16_t* dy = c.bf16(a[6], c.R * c.H);
        float* dw = c.f32(a[7], c.R);
        return call(c, [&] {
            return g_combine_backward(c.cfg, dout, y, perm_row, w, c.T, dy, dw, c.ws, c.ws_bytes, c.stream);
        });
    });
}

// cfg, x, T, logits, topk_idx, topk_w, dtopk_w, offsets, perm_row, row_token, dlogits, dw_router, ws, ws_bytes, stream
PyObject* route_backward(ARGS) {
    return guarded(n, 15, [&] {
        Call c(a[0], a[2], a[12], a[13], a[14]);
        const smoe_bf16_t* x = c.bf16(a[1], c.T * c.H);
        const float* logits = c.f32(a[3], c.T * c.E);
        const int32_t* idx = c.i32(a[4], c.R);
        const float *w = c.f32(a[5], c.R), *dw = c.f32(a[6], c.R);
        const int32_t *offsets = c.i32(a[7], c.E + 1), *perm_row = c.i32(a[8], c.R), *row_token = c.i32(a[9], c.R);
        float *dl = c.f32(a[10], c.R), *dwr = c.f32(a[11], c.E * c.H);
        return call(c, [&] {
            return g_route_backward(c.cfg, x, c.T, logits, idx, w, dw, offsets, perm_row, row_token, dl, dwr, c.ws, c.ws_bytes,
                                    c.stream);
        });
    });
}

// cfg, x, x_perm, offsets, T, packed, gu_q, gu_scale, dy, dout, dx_rows, dw_gate, dw_up, dw_down, dws_gate, dws_up,
// dws_down, ws, ws_bytes, stream
PyObject* expert_ffn_backward(ARGS) {
    return guarded(n, 20, [&] {
        Call c(a[0], a[4], a[17], a[18], a[19]);
        const int64_t rows = c.R + c.T, w = c.H * c.I;
        const auto *x = c.bf16(a[1], c.T * c.H), *x_perm = c.bf16(a[2], c.R * c.H);
        const int32_t* offsets = c.i32(a[3], c.E + 1);
        const void* packed = c.packed(a[5]);
        const uint8_t *q = c.u8(a[6], rows * 2 * c.I), *s = c.u8(a[7], 2 * c.I / 32 * rows);
        const auto *dy = c.bf16(a[8], c.R * c.H), *dout = c.bf16(a[9], c.T * c.H);
        smoe_bf16_t *dx = c.bf16(a[10], rows * c.H), *dg = c.bf16(a[11], c.E * w), *du = c.bf16(a[12], c.E * w),
                    *dd = c.bf16(a[13], c.E * w), *sg = c.bf16(a[14], w), *su = c.bf16(a[15], w), *sd = c.bf16(a[16], w);
        return call(c, [&] {
            return g_expert_ffn_backward(c.cfg, x, x_perm, offsets, c.T, packed, q, s, dy, dout, dx, dg, du, dd, sg, su, sd, c.ws,
                                         c.ws_bytes, c.stream);
        });
    });
}

// cfg, dx_rows, perm_row, topk_idx, dlogits, w_router, T, dx, ws, ws_bytes, stream
PyObject* permute_backward(ARGS) {
    return guarded(n, 11, [&] {
        Call c(a[0], a[6], a[8], a[9], a[10]);
        const smoe_bf16_t* rows = c.bf16(a[1], (c.R + c.T) * c.H);
        const int32_t *perm_row = c.i32(a[2], c.R), *idx = c.i32(a[3], c.R);
        const float *dl = c.f32(a[4], c.R), *wr = c.f32(a[5], c.E * c.H);
        smoe_bf16_t* dx = c.bf16(a[7], c.T * c.H);
        return call(c, [&] {
            return g_permute_backward(c.cfg, rows, perm_row, idx, dl, wr, c.T, dx, c.ws, c.ws_bytes, c.stream);
        });
    });
}

// use(addresses): the library's functions, in the order of the declarations above
PyObject* use(ARGS) {
    if (n != 6) {
        PyErr_SetString(PyExc_TypeError, "six addresses");
        return nullptr;
    }
    void* p[6];
    for (int i = 0; i < 6; ++i) {
        p[i] = PyLong_AsVoidPtr(a[i]);
        if (p[i] == nullptr) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "a null address");
            return nullptr;
        }
    }
    g_expert_ffn_save = reinterpret_cast<decltype(g_expert_ffn_save)>(p[0]);
    g_checkpoint_values = reinterpret_cast<decltype(g_checkpoint_values)>(p[1]);
    g_combine_backward = reinterpret_cast<decltype(g_combine_backward)>(p[2]);
    g_route_backward = reinterpret_cast<decltype(g_route_backward)>(p[3]);
    g_expert_ffn_backward = reinterpret_cast<decltype(g_expert_ffn_backward)>(p[4]);
    g_permute_backward = reinterpret_cast<decltype(g_permute_backward)>(p[5]);
    Py_RETURN_NONE;
}

#define METHOD(f) {#f, (PyCFunction)(void (*)(void))f, METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {METHOD(expert_ffn_save),     METHOD(checkpoint_values), METHOD(combine_backward),
                           METHOD(route_backward),      METHOD(expert_ffn_backward), METHOD(permute_backward),
                           METHOD(use),                 {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_pyargs", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__pyargs(void) { return PyModule_Create(&g_module); }
