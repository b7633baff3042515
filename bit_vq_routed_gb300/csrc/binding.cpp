// The short way from Python to the calls that take less time on the GPU than
// ctypes takes to make them: looks at the tensors, fills the call's struct and makes it
// (a norm with its launch: 2.2 us, by way of Python and ctypes 5.0).
//
// Each function returns the call's status, or LOOK_AGAIN without having made it
// where an argument is not exactly what it expects (a wrong type or shape, a CPU tensor, an
// unusual stride or stream): the Python function then goes its own way, which
// takes the unusual and names the fault.  Nothing is kept from one call to the next
// but the entry points' addresses.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "moe_vq2.h"

namespace {

constexpr long LOOK_AGAIN = 1;

struct {
    decltype(&moe_rms_norm_packed) rms_norm;
    decltype(&moe_quantize_rows_packed) quantize_rows;
    decltype(&moe_linear_8bit_packed) linear_8bit;
    decltype(&moe_route_scored_packed) route_scored;
} entry = {};

using at::ScalarType;

int dtype_of(ScalarType t) {
    return t == ScalarType::BFloat16 ? MOE_DT_BF16 : t == ScalarType::Half ? MOE_DT_F16 : t == ScalarType::Float ? MOE_DT_F32 : -1;
}

const at::Tensor* tensor(PyObject* o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

// [T, H] of that type on the GPU with contiguous rows: its pointer and row stride
template <typename P>
bool rows(const at::Tensor* t, ScalarType type, int64_t T, int64_t H, P** p, int64_t* ld) {
    if (!t || !t->is_cuda() || t->scalar_type() != type || t->dim() != 2 || t->size(0) != T || t->size(1) != H ||
        t->stride(1) != 1)
        return false;
    *p = static_cast<P*>(t->data_ptr());
    *ld = t->stride(0);
    return true;
}
// contiguous, of n elements (any shape: checked by the caller where it matters)
template <typename P>
bool vec(const at::Tensor* t, ScalarType type, int64_t n, P** p) {
    if (!t || !t->is_cuda() || t->scalar_type() != type || t->dim() != 1 || t->size(0) != n || !t->is_contiguous()) return false;
    *p = static_cast<P*>(t->data_ptr());
    return true;
}
template <typename P>
bool table(const at::Tensor* t, ScalarType type, int64_t T, int64_t n, P** p) {
    if (!t || !t->is_cuda() || t->scalar_type() != type || t->dim() != 2 || t->size(0) != T || t->size(1) != n ||
        !t->is_contiguous())
        return false;
    *p = static_cast<P*>(t->data_ptr());
    return true;
}

// None: the current stream; an int: a stream's handle
bool stream_of(PyObject* o, cudaStream_t* s) {
    if (o == Py_None) {
        *s = c10::cuda::getCurrentCUDAStream().stream();
        return true;
    }
    if (!PyLong_Check(o)) return false;
    *s = static_cast<cudaStream_t>(PyLong_AsVoidPtr(o));
    return !PyErr_Occurred();
}
bool int_of(PyObject* o, int* v) {
    const long l = PyLong_AsLong(o);
    *v = static_cast<int>(l);
    return !PyErr_Occurred() && l == *v;
}
bool float_of(PyObject* o, float* v) {
    *v = static_cast<float>(PyFloat_AsDouble(o));
    return !PyErr_Occurred();
}
bool fits(int64_t n) { return n <= INT32_MAX; }

// The call itself, without the interpreter's lock: a launch waits where the GPU's
// queue is full, and what that waits for may need Python.
template <typename F>
long unlocked(F&& call) {
    PyThreadState* state = PyEval_SaveThread();
    const long status = call();
    PyEval_RestoreThread(state);
    return status;
}

// f() returns a status; what it throws, or a Python error it meets, sends the caller
// the other way
template <typename F>
PyObject* answer(Py_ssize_t n, Py_ssize_t want, F&& f) {
    long status = LOOK_AGAIN;
    try {
        if (n == want) status = f();
    } catch (...) {
        status = LOOK_AGAIN;
    }
    if (PyErr_Occurred()) {
        PyErr_Clear();
        status = LOOK_AGAIN;
    }
    return PyLong_FromLong(status);
}

// (x, weight, eps, residual, h, y, q, scales, stream)
PyObject* rms_norm(PyObject*, PyObject* const* o, Py_ssize_t n) {
    return answer(n, 9, [&]() -> long {
        const at::Tensor *x = tensor(o[0]), *w = tensor(o[1]), *r = tensor(o[3]), *h = tensor(o[4]), *y = tensor(o[5]),
                         *q = tensor(o[6]), *s = tensor(o[7]);
        const at::Tensor* typed = w ? w : r ? r : y;
        if (!entry.rms_norm || !x || !typed || x->dim() != 2) return LOOK_AGAIN;
        const ScalarType dt = typed->scalar_type(), xt = x->scalar_type();
        const int64_t T = x->size(0), H = x->size(1);
        moe_rms_norm_args a = {};
        void* p = nullptr;
        cudaStream_t stream;
        a.dtype = dtype_of(dt), a.x_dtype = dtype_of(xt);
        if (a.dtype < 0 || a.dtype == MOE_DT_F32 || (xt != dt && xt != ScalarType::Float) || !fits(T) || !fits(H)) return LOOK_AGAIN;
        if (!rows(x, xt, T, H, &p, &a.ldx)) return LOOK_AGAIN;
        a.x = p;
        if (o[1] != Py_None) {
            if (!vec(w, dt, H, &p)) return LOOK_AGAIN;
            a.weight = p;
        }
        if (o[3] != Py_None) {
            if (!rows(r, dt, T, H, &p, &a.ldr)) return LOOK_AGAIN;
            a.residual = p;
        }
        if (o[4] != Py_None && !rows(h, dt, T, H, &a.h, &a.ldh)) return LOOK_AGAIN;
        if (o[5] != Py_None && !rows(y, dt, T, H, &a.y, &a.ldy)) return LOOK_AGAIN;
        if (o[6] != Py_None && !rows(q, ScalarType::Float8_e4m3fn, T, H, &a.q, &a.ldq)) return LOOK_AGAIN;
        if (o[7] != Py_None && !vec(s, ScalarType::Float, T, &a.scales)) return LOOK_AGAIN;
        if (!float_of(o[2], &a.eps) || !stream_of(o[8], &stream)) return LOOK_AGAIN;
        a.T = (int)T, a.H = (int)H;
        return unlocked([&] { return entry.rms_norm(&a, stream); });
    });
}

// (x, q, scales, stream)
PyObject* quantize_rows(PyObject*, PyObject* const* o, Py_ssize_t n) {
    return answer(n, 4, [&]() -> long {
        const at::Tensor* x = tensor(o[0]);
        if (!entry.quantize_rows || !x || x->dim() != 2) return LOOK_AGAIN;
        const int64_t T = x->size(0), H = x->size(1);
        moe_quantize_rows_args a = {};
        void* p = nullptr;
        cudaStream_t stream;
        a.x_dtype = dtype_of(x->scalar_type());
        if (a.x_dtype < 0 || !fits(T) || !fits(H) || !rows(x, x->scalar_type(), T, H, &p, &a.ldx) ||
            !rows(tensor(o[1]), ScalarType::Float8_e4m3fn, T, H, &a.q, &a.ldq) ||
            !vec(tensor(o[2]), ScalarType::Float, T, &a.scales) || !stream_of(o[3], &stream))
            return LOOK_AGAIN;
        a.x = p, a.T = (int)T, a.H = (int)H;
        return unlocked([&] { return entry.quantize_rows(&a, stream); });
    });
}

// (x, x_scales, w, w_scales, y, bias, act, residual, ws, stream)
PyObject* linear_8bit(PyObject*, PyObject* const* o, Py_ssize_t n) {
    return answer(n, 10, [&]() -> long {
        const at::Tensor *x = tensor(o[0]), *w = tensor(o[2]), *y = tensor(o[4]), *ws = tensor(o[8]);
        if (!entry.linear_8bit || !x || !w || !y || !ws || x->dim() != 2 || w->dim() != 2) return LOOK_AGAIN;
        const int64_t T = x->size(0), K = x->size(1), N = w->size(0);
        const ScalarType dt = y->scalar_type(), e8 = ScalarType::Float8_e4m3fn;
        moe_linear_8bit_args a = {};
        uint8_t* b = nullptr;
        float* f = nullptr;
        void* p = nullptr;
        cudaStream_t stream;
        a.dtype = dtype_of(dt);
        if (a.dtype < 0 || a.dtype == MOE_DT_F32 || !fits(T) || !fits(K) || !fits(N)) return LOOK_AGAIN;
        if (!rows(x, e8, T, K, &b, &a.ldx)) return LOOK_AGAIN;
        a.x = b;
        if (!rows(w, e8, N, K, &b, &a.ldw)) return LOOK_AGAIN;
        a.w = b;
        if (!vec(tensor(o[1]), ScalarType::Float, T, &f)) return LOOK_AGAIN;
        a.x_scales = f;
        if (!vec(tensor(o[3]), ScalarType::Float, N, &f)) return LOOK_AGAIN;
        a.w_scales = f;
        if (!rows(y, dt, T, N, &a.y, &a.ldy)) return LOOK_AGAIN;
        if (o[5] != Py_None) {
            if (!vec(tensor(o[5]), dt, N, &p)) return LOOK_AGAIN;
            a.bias = p;
        }
        if (o[7] != Py_None) {
            if (!rows(tensor(o[7]), dt, T, N, &p, &a.ldr)) return LOOK_AGAIN;
            a.residual = p;
        }
        if (!ws->is_cuda() || !ws->is_contiguous()) return LOOK_AGAIN;
        a.ws = ws->data_ptr(), a.ws_bytes = ws->nbytes();
        if (!int_of(o[6], &a.act) || !stream_of(o[9], &stream)) return LOOK_AGAIN;
        a.T = (int)T, a.N = (int)N, a.K = (int)K;
        return unlocked([&] { return entry.linear_8bit(&a, stream); });
    });
}

// (logits, k, ids, weights, scoring, bias, groups, top_groups, group_top, renormalize, scale, stream)
PyObject* route_scored(PyObject*, PyObject* const* o, Py_ssize_t n) {
    return answer(n, 12, [&]() -> long {
        const at::Tensor* l = tensor(o[0]);
        if (!entry.route_scored || !l || l->dim() != 2) return LOOK_AGAIN;
        const int64_t T = l->size(0), E = l->size(1);
        moe_route_scored_args a = {};
        float* f = nullptr;
        cudaStream_t stream;
        if (!fits(T) || !fits(E) || !int_of(o[1], &a.k)) return LOOK_AGAIN;
        if (!table(l, ScalarType::Float, T, E, &f)) return LOOK_AGAIN;
        a.logits = f;
        if (!table(tensor(o[2]), ScalarType::Int, T, a.k, &a.ids)) return LOOK_AGAIN;
        if (!table(tensor(o[3]), ScalarType::Float, T, a.k, &a.weights)) return LOOK_AGAIN;
        if (o[5] != Py_None) {
            if (!vec(tensor(o[5]), ScalarType::Float, E, &f)) return LOOK_AGAIN;
            a.scoring.bias = f;
        }
        if (!int_of(o[4], &a.scoring.scoring) || !int_of(o[6], &a.scoring.groups) || !int_of(o[7], &a.scoring.top_groups) ||
            !int_of(o[8], &a.scoring.group_top) || !int_of(o[9], &a.scoring.renormalize) ||
            !float_of(o[10], &a.scoring.scale) || !stream_of(o[11], &stream))
            return LOOK_AGAIN;
        a.T = (int)T, a.E = (int)E;
        return unlocked([&] { return entry.route_scored(&a, stream); });
    });
}

// The entry points' addresses, in the order of `entry`.
PyObject* set_entry_points(PyObject*, PyObject* args) {
    unsigned long long p[4];
    if (!PyArg_ParseTuple(args, "KKKK", &p[0], &p[1], &p[2], &p[3])) return nullptr;
    entry.rms_norm = reinterpret_cast<decltype(entry.rms_norm)>(p[0]);
    entry.quantize_rows = reinterpret_cast<decltype(entry.quantize_rows)>(p[1]);
    entry.linear_8bit = reinterpret_cast<decltype(entry.linear_8bit)>(p[2]);
    entry.route_scored = reinterpret_cast<decltype(entry.route_scored)>(p[3]);
    Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"rms_norm", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(rms_norm)), METH_FASTCALL, nullptr},
    {"quantize_rows", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(quantize_rows)), METH_FASTCALL, nullptr},
    {"linear_8bit", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(linear_8bit)), METH_FASTCALL, nullptr},
    {"route_scored", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(route_scored)), METH_FASTCALL, nullptr},
    {"set_entry_points", set_entry_points, METH_VARARGS, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "moe_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_moe_binding() { return PyModule_Create(&module); }
