// calls.cpp — TokenSorter's calls: one function of a Python extension module checks a call's tensors and
// enqueues it. A small call's kernel is over in 2.5 us and its launch takes 2.3 us of host time; the same checks
// in Python and the call through ctypes took another 4 us (unsort with weights and an addend 6.4 us in all).
//
// Each function takes spec = (max_tokens, H, E, k, moe_dtype_t, device index, workspace address, workspace
// bytes), the stream's handle and the tensors (None where the C entry point takes NULL), and returns the
// entry point's status, kNotWanted if a tensor is not of the shape, type, device and layout that spec and the
// others call for, or kWantsGradient if autograd is recording and one requires a gradient, which the call would lose;
// the caller then says which.
#include <Python.h>

#include <c10/core/GradMode.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/moe_b200.h"

namespace {

constexpr long kNotWanted = -1, kWantsGradient = -2;

decltype(&moe_sort_tokens) sort_fn;
decltype(&moe_sort_tokens_backward) sort_backward_fn;
decltype(&moe_unsort_tokens) unsort_fn;
decltype(&moe_unsort_tokens_backward) unsort_backward_fn;

struct Spec {
    int64_t max_tokens;
    moe_token_desc desc;  // T is the call's
    c10::ScalarType type;
    int device;
    void *ws;
    size_t ws_bytes;
};

bool read_spec(PyObject *o, Spec &s)
{
    if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 8)
        return false;
    long long v[8];
    for (int i = 0; i < 8; ++i) {
        v[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(o, i));
        if (v[i] == -1 && PyErr_Occurred())
            return false;
    }
    s.max_tokens = v[0];
    s.desc = moe_token_desc{0, static_cast<int32_t>(v[1]), static_cast<int32_t>(v[2]), static_cast<int32_t>(v[3]),
                            static_cast<int32_t>(v[4])};
    s.type = v[4] == MOE_DTYPE_F32 ? c10::ScalarType::Float
                                   : (v[4] == MOE_DTYPE_BF16 ? c10::ScalarType::BFloat16 : c10::ScalarType::Half);
    s.device = static_cast<int>(v[5]);
    s.ws = reinterpret_cast<void *>(static_cast<uintptr_t>(v[6]));
    s.ws_bytes = static_cast<size_t>(v[7]);
    return true;
}

// The address of a contiguous tensor [rows, cols] (cols < 0: [rows]) of this type and device; false if it is none.
bool tensor(PyObject *o, c10::ScalarType type, int device, int64_t rows, int64_t cols, void **at)
{
    if (!THPVariable_Check(o))
        return false;
    const at::Tensor &t = THPVariable_Unpack(o);
    if (t.dim() != (cols < 0 ? 1 : 2) || t.size(0) != rows || (cols >= 0 && t.size(1) != cols) ||
        t.scalar_type() != type || t.get_device() != device || !t.is_contiguous())
        return false;
    *at = t.data_ptr();
    return true;
}

bool optional(PyObject *o, c10::ScalarType type, int device, int64_t rows, int64_t cols, void **at)
{
    *at = nullptr;
    return o == Py_None || tensor(o, type, device, rows, cols, at);
}

// A tensor's first size as the call's token count.
bool token_count(PyObject *o, Spec &s)
{
    if (!THPVariable_Check(o))
        return false;
    const at::Tensor &t = THPVariable_Unpack(o);
    if (t.dim() != 2 || t.size(0) > INT32_MAX)
        return false;
    s.desc.T = static_cast<int32_t>(t.size(0));
    return true;
}

bool wants_gradient(PyObject *const *t, Py_ssize_t n)
{
    if (!c10::GradMode::is_enabled())
        return false;
    for (Py_ssize_t i = 0; i < n; ++i)
        if (THPVariable_Check(t[i]) && THPVariable_Unpack(t[i]).requires_grad())
            return true;
    return false;
}

// body(spec, stream, tensors) -> status, with Python's and C++'s errors turned into kNotWanted.
template <typename Body>
PyObject *call(PyObject *const *a, Py_ssize_t n, Py_ssize_t tensors, Body body)
{
    if (n != 2 + tensors) {
        PyErr_SetString(PyExc_TypeError, "spec, stream and the operator's tensors are wanted");
        return nullptr;
    }
    long status = kNotWanted;
    try {
        Spec s;
        if (!read_spec(a[0], s)) {
            if (!PyErr_Occurred())
                PyErr_SetString(PyExc_TypeError, "spec is a tuple of eight integers");
            return nullptr;
        }
        void *stream = PyLong_AsVoidPtr(a[1]);
        if (!stream && PyErr_Occurred())
            return nullptr;
        if (wants_gradient(a + 2, tensors))
            status = kWantsGradient;
        else if (s.device >= 0)
            status = body(s, stream, a + 2);
    } catch (...) {  // a tensor without memory
        PyErr_Clear();
    }
    return PyLong_FromLong(status);
}

template <typename Fn>
long without_gil(Fn fn)
{
    long status;
    Py_BEGIN_ALLOW_THREADS;
    status = fn();
    Py_END_ALLOW_THREADS;
    return status;
}

constexpr c10::ScalarType kInt = c10::ScalarType::Int, kFloat = c10::ScalarType::Float;

// x, topk_idx, x_sorted, offsets, slot_of
PyObject *sort(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return call(a, n, 5, [](Spec &s, void *stream, PyObject *const *t) -> long {
        if (!sort_fn || !token_count(t[0], s) || s.desc.T > s.max_tokens)
            return kNotWanted;
        const int64_t T = s.desc.T, H = s.desc.H, k = s.desc.k;
        void *x, *idx, *xs, *off, *slot;
        if (!tensor(t[0], s.type, s.device, T, H, &x) || !tensor(t[1], kInt, s.device, T, k, &idx) ||
            !tensor(t[2], s.type, s.device, T * k, H, &xs) || !tensor(t[3], kInt, s.device, s.desc.E + 1, -1, &off) ||
            !tensor(t[4], kInt, s.device, T, k, &slot))
            return kNotWanted;
        return without_gil([&] {
            return sort_fn(&s.desc, x, static_cast<int32_t *>(idx), xs, static_cast<int32_t *>(off),
                           static_cast<int32_t *>(slot), s.ws, s.ws_bytes, stream);
        });
    });
}

// dx_sorted, slot_of, dx
PyObject *sort_backward(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return call(a, n, 3, [](Spec &s, void *stream, PyObject *const *t) -> long {
        if (!sort_backward_fn || !token_count(t[1], s))
            return kNotWanted;
        const int64_t T = s.desc.T, H = s.desc.H, k = s.desc.k;
        void *dxs, *slot, *dx;
        if (!tensor(t[0], s.type, s.device, T * k, H, &dxs) || !tensor(t[1], kInt, s.device, T, k, &slot) ||
            !tensor(t[2], s.type, s.device, T, H, &dx))
            return kNotWanted;
        return without_gil([&] { return sort_backward_fn(&s.desc, dxs, static_cast<int32_t *>(slot), dx, stream); });
    });
}

// y_sorted, slot_of, topk_w or None, add or None, y
PyObject *unsort(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return call(a, n, 5, [](Spec &s, void *stream, PyObject *const *t) -> long {
        if (!unsort_fn || !token_count(t[1], s))
            return kNotWanted;
        const int64_t T = s.desc.T, H = s.desc.H, k = s.desc.k;
        void *ys, *slot, *w, *add, *y;
        if (!tensor(t[0], s.type, s.device, T * k, H, &ys) || !tensor(t[1], kInt, s.device, T, k, &slot) ||
            !optional(t[2], kFloat, s.device, T, k, &w) || !optional(t[3], s.type, s.device, T, H, &add) ||
            !tensor(t[4], s.type, s.device, T, H, &y))
            return kNotWanted;
        return without_gil([&] {
            return unsort_fn(&s.desc, ys, static_cast<int32_t *>(slot), static_cast<float *>(w), add, y, stream);
        });
    });
}

// dy, y_sorted, slot_of, topk_w or None, dy_sorted, dtopk_w
PyObject *unsort_backward(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return call(a, n, 6, [](Spec &s, void *stream, PyObject *const *t) -> long {
        if (!unsort_backward_fn || !token_count(t[2], s))
            return kNotWanted;
        const int64_t T = s.desc.T, H = s.desc.H, k = s.desc.k;
        void *dy, *ys, *slot, *w, *dys, *dw;
        if (!tensor(t[0], s.type, s.device, T, H, &dy) || !tensor(t[1], s.type, s.device, T * k, H, &ys) ||
            !tensor(t[2], kInt, s.device, T, k, &slot) || !optional(t[3], kFloat, s.device, T, k, &w) ||
            !tensor(t[4], s.type, s.device, T * k, H, &dys) || !tensor(t[5], kFloat, s.device, T, k, &dw))
            return kNotWanted;
        return without_gil([&] {
            return unsort_backward_fn(&s.desc, dy, ys, static_cast<int32_t *>(slot), static_cast<float *>(w), dys,
                                      static_cast<float *>(dw), stream);
        });
    });
}

// Addresses of the four entry points in the loaded library.
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    void *at[4];
    if (n != 4) {
        PyErr_SetString(PyExc_TypeError, "four addresses are wanted");
        return nullptr;
    }
    for (int i = 0; i < 4; ++i)
        if (!(at[i] = PyLong_AsVoidPtr(a[i]))) {
            if (!PyErr_Occurred())
                PyErr_SetString(PyExc_ValueError, "an address is NULL");
            return nullptr;
        }
    sort_fn = reinterpret_cast<decltype(sort_fn)>(at[0]);
    sort_backward_fn = reinterpret_cast<decltype(sort_backward_fn)>(at[1]);
    unsort_fn = reinterpret_cast<decltype(unsort_fn)>(at[2]);
    unsort_backward_fn = reinterpret_cast<decltype(unsort_backward_fn)>(at[3]);
    Py_RETURN_NONE;
}

#define METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(bind),   METHOD(sort), METHOD(sort_backward), METHOD(unsort), METHOD(unsort_backward),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls()
{
    return PyModule_Create(&module);
}
