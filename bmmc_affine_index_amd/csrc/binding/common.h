// common.h -- what the calls from Python share: the library's entry points,
// arguments, the checks of tensors and the state of a call.
#pragma once

#include <Python.h>

#include <dlfcn.h>

#include <cmath>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/empty_like.h>
#include <c10/core/AutogradState.h>
#include <c10/core/GradMode.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../../include/bmmc_layer.h"

namespace bmmc_calls {

using at::Tensor;

struct Library {
    decltype(&bmmc_expert_rows) expert_rows;
    decltype(&bmmc_expert_order_workspace) expert_order_workspace;
    decltype(&bmmc_expert_order) expert_order;
    decltype(&bmmc_expert_gather) expert_gather;
    decltype(&bmmc_expert_combine) expert_combine;
    decltype(&bmmc_expert_combine_backward) expert_combine_backward;
    decltype(&bmmc_rotary) rotary;
    decltype(&bmmc_cache_append) cache_append;
    decltype(&bmmc_cache_attention_workspace) cache_attention_workspace;
    decltype(&bmmc_cache_attention) cache_attention;
    decltype(&bmmc_cache_quantize) cache_quantize;
    decltype(&bmmc_cache_read) cache_read;
    decltype(&bmmc_expert_balance_workspace) expert_balance_workspace;
    decltype(&bmmc_expert_balance) expert_balance;
    decltype(&bmmc_expert_balance_backward) expert_balance_backward;
};

extern Library lib;
extern PyObject *bmmc_error;  // BmmcError(status, what)

// The calls of layer.cpp, which calls.cpp puts into the module.
PyObject *py_attention(PyObject *, PyObject *const *, Py_ssize_t);
PyObject *py_quantize(PyObject *, PyObject *const *, Py_ssize_t);
PyObject *py_read(PyObject *, PyObject *const *, Py_ssize_t);
PyObject *py_balance(PyObject *, PyObject *const *, Py_ssize_t);
PyObject *py_balance_backward(PyObject *, PyObject *const *, Py_ssize_t);

namespace {

// ---- arguments -------------------------------------------------------------

const Tensor &tensor(PyObject *o, const char *what) {
    TORCH_CHECK_TYPE(THPVariable_Check(o), what, " must be a tensor");
    return THPVariable_Unpack(o);
}

const Tensor *maybe(PyObject *o, const char *what) {
    return o == Py_None ? nullptr : &tensor(o, what);
}

int64_t whole(PyObject *o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw python_error();
    return v;
}

bool truth(PyObject *o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw python_error();
    return v != 0;
}

float real(PyObject *o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw python_error();
    return (float)v;
}

void *address(const Tensor *t) { return t ? t->data_ptr() : nullptr; }

// BMMC_F32, BMMC_F16 or BMMC_BF16; -1 for another type.
int data_type(const Tensor &t) {
    switch (t.scalar_type()) {
    case at::kFloat: return BMMC_F32;
    case at::kHalf: return BMMC_F16;
    case at::kBFloat16: return BMMC_BF16;
    default: return -1;
    }
}

// BMMC_I32 or BMMC_I64; -1 for another type.
int index_type(const Tensor &t) {
    switch (t.scalar_type()) {
    case at::kInt: return BMMC_I32;
    case at::kLong: return BMMC_I64;
    default: return -1;
    }
}

// Elements along the last dimension lie next to each other; without elements
// any stride will do (that of an expanded gradient is 0).
bool adjacent(const Tensor &t) {
    return t.stride(-1) == 1 || t.size(-1) == 1 || t.numel() == 0;
}

void check_matrix(const Tensor &x, const char *what) {
    TORCH_CHECK_VALUE(x.dim() == 2 && data_type(x) >= 0, what,
                      " must be [rows, width] of float32, float16 or bfloat16");
    TORCH_CHECK_VALUE(x.size(1) > 0, what, " has rows of no elements");
    TORCH_CHECK_VALUE(adjacent(x), "the elements of a row of ", what, " must be adjacent");
}

void check_int32(const Tensor &x, const char *what) {
    TORCH_CHECK_VALUE(x.scalar_type() == at::kInt && x.is_contiguous(), what,
                      " must be contiguous int32");
}

void check_index(const Tensor &x, const char *what) {
    TORCH_CHECK_VALUE(index_type(x) >= 0 && x.is_contiguous(), what,
                      " must be contiguous int32 or int64");
}

// ---- the call --------------------------------------------------------------

const Tensor *pointer(const Tensor &t) { return &t; }
const Tensor *pointer(const Tensor *t) { return t; }

// A dual tensor's tangent would be lost: the calls have no forward-mode derivative.
void check_tangent(const Tensor &t) {
    TORCH_CHECK_VALUE(!t._fw_grad(0).defined() ||
                          !c10::AutogradState::get_tls_state().get_fw_grad_mode(),
                      "there is no forward-mode derivative: unpack the dual tensor");
}

// Tensors, and pointers to those that may be left out.
template <typename... T> void on_device(const T &...all) {
    const Tensor *const ts[] = {pointer(all)...};
    for (const Tensor *t : ts)
        if (t) check_tangent(*t);
    for (const Tensor *t : ts)
        TORCH_CHECK_VALUE(!t || t->is_cuda(), "tensors must be device tensors");
    const auto current = c10::hip::current_device();
    for (const Tensor *t : ts)
        TORCH_CHECK_VALUE(!t || t->get_device() == current,
                          "tensors must be on the current device");
}

// As at::empty_like, which takes longer over the usual order of dimensions.
Tensor like(const Tensor &x) {
    bool falling = true;
    for (int64_t i = 1; i < x.dim(); ++i) falling &= x.stride(i - 1) >= x.stride(i);
    return falling ? at::empty(x.sizes(), x.options()) : at::empty_like(x);
}

bool asks_gradient(const Tensor &t) { return t.requires_grad() && c10::GradMode::is_enabled(); }

// A caller's tensor that is written has no gradient to ask for: no call makes it.
void check_written(const Tensor &t, const char *what) {
    TORCH_CHECK_VALUE(!asks_gradient(t), what, " must not ask for a gradient");
}

// An input whose gradient no call makes; asking for it would lose it.
void check_constant(const Tensor *t, const char *what) {
    TORCH_CHECK_VALUE(!t || !asks_gradient(*t), what,
                      " has no gradient: detach it, or call under no_grad");
}

// A caller's tensor has been written: autograd raises where it was saved for a
// backward pass before.  Inference tensors are never saved and count nothing.
void written(const Tensor &t) {
    if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

// A stream's handle, torch's current stream for None.
void *stream_of(PyObject *o) {
    if (o == Py_None) return c10::hip::getCurrentHIPStream().stream();
    void *h = PyLong_AsVoidPtr(o);
    if (!h && PyErr_Occurred()) throw python_error();
    return h;
}

void check_status(int status, const char *what) {
    if (status == BMMC_OK) return;
    PyObject *e = PyObject_CallFunction(bmmc_error, "is", status, what);
    if (e) {
        PyErr_SetObject(bmmc_error, e);
        Py_DECREF(e);
    }
    throw python_error();
}

// A caller's out, or a new one, for `rows` rows like x's.
Tensor out_of(PyObject *o, int64_t rows, const Tensor &x) {
    if (o == Py_None) return at::empty({rows, x.size(1)}, x.options());
    const Tensor &out = tensor(o, "out");
    check_matrix(out, "out");
    TORCH_CHECK_VALUE(out.scalar_type() == x.scalar_type() && out.size(0) == rows &&
                          out.size(1) == x.size(1),
                      "out must be [", rows, ", ", x.size(1), "] of the input's type");
    check_written(out, "out");
    return out;
}

// ---- heads and positions ---------------------------------------------------

// x and its output, if it has one, [T, H, D] or [B, S, H, D].
bmmc_heads heads_of(const Tensor &x, const Tensor *out, const char *what) {
    TORCH_CHECK_VALUE(adjacent(x), "the elements of a head of ", what, " must be adjacent");
    bmmc_heads h{};
    h.in = x.data_ptr();
    h.heads = x.size(-2);
    h.in_batch = x.dim() == 4 ? x.stride(0) : 0;
    h.in_token = x.stride(-3);
    h.in_head = x.stride(-2);
    if (!out) return h;
    TORCH_CHECK_VALUE(out->sizes() == x.sizes() && out->scalar_type() == x.scalar_type(),
                      "the output of ", what, " must have its shape and type");
    TORCH_CHECK_VALUE(adjacent(*out), "the elements of a head of ", what,
                      "'s output must be adjacent");
    h.out = out->data_ptr();
    h.out_batch = out->dim() == 4 ? out->stride(0) : 0;
    h.out_token = out->stride(-3);
    h.out_head = out->stride(-2);
    return h;
}

// Positions of one axis have the shape `tokens`, those of several one more
// dimension before it; without positions the entry point's own are meant.
bmmc_rotation rotation_of(const Tensor *positions, at::IntArrayRef tokens, const Tensor &freqs,
                          const Tensor *axes, int64_t dim) {
    TORCH_CHECK_VALUE(freqs.dim() == 1 && freqs.is_contiguous() && freqs.size(0) > 0 &&
                          (freqs.scalar_type() == at::kFloat || freqs.scalar_type() == at::kDouble),
                      "freqs must be [pairs], contiguous, of float32 or float64");
    TORCH_CHECK_VALUE(2 * freqs.size(0) <= dim, "freqs must be [pairs] with at most half as many "
                                                "pairs as a head has elements");
    bmmc_rotation r{};
    r.freqs = freqs.data_ptr();
    r.freqs_are_64 = freqs.scalar_type() == at::kDouble;
    r.pairs = (int)freqs.size(0);
    r.axes = 1;
    r.position_type = BMMC_I32;
    if (positions) {
        const at::IntArrayRef shape = positions->sizes(), strides = positions->strides();
        TORCH_CHECK_VALUE(index_type(*positions) >= 0, "positions must be int32 or int64");
        const size_t before = shape == tokens ? 0 : 1;
        TORCH_CHECK_VALUE(shape.size() == tokens.size() + before && shape.slice(before) == tokens,
                          "positions must have the tokens' shape, or that of axes before it");
        if (before) {
            TORCH_CHECK_VALUE(shape[0] >= 1 && shape[0] <= BMMC_MAX_AXES, "there must be 1 to ",
                              BMMC_MAX_AXES, " axes");
            r.axes = (int)shape[0];
            r.axis_stride = strides[0];
        }
        int64_t next = 1;
        for (size_t i = shape.size(); i-- > before;) {
            TORCH_CHECK_VALUE(shape[i] <= 1 || strides[i] == next,
                              "the positions of an axis must be contiguous");
            next *= shape[i];
        }
        r.position_type = index_type(*positions);
        r.positions = positions->data_ptr();
    }
    if (axes) {
        check_int32(*axes, "axes");
        TORCH_CHECK_VALUE(axes->dim() == 1 && axes->size(0) == freqs.size(0),
                          "axes must have one entry for each pair");
        r.axis_of_pair = axes->data_ptr<int32_t>();
    }
    return r;
}

}  // namespace
}  // namespace bmmc_calls
