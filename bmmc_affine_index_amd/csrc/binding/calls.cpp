// calls.cpp -- the Python calls on token rows, from torch tensors to the C
// entry points of include/bmmc_tokens.h.
//
// A decoding step's moves run for 3 to 5 us on the card, so that the call
// around them is what such a step waits for.  Here a call's checks, new tensors
// and launch take 4.8 us of host time for expert_combine of 17 tokens (13.9 us
// with the checks in Python and the call through ctypes), 5.1 us for
// cache_append of 64 (24.2 us), 9.3 us for an order and its gather (28.6 us); a
// launch alone takes 2.8 to 3.4 us.
// Python keeps what is not on that way: autograd, other streams, documentation.
//
// The library is opened by the path that Python names, so that this module
// and ctypes share one copy of it.
#include <Python.h>

#include <dlfcn.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/empty_like.h>
#include <c10/core/AutogradState.h>
#include <c10/core/GradMode.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../../include/bmmc_tokens.h"

namespace {

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
};

Library lib;
PyObject *bmmc_error;  // BmmcError(status, what)

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

// ---- tokens by expert ------------------------------------------------------

// The elements of `all` from `first` on as a contiguous tensor of its own shape.
Tensor part_of(const Tensor &all, int64_t first, at::IntArrayRef shape) {
    Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(all.storage()),
                                                        all.key_set(), all.dtype());
    t.unsafeGetTensorImpl()->set_storage_offset(first);
    t.unsafeGetTensorImpl()->set_sizes_contiguous(shape);
    return t;
}

// order(experts, num_experts, align, stream) -> offsets, counts, rows, slots
// and the workspace or None, which other streams than the current one use.
PyObject *py_order(PyObject *, PyObject *const *a, Py_ssize_t) {
    HANDLE_TH_ERRORS
    const Tensor &experts = tensor(a[0], "experts");
    const int64_t num = whole(a[1]), align = whole(a[2]);
    check_index(experts, "experts");
    const int64_t n = experts.numel();
    const int e = num < 0 || num > BMMC_MAX_EXPERTS ? 0 : (int)num;
    const int64_t capacity = lib.expert_rows(n, e, align);
    TORCH_CHECK_VALUE(capacity >= 0,
                      "the number of experts, the alignment or the order's rows are out of range");
    on_device(experts);
    const int64_t need = lib.expert_order_workspace(n, e);
    const at::TensorOptions whole32 = experts.options().dtype(at::kInt);
    const bool flat = experts.dim() != 2;
    // one allocation for the four results
    const Tensor all = at::empty({2 * e + 1 + n + capacity}, whole32);
    Tensor offsets = part_of(all, 0, {e + 1}), counts = part_of(all, e + 1, {e});
    Tensor rows = part_of(all, 2 * e + 1,
                          {flat ? n : experts.size(0), flat ? 1 : experts.size(1)});
    Tensor slots = part_of(all, 2 * e + 1 + n, {capacity}), work;
    if (need) work = at::empty({need / 4}, whole32);
    check_status(lib.expert_order(experts.data_ptr(), index_type(experts), n, e, align,
                                  offsets.data_ptr<int32_t>(), counts.data_ptr<int32_t>(),
                                  rows.data_ptr<int32_t>(), slots.data_ptr<int32_t>(),
                                  need ? work.data_ptr() : nullptr, need, stream_of(a[3])),
                 "expert_order");
    PyObject *got[5] = {THPVariable_Wrap(offsets), THPVariable_Wrap(counts),
                        THPVariable_Wrap(rows), THPVariable_Wrap(slots),
                        need ? THPVariable_Wrap(work) : Py_NewRef(Py_None)};
    return Py_BuildValue("NNNNN", got[0], got[1], got[2], got[3], got[4]);
    END_HANDLE_TH_ERRORS
}

struct Order {
    const Tensor &rows, &slots;
    int64_t tokens, capacity;
    int choices;
};

Order order_of(PyObject *r, PyObject *s) {
    const Tensor &rows = tensor(r, "order.rows"), &slots = tensor(s, "order.slots");
    check_int32(rows, "order.rows");
    check_int32(slots, "order.slots");
    TORCH_CHECK_VALUE(rows.dim() == 2 && slots.dim() == 1 && rows.size(1) >= 1 &&
                          rows.size(1) <= BMMC_MAX_CHOICES,
                      "order.rows must be [tokens, choices] and order.slots [rows]");
    TORCH_CHECK_VALUE(slots.size(0) >= rows.numel(), "the order has fewer rows than choices");
    return Order{rows, slots, rows.size(0), slots.size(0), (int)rows.size(1)};
}

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

void check_weights(const Tensor &w, const Order &order, const Tensor &rows) {
    TORCH_CHECK_VALUE(w.dim() == 2 && w.size(0) == order.tokens && w.size(1) == order.choices &&
                          w.is_contiguous(),
                      "weights must be contiguous [tokens, choices]");
    TORCH_CHECK_VALUE(w.scalar_type() == at::kFloat || w.scalar_type() == rows.scalar_type(),
                      "weights must be float32 or of the rows' type");
}

// gather(x, order.rows, order.slots, out or None, stream) -> out
PyObject *py_gather(PyObject *, PyObject *const *a, Py_ssize_t) {
    HANDLE_TH_ERRORS
    const Tensor &x = tensor(a[0], "x");
    const Order order = order_of(a[1], a[2]);
    check_matrix(x, "x");
    TORCH_CHECK_VALUE(x.size(0) == order.tokens,
                      "x must have one row for each token of the order");
    Tensor out = out_of(a[3], order.capacity, x);
    on_device(x, order.rows, order.slots, out);
    if (order.capacity)
        check_status(lib.expert_gather(x.data_ptr(), x.stride(0), order.rows.data_ptr<int32_t>(),
                                       order.slots.data_ptr<int32_t>(), order.tokens,
                                       order.choices, order.capacity, x.size(1), data_type(x),
                                       out.data_ptr(), out.stride(0), stream_of(a[4])),
                     "expert_gather");
    if (a[3] != Py_None) written(out);
    return THPVariable_Wrap(out);
    END_HANDLE_TH_ERRORS
}

// combine(rows, order.rows, order.slots, weights or None, out or None, stream) -> out
PyObject *py_combine(PyObject *, PyObject *const *a, Py_ssize_t) {
    HANDLE_TH_ERRORS
    const Tensor &in = tensor(a[0], "rows");
    const Order order = order_of(a[1], a[2]);
    const Tensor *w = maybe(a[3], "weights");
    check_matrix(in, "rows");
    TORCH_CHECK_VALUE(in.size(0) == order.capacity, "rows must have the order's rows");
    if (w) check_weights(*w, order, in);
    Tensor out = out_of(a[4], order.tokens, in);
    on_device(in, order.rows, order.slots, out, w);
    if (order.tokens)
        check_status(lib.expert_combine(in.data_ptr(), in.stride(0),
                                        order.rows.data_ptr<int32_t>(), address(w),
                                        w ? data_type(*w) : BMMC_F32, order.tokens, order.choices,
                                        order.capacity, in.size(1), data_type(in),
                                        out.data_ptr(), out.stride(0), stream_of(a[5])),
                     "expert_combine");
    if (a[4] != Py_None) written(out);
    return THPVariable_Wrap(out);
    END_HANDLE_TH_ERRORS
}

// combine_backward(grad, rows, order.rows, order.slots, weights, stream)
// -> gradients of the rows and of the weights
PyObject *py_combine_backward(PyObject *, PyObject *const *a, Py_ssize_t) {
    HANDLE_TH_ERRORS
    const Tensor &grad = tensor(a[0], "grad"), &in = tensor(a[1], "rows");
    const Order order = order_of(a[2], a[3]);
    const Tensor &w = tensor(a[4], "weights");
    check_matrix(grad, "grad");
    check_matrix(in, "rows");
    TORCH_CHECK_VALUE(in.size(0) == order.capacity, "rows must have the order's rows");
    TORCH_CHECK_VALUE(grad.scalar_type() == in.scalar_type() && grad.size(0) == order.tokens &&
                          grad.size(1) == in.size(1),
                      "grad must be [tokens, width] of the rows' type");
    check_weights(w, order, in);
    Tensor grad_rows = at::empty({order.capacity, in.size(1)}, in.options());
    Tensor grad_weights = at::empty({order.tokens, order.choices}, w.options());
    on_device(grad, in, order.rows, order.slots, w);
    if (order.capacity)
        check_status(
            lib.expert_combine_backward(
                grad.data_ptr(), grad.stride(0), in.data_ptr(), in.stride(0),
                order.rows.data_ptr<int32_t>(), order.slots.data_ptr<int32_t>(), w.data_ptr(),
                data_type(w), order.tokens, order.choices, order.capacity, in.size(1),
                data_type(in), grad_rows.data_ptr(), grad_rows.stride(0),
                grad_weights.data_ptr(), stream_of(a[5])),
            "expert_combine_backward");
    return Py_BuildValue("NN", THPVariable_Wrap(grad_rows), THPVariable_Wrap(grad_weights));
    END_HANDLE_TH_ERRORS
}

// ---- rotary positions and the paged cache ----------------------------------

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

// rotary(tensors, positions, freqs, axes or None, interleaved, scale, outs or
// None, inverse, stream) -> outputs
PyObject *py_rotary(PyObject *, PyObject *const *a, Py_ssize_t) {
    HANDLE_TH_ERRORS
    const Py_ssize_t count = PyTuple_GET_SIZE(a[0]);
    TORCH_CHECK_VALUE(count >= 1 && count <= 2 &&
                          (a[6] == Py_None || PyTuple_GET_SIZE(a[6]) == count),
                      "one or two tensors of heads are turned");
    const Tensor *xs[2];
    for (Py_ssize_t i = 0; i < count; ++i) xs[i] = &tensor(PyTuple_GET_ITEM(a[0], i), "x");
    const Tensor &x = *xs[0];
    const int64_t nd = x.dim();
    TORCH_CHECK_VALUE((nd == 3 || nd == 4) && data_type(x) >= 0,
                      "heads must be [tokens, heads, size] or [batch, tokens, heads, size] of "
                      "float32, float16 or bfloat16");
    const at::IntArrayRef lead = x.sizes().slice(0, nd - 2);
    const int64_t dim = x.size(-1);
    for (Py_ssize_t i = 0; i < count; ++i) {
        const Tensor &y = *xs[i];
        TORCH_CHECK_VALUE(y.scalar_type() == x.scalar_type() && y.dim() == nd &&
                              y.size(-1) == dim && y.sizes().slice(0, nd - 2) == lead,
                          "the tensors must have the same tokens, size of heads and type");
        TORCH_CHECK_VALUE(dim > 0 && dim <= BMMC_MAX_HEAD_DIM && y.size(-2) > 0,
                          "there must be heads, of up to ", BMMC_MAX_HEAD_DIM, " elements");
    }
    const Tensor *positions = maybe(a[1], "positions");
    TORCH_CHECK_VALUE(positions, "positions are needed");
    const Tensor &freqs = tensor(a[2], "freqs"), *axes = maybe(a[3], "axes");
    bmmc_rotation r = rotation_of(positions, lead, freqs, axes, dim);
    check_constant(&freqs, "freqs");
    r.interleaved = truth(a[4]);
    r.scale = real(a[5]);
    r.inverse = truth(a[7]);
    Tensor outs[2];
    bmmc_heads heads[2];
    for (Py_ssize_t i = 0; i < count; ++i) {
        PyObject *o = a[6] == Py_None ? Py_None : PyTuple_GET_ITEM(a[6], i);
        outs[i] = o == Py_None ? like(*xs[i]) : tensor(o, "out");
        check_written(outs[i], "out");
        heads[i] = heads_of(*xs[i], &outs[i], "x");
    }
    on_device(x, outs[0], xs[count - 1], outs[count - 1], *positions, freqs, axes);
    if (x.numel())
        check_status(lib.rotary(heads, (int)count, nd == 4 ? lead[0] : 1, lead[nd - 3], (int)dim,
                                data_type(x), &r, stream_of(a[8])),
                     "rotary");
    for (Py_ssize_t i = 0; i < count && a[6] != Py_None; ++i)
        if (PyTuple_GET_ITEM(a[6], i) != Py_None) written(outs[i]);
    if (count == 1) return Py_BuildValue("(N)", THPVariable_Wrap(outs[0]));
    return Py_BuildValue("NN", THPVariable_Wrap(outs[0]), THPVariable_Wrap(outs[1]));
    END_HANDLE_TH_ERRORS
}

bmmc_paged_cache paged(const Tensor &cache, const Tensor &x, const Tensor *scale,
                       const char *what) {
    TORCH_CHECK_VALUE(cache.dim() == 4 && cache.size(2) == x.size(1) && cache.size(3) == x.size(2),
                      what, " must be [pages, places, heads, size]");
    TORCH_CHECK_VALUE(adjacent(cache), "the elements of a head of ", what, " must be adjacent");
    const bool narrow = cache.scalar_type() == at::kFloat8_e4m3fn;
    TORCH_CHECK_VALUE(narrow || cache.scalar_type() == x.scalar_type(), what,
                      " must be of the inputs' type or float8_e4m3fn");
    TORCH_CHECK_VALUE(narrow == (scale != nullptr), "an 8-bit ", what,
                      " has a scale, no other has");
    bmmc_paged_cache c{};
    if (narrow) {
        TORCH_CHECK_VALUE(scale->scalar_type() == at::kFloat && scale->is_contiguous() &&
                              (scale->numel() == 1 || scale->numel() == x.size(1)),
                          "a scale of ", what, " is float32, one value or one for each head");
        c.scale = scale->data_ptr<float>();
        c.scale_stride = scale->numel() > 1;
    }
    c.data = cache.data_ptr();
    c.page_stride = cache.stride(0);
    c.place_stride = cache.stride(1);
    c.head_stride = cache.stride(2);
    c.type = narrow ? BMMC_E4M3 : data_type(x);
    return c;
}

// append(k, v, k_cache, v_cache, page_table, positions, sequences, freqs,
// axes, turns, interleaved, scale, q, q_out, k_scale, v_scale, stream) -> q_out
// or None; sequences to turns, q, q_out and the scales may be None.
PyObject *py_append(PyObject *, PyObject *const *a, Py_ssize_t) {
    HANDLE_TH_ERRORS
    const Tensor &k = tensor(a[0], "k"), &v = tensor(a[1], "v");
    const Tensor &k_cache = tensor(a[2], "k_cache"), &v_cache = tensor(a[3], "v_cache");
    const Tensor &table = tensor(a[4], "page_table"), &positions = tensor(a[5], "positions");
    const Tensor *sequences = maybe(a[6], "sequences"), *freqs = maybe(a[7], "freqs");
    const Tensor *axes = maybe(a[8], "axes"), *turns = maybe(a[9], "turns");
    const Tensor *q = maybe(a[12], "q"), *given = maybe(a[13], "q_out");
    const Tensor *k_scale = maybe(a[14], "k_scale"), *v_scale = maybe(a[15], "v_scale");
    TORCH_CHECK_VALUE(k.dim() == 3 && v.dim() == 3 && data_type(k) >= 0 &&
                          v.scalar_type() == k.scalar_type() && k.size(0) == v.size(0) &&
                          k.size(1) == v.size(1) && k.size(1) > 0,
                      "k and v must be [tokens, heads, size] of one type: float32, float16 or "
                      "bfloat16");
    const int64_t tokens = k.size(0), dim = k.size(2), v_dim = v.size(2);
    TORCH_CHECK_VALUE(dim > 0 && dim <= BMMC_MAX_HEAD_DIM && v_dim > 0 &&
                          v_dim <= BMMC_MAX_HEAD_DIM,
                      "heads may have up to ", BMMC_MAX_HEAD_DIM, " elements");
    TORCH_CHECK_VALUE(!(asks_gradient(k) || asks_gradient(v) || (q && asks_gradient(*q))),
                      "cache_append has no gradient: call it under no_grad");
    check_constant(freqs, "freqs");
    check_constant(k_scale, "k_scale");
    check_constant(v_scale, "v_scale");
    check_written(k_cache, "k_cache");
    check_written(v_cache, "v_cache");
    if (given) check_written(*given, "q_out");
    const bmmc_paged_cache kc = paged(k_cache, k, k_scale, "k_cache");
    const bmmc_paged_cache vc = paged(v_cache, v, v_scale, "v_cache");
    TORCH_CHECK_VALUE(k_cache.size(0) == v_cache.size(0) && k_cache.size(1) == v_cache.size(1) &&
                          k_cache.scalar_type() == v_cache.scalar_type(),
                      "the two caches must have the same pages, places and type");
    TORCH_CHECK_VALUE(k_cache.size(1) > 0, "pages have no places");
    TORCH_CHECK_VALUE(table.dim() == 2 && table.scalar_type() == at::kInt &&
                          (table.stride(1) == 1 || table.size(1) <= 1),
                      "page_table must be int32 [sequences, pages], the pages of a sequence "
                      "adjacent");
    check_index(positions, "positions");
    TORCH_CHECK_VALUE(positions.dim() == 1 && positions.size(0) == tokens,
                      "positions must be [tokens]");
    if (sequences) {
        check_int32(*sequences, "sequences");
        TORCH_CHECK_VALUE(sequences->dim() == 1 && sequences->size(0) == tokens,
                          "sequences must be [tokens]");
    }
    bmmc_rotation r{};
    if (freqs) {
        r = rotation_of(turns, k.sizes().slice(0, 1), *freqs, axes, dim);
        r.interleaved = truth(a[10]);
        r.scale = real(a[11]);
    } else {
        TORCH_CHECK_VALUE(!q && !given && !turns && !axes, "queries, turns and axes go with freqs");
    }
    TORCH_CHECK_VALUE(q || !given, "q_out goes with q");
    bmmc_heads qh{};
    Tensor q_out;
    if (q) {
        TORCH_CHECK_VALUE(q->dim() == 3 && q->scalar_type() == k.scalar_type() &&
                              q->size(0) == tokens && q->size(1) > 0 && q->size(2) == dim,
                          "q must be [tokens, heads, size] as k");
        q_out = given ? *given : like(*q);
        qh = heads_of(*q, &q_out, "q");
    }
    on_device(k, v, k_cache, v_cache, table, positions, sequences, freqs, axes, turns, k_scale,
              v_scale, q, q ? &q_out : nullptr);
    const bmmc_heads kh = heads_of(k, nullptr, "k"), vh = heads_of(v, nullptr, "v");
    if (tokens)
        check_status(lib.cache_append(q ? &qh : nullptr, &kh, &vh, &kc, &vc, k_cache.size(0),
                                      k_cache.size(1), table.data_ptr<int32_t>(), table.size(0),
                                      table.size(1), table.stride(0),
                                      static_cast<const int32_t *>(address(sequences)),
                                      positions.data_ptr(), index_type(positions),
                                      freqs ? &r : nullptr, tokens, (int)dim, (int)v_dim,
                                      data_type(k), stream_of(a[16])),
                     "cache_append");
    written(k_cache);
    written(v_cache);
    if (given) written(*given);
    if (!q) Py_RETURN_NONE;
    return THPVariable_Wrap(q_out);
    END_HANDLE_TH_ERRORS
}

// ---- the module ------------------------------------------------------------

// asks(tensors, None or tuples of them ...): whether one asks for a gradient;
// none may have a tangent.
bool asks(PyObject *o) {
    if (THPVariable_Check(o)) {
        check_tangent(THPVariable_Unpack(o));
        return asks_gradient(THPVariable_Unpack(o));
    }
    bool one = false;
    for (Py_ssize_t i = 0; PyTuple_Check(o) && i < PyTuple_GET_SIZE(o); ++i)
        one |= asks(PyTuple_GET_ITEM(o, i));
    return one;
}
PyObject *py_asks(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    bool one = false;
    for (Py_ssize_t i = 0; i < n; ++i) one |= asks(a[i]);
    return PyBool_FromLong(one);
    END_HANDLE_TH_ERRORS
}

// load(path of libbmmc.so, BmmcError)
PyObject *py_load(PyObject *, PyObject *const *a, Py_ssize_t) {
    HANDLE_TH_ERRORS
    const char *path = PyUnicode_AsUTF8(a[0]);
    if (!path) throw python_error();
    void *so = dlopen(path, RTLD_NOW | RTLD_LOCAL);
    TORCH_CHECK(so, "cannot open ", path, ": ", dlerror());
    const auto find = [&](const char *name, auto &f) {
        f = reinterpret_cast<std::decay_t<decltype(f)>>(dlsym(so, name));
        TORCH_CHECK(f, path, " has no ", name);
    };
    find("bmmc_expert_rows", lib.expert_rows);
    find("bmmc_expert_order_workspace", lib.expert_order_workspace);
    find("bmmc_expert_order", lib.expert_order);
    find("bmmc_expert_gather", lib.expert_gather);
    find("bmmc_expert_combine", lib.expert_combine);
    find("bmmc_expert_combine_backward", lib.expert_combine_backward);
    find("bmmc_rotary", lib.rotary);
    find("bmmc_cache_append", lib.cache_append);
    Py_XSETREF(bmmc_error, Py_NewRef(a[1]));
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

// The wrappers above index their arguments; this counts them first.
template <PyObject *(*CALL)(PyObject *, PyObject *const *, Py_ssize_t), int COUNT>
PyObject *counted(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    if (n != COUNT || (CALL != py_load && !bmmc_error))
        return PyErr_Format(PyExc_TypeError, "%d arguments are needed, after load()", COUNT);
    return CALL(self, a, n);
}

template <PyObject *(*CALL)(PyObject *, PyObject *const *, Py_ssize_t), int COUNT>
PyMethodDef method(const char *name) {
    return PyMethodDef{name, reinterpret_cast<PyCFunction>(
                                 reinterpret_cast<void (*)(void)>(counted<CALL, COUNT>)),
                       METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {
    method<py_load, 2>("load"),
    method<py_order, 4>("order"),
    method<py_gather, 5>("gather"),
    method<py_combine, 6>("combine"),
    method<py_combine_backward, 6>("combine_backward"),
    method<py_rotary, 9>("rotary"),
    method<py_append, 17>("append"),
    PyMethodDef{"asks", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(py_asks)),
                METH_FASTCALL, nullptr},
    PyMethodDef{nullptr, nullptr, 0, nullptr},
};

PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__calls(void) { return PyModule_Create(&module_def); }
