// layer.cpp -- the Python calls of a layer over a paged cache, from torch
// tensors to the C entry points of include/bmmc_layer.h.
#include "common.h"

namespace bmmc_calls {

namespace {

// A cache [pages, places, heads, size] and its scales: none, one value, one for each
// head, or [pages, places, heads] with any strides.
bmmc_scaled_cache scaled(const Tensor &cache, const Tensor *scale, int data, const char *what) {
    TORCH_CHECK_VALUE(cache.dim() == 4, what, " must be [pages, places, heads, size]");
    TORCH_CHECK_VALUE(cache.size(1) > 0 && cache.size(2) > 0, what, " has pages of no places or heads");
    TORCH_CHECK_VALUE(cache.size(3) > 0 && cache.size(3) <= BMMC_MAX_HEAD_DIM,
                      "heads may have up to ", BMMC_MAX_HEAD_DIM, " elements");
    TORCH_CHECK_VALUE(adjacent(cache), "the elements of a head of ", what, " must be adjacent");
    const bool narrow = cache.scalar_type() == at::kFloat8_e4m3fn;
    TORCH_CHECK_VALUE(narrow || (data >= 0 && data_type(cache) == data), what,
                      " must be of the call's type or float8_e4m3fn");
    TORCH_CHECK_VALUE(narrow == (scale != nullptr), "an 8-bit ", what,
                      " has a scale, no other has");
    bmmc_scaled_cache c{};
    c.data = cache.data_ptr();
    c.page_stride = cache.stride(0);
    c.place_stride = cache.stride(1);
    c.head_stride = cache.stride(2);
    c.type = narrow ? BMMC_E4M3 : data;
    if (!narrow) return c;
    TORCH_CHECK_VALUE(scale->scalar_type() == at::kFloat, "a scale of ", what, " is float32");
    c.scale = scale->data_ptr<float>();
    if (scale->dim() == 3 && scale->sizes() == cache.sizes().slice(0, 3)) {
        c.scale_page = scale->stride(0);
        c.scale_place = scale->stride(1);
        c.scale_head = scale->stride(2);
        return c;
    }
    TORCH_CHECK_VALUE(scale->numel() == 1 ||
                          (scale->dim() == 1 && scale->size(0) == cache.size(2)),
                      "a scale of ", what,
                      " is one value, one for each head or [pages, places, heads]");
    c.scale_head = scale->numel() == 1 ? 0 : scale->stride(0);
    return c;
}

void check_two(const Tensor &k, const Tensor &v) {
    TORCH_CHECK_VALUE(k.size(0) == v.size(0) && k.size(1) == v.size(1) && k.size(2) == v.size(2) &&
                          k.scalar_type() == v.scalar_type(),
                      "the two caches must have the same pages, places, heads and type");
}

void check_table(const Tensor &table) {
    TORCH_CHECK_VALUE(table.dim() == 2 && table.scalar_type() == at::kInt &&
                          (table.stride(1) == 1 || table.size(1) <= 1),
                      "page_table must be int32 [sequences, pages], the pages of a sequence "
                      "adjacent");
}

void check_places(const Tensor &positions, const Tensor *sequences, int64_t tokens) {
    check_index(positions, "positions");
    TORCH_CHECK_VALUE(positions.dim() == 1 && positions.size(0) == tokens,
                      "positions must be [tokens]");
    if (!sequences) return;
    check_int32(*sequences, "sequences");
    TORCH_CHECK_VALUE(sequences->dim() == 1 && sequences->size(0) == tokens,
                      "sequences must be [tokens]");
}

PyObject *wrapped(const Tensor &t) { return THPVariable_Wrap(t); }

const int32_t *whole32(const Tensor *t) { return static_cast<const int32_t *>(address(t)); }

}  // namespace

// attention(q, k_cache, v_cache, page_table, lengths, starts, k_scale, v_scale, scale, window,
// out, stream) -> out and the workspace or None; starts, the scales, scale and
// out may be None.
PyObject *py_attention(PyObject *, PyObject *const *a, Py_ssize_t) {
    HANDLE_TH_ERRORS
    const Tensor &q = tensor(a[0], "q");
    const Tensor &k_cache = tensor(a[1], "k_cache"), &v_cache = tensor(a[2], "v_cache");
    const Tensor &table = tensor(a[3], "page_table"), &lengths = tensor(a[4], "lengths");
    const Tensor *starts = maybe(a[5], "starts");
    const Tensor *k_scale = maybe(a[6], "k_scale"), *v_scale = maybe(a[7], "v_scale");
    const Tensor *given = maybe(a[10], "out");
    TORCH_CHECK_VALUE(q.dim() == 3 && data_type(q) >= 0 && q.size(1) > 0,
                      "q must be [tokens, heads, size] of float32, float16 or bfloat16");
    TORCH_CHECK_VALUE(adjacent(q), "the elements of a head of q must be adjacent");
    const int type = data_type(q);
    const bmmc_scaled_cache kc = scaled(k_cache, k_scale, type, "k_cache");
    const bmmc_scaled_cache vc = scaled(v_cache, v_scale, type, "v_cache");
    check_two(k_cache, v_cache);
    TORCH_CHECK_VALUE(k_cache.size(3) == q.size(2), "keys and queries must have heads of one size");
    TORCH_CHECK_VALUE(q.size(2) >= BMMC_LEAST_ATTENDED && v_cache.size(3) >= BMMC_LEAST_ATTENDED,
                      "heads must have ", BMMC_LEAST_ATTENDED, " elements at least");
    TORCH_CHECK_VALUE(q.size(1) % k_cache.size(2) == 0,
                      "q's heads must be a multiple of the caches'");
    check_table(table);
    check_int32(lengths, "lengths");
    TORCH_CHECK_VALUE(lengths.dim() == 1 && lengths.size(0) == table.size(0),
                      "lengths must be [sequences]");
    if (starts) {
        check_int32(*starts, "starts");
        TORCH_CHECK_VALUE(starts->dim() == 1 && starts->size(0) == lengths.size(0) + 1,
                          "starts must be [sequences + 1]");
    } else {
        TORCH_CHECK_VALUE(q.size(0) == lengths.size(0),
                          "without starts there is one token for each sequence");
    }
    for (const Tensor *t : {&q, &k_cache, &v_cache})
        TORCH_CHECK_VALUE(!asks_gradient(*t), "cache_attention has no gradient: call it under "
                                              "no_grad");
    check_constant(k_scale, "k_scale");
    check_constant(v_scale, "v_scale");
    bmmc_attention x{};
    x.tokens = q.size(0);
    x.q_heads = q.size(1);
    x.heads = k_cache.size(2);
    x.k_dim = (int)q.size(2);
    x.v_dim = (int)v_cache.size(3);
    x.scale = a[8] == Py_None ? (float)(1.0 / std::sqrt((double)x.k_dim)) : real(a[8]);
    TORCH_CHECK_VALUE(x.scale > 0.0f && std::isfinite(x.scale), "scale must be above 0 and finite");
    x.window = whole(a[9]);
    TORCH_CHECK_VALUE(x.window >= 0, "window must not be below 0");
    const Tensor out = given ? *given : at::empty({x.tokens, x.q_heads, x.v_dim}, q.options());
    if (given) {
        TORCH_CHECK_VALUE(out.dim() == 3 && out.size(0) == x.tokens && out.size(1) == x.q_heads &&
                              out.size(2) == x.v_dim && out.scalar_type() == q.scalar_type(),
                          "out must be [tokens, heads, size of a value] of q's type");
        TORCH_CHECK_VALUE(adjacent(out), "the elements of a head of out must be adjacent");
        check_written(out, "out");
    }
    on_device(q, k_cache, v_cache, table, lengths, starts, k_scale, v_scale, out);
    x.q = q.data_ptr();
    x.q_token = q.stride(0);
    x.q_head = q.stride(1);
    x.out = out.data_ptr();
    x.out_token = out.stride(0);
    x.out_head = out.stride(1);
    x.table = table.data_ptr<int32_t>();
    x.lengths = lengths.data_ptr<int32_t>();
    x.starts = whole32(starts);
    x.pages = k_cache.size(0);
    x.page_size = k_cache.size(1);
    x.batch = table.size(0);
    x.table_width = table.size(1);
    x.table_stride = table.stride(0);
    x.type = type;
    x.clear_rest = !given;
    Tensor work;
    if (x.tokens) {
        const int64_t need = lib.cache_attention_workspace(&x);
        TORCH_CHECK_VALUE(need >= 0, "the sizes of an attention are out of range");
        if (need) work = at::empty({need}, q.options().dtype(at::kByte));
        check_status(lib.cache_attention(&x, &kc, &vc, address(need ? &work : nullptr), need,
                                         stream_of(a[11])),
                     "cache_attention");
    }
    if (given) written(out);
    return Py_BuildValue("NN", wrapped(out),
                         work.defined() ? wrapped(work) : Py_NewRef(Py_None));
    END_HANDLE_TH_ERRORS
}

// quantize(k, v, k_cache, v_cache, k_scale, v_scale, page_table, positions, sequences, freqs,
// axes, turns, interleaved, scale, q, q_out, stream) -> q_out or None; sequences to turns, q
// and q_out may be None.
PyObject *py_quantize(PyObject *, PyObject *const *a, Py_ssize_t) {
    HANDLE_TH_ERRORS
    const Tensor &k = tensor(a[0], "k"), &v = tensor(a[1], "v");
    const Tensor &k_cache = tensor(a[2], "k_cache"), &v_cache = tensor(a[3], "v_cache");
    const Tensor &k_scale = tensor(a[4], "k_scale"), &v_scale = tensor(a[5], "v_scale");
    const Tensor &table = tensor(a[6], "page_table"), &positions = tensor(a[7], "positions");
    const Tensor *sequences = maybe(a[8], "sequences"), *freqs = maybe(a[9], "freqs");
    const Tensor *axes = maybe(a[10], "axes"), *turns = maybe(a[11], "turns");
    const Tensor *q = maybe(a[14], "q"), *given = maybe(a[15], "q_out");
    TORCH_CHECK_VALUE(k.dim() == 3 && v.dim() == 3 && data_type(k) >= 0 &&
                          v.scalar_type() == k.scalar_type() && k.size(0) == v.size(0) &&
                          k.size(1) == v.size(1) && k.size(1) > 0,
                      "k and v must be [tokens, heads, size] of one type: float32, float16 or "
                      "bfloat16");
    const int64_t tokens = k.size(0), dim = k.size(2), v_dim = v.size(2);
    TORCH_CHECK_VALUE(!(asks_gradient(k) || asks_gradient(v) || (q && asks_gradient(*q))),
                      "cache_quantize has no gradient: call it under no_grad");
    check_constant(freqs, "freqs");
    for (const Tensor *t : {&k_cache, &v_cache})
        TORCH_CHECK_VALUE(t->scalar_type() == at::kFloat8_e4m3fn, "the caches must be float8_e4m3fn");
    const bmmc_scaled_cache kc = scaled(k_cache, &k_scale, -1, "k_cache");
    const bmmc_scaled_cache vc = scaled(v_cache, &v_scale, -1, "v_cache");
    check_two(k_cache, v_cache);
    for (const Tensor *t : {&k_scale, &v_scale})
        TORCH_CHECK_VALUE(t->dim() == 3 && t->sizes() == k_cache.sizes().slice(0, 3),
                          "the scales must be [pages, places, heads]");
    TORCH_CHECK_VALUE(k_cache.size(2) == k.size(1) && k_cache.size(3) == dim &&
                          v_cache.size(3) == v_dim,
                      "the caches must have the heads and sizes of k and v");
    check_written(k_cache, "k_cache");
    check_written(v_cache, "v_cache");
    check_written(k_scale, "k_scale");
    check_written(v_scale, "v_scale");
    if (given) check_written(*given, "q_out");
    check_table(table);
    check_places(positions, sequences, tokens);
    bmmc_rotation r{};
    if (freqs) {
        r = rotation_of(turns, k.sizes().slice(0, 1), *freqs, axes, dim);
        r.interleaved = truth(a[12]);
        r.scale = real(a[13]);
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
    on_device(k, v, k_cache, v_cache, k_scale, v_scale, table, positions, sequences, freqs, axes,
              turns, q, q ? &q_out : nullptr);
    const bmmc_heads kh = heads_of(k, nullptr, "k"), vh = heads_of(v, nullptr, "v");
    if (tokens)
        check_status(lib.cache_quantize(q ? &qh : nullptr, &kh, &vh, &kc, &vc, k_cache.size(0),
                                        k_cache.size(1), table.data_ptr<int32_t>(), table.size(0),
                                        table.size(1), table.stride(0), whole32(sequences),
                                        positions.data_ptr(), index_type(positions),
                                        freqs ? &r : nullptr, tokens, (int)dim, (int)v_dim,
                                        data_type(k), stream_of(a[16])),
                     "cache_quantize");
    for (const Tensor *t : {&k_cache, &v_cache, &k_scale, &v_scale}) written(*t);
    if (given) written(*given);
    if (!q) Py_RETURN_NONE;
    return wrapped(q_out);
    END_HANDLE_TH_ERRORS
}

// read(k_cache, v_cache, page_table, positions, sequences, k_scale, v_scale, a tensor of the
// results' type or None, k_out, v_out, stream) -> k, v; sequences, the scales and the outs may
// be None.
PyObject *py_read(PyObject *, PyObject *const *a, Py_ssize_t) {
    HANDLE_TH_ERRORS
    const Tensor &k_cache = tensor(a[0], "k_cache"), &v_cache = tensor(a[1], "v_cache");
    const Tensor &table = tensor(a[2], "page_table"), &positions = tensor(a[3], "positions");
    const Tensor *sequences = maybe(a[4], "sequences");
    const Tensor *k_scale = maybe(a[5], "k_scale"), *v_scale = maybe(a[6], "v_scale");
    const Tensor *given[2] = {maybe(a[8], "k_out"), maybe(a[9], "v_out")};
    at::ScalarType kind = k_cache.scalar_type();
    if (a[7] != Py_None) {
        TORCH_CHECK_TYPE(THPDtype_Check(a[7]), "dtype must be a torch dtype");
        kind = reinterpret_cast<THPDtype *>(a[7])->scalar_type;
    }
    const int type = kind == at::kFloat ? BMMC_F32 : kind == at::kHalf ? BMMC_F16
                     : kind == at::kBFloat16 ? BMMC_BF16 : -1;
    TORCH_CHECK_VALUE(type >= 0, "dtype must be float32, float16 or bfloat16, and is needed for "
                                 "an 8-bit cache");
    const bmmc_scaled_cache kc = scaled(k_cache, k_scale, type, "k_cache");
    const bmmc_scaled_cache vc = scaled(v_cache, v_scale, type, "v_cache");
    check_two(k_cache, v_cache);
    check_table(table);
    const int64_t tokens = positions.dim() == 1 ? positions.size(0) : -1;
    check_places(positions, sequences, tokens);
    for (const Tensor *t : {&k_cache, &v_cache})
        TORCH_CHECK_VALUE(!asks_gradient(*t), "cache_read has no gradient: call it under no_grad");
    check_constant(k_scale, "k_scale");
    check_constant(v_scale, "v_scale");
    Tensor outs[2];
    bmmc_heads heads[2];
    const Tensor *const caches[2] = {&k_cache, &v_cache};
    for (int i = 0; i < 2; ++i) {
        const int64_t shape[3] = {tokens, caches[i]->size(2), caches[i]->size(3)};
        outs[i] = given[i] ? *given[i] : at::empty(shape, k_cache.options().dtype(kind));
        TORCH_CHECK_VALUE(outs[i].sizes() == at::IntArrayRef(shape, 3) &&
                              outs[i].scalar_type() == kind,
                          "the results are [tokens, heads, size] of dtype");
        check_written(outs[i], i ? "v_out" : "k_out");
        heads[i] = heads_of(outs[i], &outs[i], i ? "v" : "k");
    }
    on_device(k_cache, v_cache, table, positions, sequences, k_scale, v_scale, outs[0], outs[1]);
    if (tokens)
        check_status(lib.cache_read(&heads[0], &heads[1], &kc, &vc, k_cache.size(0), k_cache.size(1),
                                    table.data_ptr<int32_t>(), table.size(0), table.size(1),
                                    table.stride(0), whole32(sequences), positions.data_ptr(),
                                    index_type(positions), tokens, (int)k_cache.size(3),
                                    (int)v_cache.size(3), type, stream_of(a[10])),
                     "cache_read");
    for (int i = 0; i < 2; ++i)
        if (given[i]) written(outs[i]);
    return Py_BuildValue("NN", wrapped(outs[0]), wrapped(outs[1]));
    END_HANDLE_TH_ERRORS
}

namespace {

const uint8_t *mask_of(const Tensor *mask, int64_t tokens) {
    if (!mask) return nullptr;
    TORCH_CHECK_VALUE(mask->scalar_type() == at::kBool && mask->is_contiguous() &&
                          mask->dim() == 1 && mask->size(0) == tokens,
                      "mask must be bool [tokens], contiguous");
    return static_cast<const uint8_t *>(mask->data_ptr());
}

void check_logits(const Tensor &logits) {
    check_matrix(logits, "logits");
    TORCH_CHECK_VALUE(logits.size(1) <= BMMC_MAX_EXPERTS, "there may be up to ", BMMC_MAX_EXPERTS,
                      " experts");
}

}  // namespace

// balance(logits, experts, mask or None, stream) -> loss, counts, slopes and the workspace,
// which other streams than the current one use.
PyObject *py_balance(PyObject *, PyObject *const *a, Py_ssize_t) {
    HANDLE_TH_ERRORS
    const Tensor &logits = tensor(a[0], "logits"), &experts = tensor(a[1], "experts");
    const Tensor *mask = maybe(a[2], "mask");
    check_logits(logits);
    const int64_t tokens = logits.size(0), e = logits.size(1);
    check_index(experts, "experts");
    TORCH_CHECK_VALUE(experts.dim() == 2 && experts.size(0) == tokens && experts.size(1) >= 1 &&
                          experts.size(1) <= BMMC_MAX_CHOICES,
                      "experts must be [tokens, choices], with 1 to ", BMMC_MAX_CHOICES, " choices");
    const uint8_t *masked = mask_of(mask, tokens);
    on_device(logits, experts, mask);
    const int64_t need = lib.expert_balance_workspace(tokens, (int)e);
    TORCH_CHECK_VALUE(need >= 0, "there are too many tokens");
    Tensor loss = at::empty({}, logits.options().dtype(at::kFloat));
    Tensor counts = at::empty({e}, logits.options().dtype(at::kInt));
    Tensor slopes = at::empty({e}, logits.options().dtype(at::kFloat));
    Tensor work = at::empty({need / 4}, logits.options().dtype(at::kInt));
    check_status(lib.expert_balance(logits.data_ptr(), logits.stride(0), data_type(logits), (int)e,
                                    experts.data_ptr(), index_type(experts), tokens,
                                    (int)experts.size(1), masked, loss.data_ptr<float>(),
                                    counts.data_ptr<int32_t>(), slopes.data_ptr<float>(),
                                    work.data_ptr(), need, stream_of(a[3])),
                 "expert_balance");
    return Py_BuildValue("NNNN", wrapped(loss), wrapped(counts), wrapped(slopes), wrapped(work));
    END_HANDLE_TH_ERRORS
}

// balance_backward(grad, logits, slopes, mask or None, out or None, stream) -> gradient of the logits
PyObject *py_balance_backward(PyObject *, PyObject *const *a, Py_ssize_t) {
    HANDLE_TH_ERRORS
    const Tensor &grad = tensor(a[0], "grad"), &logits = tensor(a[1], "logits");
    const Tensor &slopes = tensor(a[2], "slopes");
    const Tensor *mask = maybe(a[3], "mask");
    check_logits(logits);
    const int64_t tokens = logits.size(0), e = logits.size(1);
    TORCH_CHECK_VALUE(grad.numel() == 1 && grad.scalar_type() == at::kFloat,
                      "grad must be one float32 value");
    TORCH_CHECK_VALUE(slopes.dim() == 1 && slopes.size(0) == e &&
                          slopes.scalar_type() == at::kFloat && slopes.is_contiguous(),
                      "slopes must be float32 [experts], contiguous");
    const uint8_t *masked = mask_of(mask, tokens);
    Tensor out = out_of(a[4], tokens, logits);
    on_device(grad, logits, slopes, mask, out);
    if (tokens)
        check_status(lib.expert_balance_backward(grad.data_ptr<float>(), logits.data_ptr(),
                                                 logits.stride(0), data_type(logits), (int)e,
                                                 slopes.data_ptr<float>(), tokens, masked,
                                                 out.data_ptr(), out.stride(0), stream_of(a[5])),
                     "expert_balance_backward");
    if (a[4] != Py_None) written(out);
    return wrapped(out);
    END_HANDLE_TH_ERRORS
}

}  // namespace bmmc_calls
