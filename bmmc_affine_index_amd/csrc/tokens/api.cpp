// api.cpp -- the extern "C" entry points declared in include/bmmc_tokens.h:
// every argument check, before any HIP call, and the kernels' arguments.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "../../../include/bmmc_tokens.h"
#include "tokens.h"

namespace {

constexpr int64_t kMaxIndex = (int64_t(1) << 31) - 1;
// A stride or a width past this is no address on any card; below it the
// products below stay in 64 bits.
constexpr int64_t kMaxStride = int64_t(1) << 40;
constexpr int64_t kMaxHeads = 65536;

int element_bytes(int type) { return type == BMMC_F32 ? 4 : type == BMMC_E4M3 ? 1 : 2; }

bool data_type(int type) { return type == BMMC_F32 || type == BMMC_F16 || type == BMMC_BF16; }

bool index_type_ok(int type) { return type == BMMC_I32 || type == BMMC_I64; }

bool aligned(const void *p, size_t bytes) { return (uintptr_t)p % bytes == 0; }

bool stride_ok(int64_t s) { return s >= 0 && s <= kMaxStride; }

// The bytes [lo, hi) that a strided array touches.
struct Extent {
    uintptr_t lo, hi;
};

Extent extent(const void *p, int bytes, int64_t inner, const int64_t *sizes,
              const int64_t *strides, int dims) {
    unsigned __int128 last = (unsigned __int128)inner;
    for (int i = 0; i < dims; ++i) {
        if (sizes[i] <= 0) return Extent{(uintptr_t)p, (uintptr_t)p};
        last += (unsigned __int128)(sizes[i] - 1) * (unsigned __int128)strides[i];
    }
    const unsigned __int128 hi = (unsigned __int128)(uintptr_t)p + last * (unsigned)bytes;
    return Extent{(uintptr_t)p, hi > UINTPTR_MAX ? UINTPTR_MAX : (uintptr_t)hi};
}

bool meet(const Extent &a, const Extent &b) { return a.lo < b.hi && b.lo < a.hi; }

// No two elements of a written array share an address: taken by rising
// stride, each dimension steps past all that the ones before it cover.
bool apart(int64_t inner, const int64_t *sizes, const int64_t *strides, int dims) {
    int order[3] = {0, 1, 2};
    std::sort(order, order + dims, [&](int x, int y) { return strides[x] < strides[y]; });
    __int128 covered = inner;
    for (int i = 0; i < dims; ++i) {
        const int d = order[i];
        if (sizes[d] <= 1) continue;
        if (strides[d] < covered) return false;
        covered += (__int128)(sizes[d] - 1) * strides[d];
    }
    return true;
}

// An array's steps, widest first: without those that lead nowhere.
struct Steps {
    int64_t inner;  // adjacent elements at each step
    int dims = 0;
    int64_t sizes[3], strides[3];

    Steps(int64_t elements, const int64_t *n, const int64_t *s, int count) : inner(elements) {
        for (int i = 0; i < count; ++i) {
            if (n[i] <= 1 || s[i] == 0) continue;
            int at = dims++;
            for (; at > 0 && strides[at - 1] < s[i]; --at) {
                sizes[at] = sizes[at - 1];
                strides[at] = strides[at - 1];
            }
            sizes[at] = n[i];
            strides[at] = s[i];
        }
    }
    // Elements from the first to past the last of one step of the first `from`.
    __int128 reach(int from) const {
        __int128 r = inner;
        for (int i = from; i < dims; ++i) r += (__int128)(sizes[i] - 1) * strides[i];
        return r;
    }
};

__int128 floor_div(__int128 a, int64_t b) { return a / b - (a % b < 0); }

// Whether b, `off` elements from a, has an element that a has too.  Without
// their i and j widest steps the two are compared for each difference of the
// next step that brings their stretches together, which is one or none for
// arrays in step; after `looks` comparisons the answer is yes.
bool shared(const Steps &a, int i, const Steps &b, int j, __int128 off, int *looks) {
    if (off >= a.reach(i) || -off >= b.reach(j)) return false;
    if (i == a.dims && j == b.dims) return true;
    if (--*looks < 0) return true;
    const int64_t sa = i < a.dims ? a.strides[i] : 0, sb = j < b.dims ? b.strides[j] : 0;
    const int64_t step = std::max(sa, sb);
    const int64_t na = sa == step ? a.sizes[i] : 1, nb = sb == step ? b.sizes[j] : 1;
    i += sa == step;
    j += sb == step;
    const __int128 lo = std::max<__int128>(1 - na, floor_div(-b.reach(j) - off, step) + 1);
    const __int128 hi = std::min<__int128>(nb - 1, floor_div(a.reach(i) - off - 1, step));
    for (__int128 k = lo; k <= hi; ++k)
        if (shared(a, i, b, j, off + k * step, looks)) return true;
    return false;
}

bool share(const void *p, const Steps &a, const void *q, const Steps &b, int bytes) {
    int looks = 256;
    const __int128 off = ((__int128)(uintptr_t)q - (__int128)(uintptr_t)p) / bytes;
    return shared(a, 0, b, 0, off, &looks);
}

Extent matrix(const void *p, int type, int64_t rows, int64_t stride, int64_t dim) {
    return extent(p, element_bytes(type), dim, &rows, &stride, 1);
}

// What the moves between tokens and rows have in common.
int check_move(int64_t tokens, int choices, int64_t capacity, int64_t dim, int type) {
    if (tokens < 0 || choices < 1 || choices > BMMC_MAX_CHOICES || capacity < 0 || dim < 1 ||
        dim > kMaxIndex / 2 || capacity > kMaxIndex || tokens > kMaxIndex / choices ||
        !data_type(type))
        return BMMC_ERR_INVALID_ARG;
    return BMMC_OK;
}

bool read_matrix_ok(const void *p, int type, int64_t stride) {
    return p && aligned(p, element_bytes(type)) && stride_ok(stride);
}

bool written_matrix_ok(const void *p, int type, int64_t rows, int64_t stride, int64_t dim) {
    return read_matrix_ok(p, type, stride) && (rows <= 1 || stride >= dim);
}

bool weights_ok(const void *p, int weight_type, int type) {
    return (weight_type == BMMC_F32 || weight_type == type) &&
           aligned(p, element_bytes(weight_type));
}

int check_rotation(const bmmc_rotation &r, int head_dim) {
    if (r.pairs < 1 || 2 * (int64_t)r.pairs > head_dim || r.axes < 1 || r.axes > BMMC_MAX_AXES ||
        !stride_ok(r.axis_stride) || !index_type_ok(r.position_type) || !r.freqs)
        return BMMC_ERR_INVALID_ARG;
    if (!aligned(r.freqs, r.freqs_are_64 ? 8 : 4) || !aligned(r.axis_of_pair, 4) ||
        !aligned(r.positions, r.position_type == BMMC_I64 ? 8 : 4))
        return BMMC_ERR_INVALID_ARG;
    return BMMC_OK;
}

struct HeadsExtent {
    Extent in, out;
};

// The heads' strides and pointers; `writes`: they have an out.
int check_heads(const bmmc_heads &x, int64_t batch, int64_t tokens, int dim, int type,
                bool writes, HeadsExtent *e) {
    const int bytes = element_bytes(type);
    if (x.heads < 1 || x.heads > kMaxHeads || !x.in || !aligned(x.in, bytes) ||
        !stride_ok(x.in_batch) || !stride_ok(x.in_token) || !stride_ok(x.in_head))
        return BMMC_ERR_INVALID_ARG;
    const int64_t sizes[3] = {batch, tokens, x.heads};
    const int64_t is[3] = {x.in_batch, x.in_token, x.in_head};
    e->in = extent(x.in, bytes, dim, sizes, is, 3);
    if (!writes) return BMMC_OK;
    if (!x.out || !aligned(x.out, bytes) || !stride_ok(x.out_batch) || !stride_ok(x.out_token) ||
        !stride_ok(x.out_head))
        return BMMC_ERR_INVALID_ARG;
    const int64_t os[3] = {x.out_batch, x.out_token, x.out_head};
    if (!apart(dim, sizes, os, 3)) return BMMC_ERR_ALIAS;
    e->out = extent(x.out, bytes, dim, sizes, os, 3);
    bool same = x.in == x.out;
    for (int i = 0; i < 3; ++i) same &= sizes[i] <= 1 || is[i] == os[i];
    if (!same && meet(e->in, e->out)) return BMMC_ERR_ALIAS;
    return BMMC_OK;
}

Steps steps_in(const bmmc_heads &x, int64_t batch, int64_t tokens, int dim) {
    const int64_t sizes[3] = {batch, tokens, x.heads};
    const int64_t strides[3] = {x.in_batch, x.in_token, x.in_head};
    return Steps(dim, sizes, strides, 3);
}

Steps steps_out(const bmmc_heads &x, int64_t batch, int64_t tokens, int dim) {
    const int64_t sizes[3] = {batch, tokens, x.heads};
    const int64_t strides[3] = {x.out_batch, x.out_token, x.out_head};
    return Steps(dim, sizes, strides, 3);
}

int check_cache(const bmmc_paged_cache &c, int64_t pages, int64_t page_size, int64_t heads,
                int dim, int type, Extent *e) {
    if ((c.type != type && c.type != BMMC_E4M3) || !stride_ok(c.page_stride) ||
        !stride_ok(c.place_stride) || !stride_ok(c.head_stride))
        return BMMC_ERR_INVALID_ARG;
    if (c.type == BMMC_E4M3 ? !c.scale || !aligned(c.scale, 4) ||
                                  (c.scale_stride != 0 && c.scale_stride != 1)
                            : c.scale != nullptr)
        return BMMC_ERR_INVALID_ARG;
    const int bytes = element_bytes(c.type);
    if (pages && (!c.data || !aligned(c.data, bytes))) return BMMC_ERR_INVALID_ARG;
    const int64_t sizes[3] = {pages, page_size, heads};
    const int64_t strides[3] = {c.page_stride, c.place_stride, c.head_stride};
    if (!apart(dim, sizes, strides, 3)) return BMMC_ERR_ALIAS;
    *e = extent(c.data, bytes, dim, sizes, strides, 3);
    return BMMC_OK;
}

Steps steps_of(const bmmc_paged_cache &c, int64_t pages, int64_t page_size, int64_t heads, int dim) {
    const int64_t sizes[3] = {pages, page_size, heads};
    const int64_t strides[3] = {c.page_stride, c.place_stride, c.head_stride};
    return Steps(dim, sizes, strides, 3);
}

}  // namespace

extern "C" {

int64_t bmmc_expert_rows(int64_t n, int num_experts, int64_t align) {
    if (n < 0 || n > kMaxIndex || num_experts < 1 || num_experts > BMMC_MAX_EXPERTS ||
        align < 1 || align > kMaxIndex)
        return -1;
    const int64_t held = n < num_experts ? n : num_experts;
    const int64_t rows = n + held * (align - 1);
    return rows > kMaxIndex ? -1 : rows;
}

int64_t bmmc_expert_order_workspace(int64_t n, int num_experts) {
    if (n < 0 || n > kMaxIndex || num_experts < 1 || num_experts > BMMC_MAX_EXPERTS) return -1;
    const int blocks = bmmc::order_cut(n).blocks;
    return blocks > 1 ? (int64_t)blocks * num_experts * (int64_t)sizeof(int32_t) : 0;
}

int bmmc_expert_order(const void *experts, int index_type, int64_t n, int num_experts,
                      int64_t align, int32_t *offsets, int32_t *counts, int32_t *rows,
                      int32_t *slots, void *workspace, int64_t workspace_bytes, void *stream) {
    const int64_t capacity = bmmc_expert_rows(n, num_experts, align);
    if (capacity < 0 || !index_type_ok(index_type) || !offsets || !counts)
        return BMMC_ERR_INVALID_ARG;
    if (n && (!experts || !rows || !slots)) return BMMC_ERR_INVALID_ARG;
    if (!aligned(experts, index_type == BMMC_I64 ? 8 : 4) || !aligned(offsets, 4) ||
        !aligned(counts, 4) || !aligned(rows, 4) || !aligned(slots, 4) || !aligned(workspace, 4))
        return BMMC_ERR_INVALID_ARG;
    const int64_t need = bmmc_expert_order_workspace(n, num_experts);
    if (need && (!workspace || workspace_bytes < need)) return BMMC_ERR_INVALID_ARG;
    const bmmc::OrderCut cut = bmmc::order_cut(n);
    bmmc::OrderArgs a{};
    a.experts = experts;
    a.is64 = index_type == BMMC_I64;
    a.num_experts = num_experts;
    a.n = n;
    a.align = align;
    a.capacity = capacity;
    a.chunk = cut.chunk;
    a.offsets = offsets;
    a.counts = counts;
    a.rows = rows;
    a.slots = slots;
    a.hist = static_cast<int32_t *>(workspace);
    return bmmc::launch_expert_order(a, cut.blocks, static_cast<hipStream_t>(stream));
}

int bmmc_expert_gather(const void *x, int64_t x_stride, const int32_t *rows,
                       const int32_t *slots, int64_t tokens, int choices, int64_t capacity,
                       int64_t dim, int type, void *out, int64_t out_stride, void *stream) {
    const int st = check_move(tokens, choices, capacity, dim, type);
    if (st != BMMC_OK) return st;
    if (capacity == 0 && tokens) return BMMC_ERR_INVALID_ARG;
    if (capacity == 0) return BMMC_OK;
    if (!slots || !aligned(slots, 4) || (tokens && (!rows || !aligned(rows, 4))))
        return BMMC_ERR_INVALID_ARG;
    if ((tokens && !read_matrix_ok(x, type, x_stride)) ||
        !written_matrix_ok(out, type, capacity, out_stride, dim))
        return BMMC_ERR_INVALID_ARG;
    if (meet(matrix(x, type, tokens, x_stride, dim), matrix(out, type, capacity, out_stride, dim)))
        return BMMC_ERR_ALIAS;
    bmmc::MoveArgs a{};
    a.x = x;
    a.rows = rows;
    a.slots = slots;
    a.out = out;
    a.x_stride = x_stride;
    a.out_stride = out_stride;
    a.tokens = tokens;
    a.capacity = capacity;
    a.dim = dim;
    a.choices = choices;
    return bmmc::launch_expert_gather(a, type, static_cast<hipStream_t>(stream));
}

int bmmc_expert_combine(const void *in, int64_t in_stride, const int32_t *rows,
                        const void *weights, int weight_type, int64_t tokens, int choices,
                        int64_t capacity, int64_t dim, int type, void *out, int64_t out_stride,
                        void *stream) {
    const int st = check_move(tokens, choices, capacity, dim, type);
    if (st != BMMC_OK) return st;
    if (tokens == 0) return BMMC_OK;
    // a dropped choice may read row 0, so that there is at least one
    if (capacity < 1 || !rows || !aligned(rows, 4) || !read_matrix_ok(in, type, in_stride) ||
        !written_matrix_ok(out, type, tokens, out_stride, dim) ||
        (weights && !weights_ok(weights, weight_type, type)))
        return BMMC_ERR_INVALID_ARG;
    if (meet(matrix(in, type, capacity, in_stride, dim), matrix(out, type, tokens, out_stride, dim)))
        return BMMC_ERR_ALIAS;
    bmmc::MoveArgs a{};
    a.x = in;
    a.rows = rows;
    a.weights = weights;
    a.weights_are_f32 = weight_type == BMMC_F32;
    a.out = out;
    a.x_stride = in_stride;
    a.out_stride = out_stride;
    a.tokens = tokens;
    a.capacity = capacity;
    a.dim = dim;
    a.choices = choices;
    return bmmc::launch_expert_combine(a, type, static_cast<hipStream_t>(stream));
}

int bmmc_expert_combine_backward(const void *grad, int64_t grad_stride, const void *in,
                                 int64_t in_stride, const int32_t *rows, const int32_t *slots,
                                 const void *weights, int weight_type, int64_t tokens,
                                 int choices, int64_t capacity, int64_t dim, int type,
                                 void *grad_in, int64_t grad_in_stride, void *grad_weights,
                                 void *stream) {
    const int st = check_move(tokens, choices, capacity, dim, type);
    if (st != BMMC_OK) return st;
    if (capacity == 0 && tokens) return BMMC_ERR_INVALID_ARG;
    if (capacity == 0) return BMMC_OK;
    if (!slots || !aligned(slots, 4) || !weights_ok(weights, weight_type, type) ||
        !written_matrix_ok(grad_in, type, capacity, grad_in_stride, dim))
        return BMMC_ERR_INVALID_ARG;
    if (tokens &&
        (!rows || !aligned(rows, 4) || !weights || !grad_weights ||
         !aligned(grad_weights, element_bytes(weight_type)) ||
         !read_matrix_ok(grad, type, grad_stride) || !read_matrix_ok(in, type, in_stride)))
        return BMMC_ERR_INVALID_ARG;
    const Extent out = matrix(grad_in, type, capacity, grad_in_stride, dim);
    if (meet(matrix(grad, type, tokens, grad_stride, dim), out) ||
        (tokens && meet(matrix(in, type, capacity, in_stride, dim), out)))
        return BMMC_ERR_ALIAS;
    bmmc::MoveArgs a{};
    a.x = grad;
    a.in = in;
    a.rows = rows;
    a.slots = slots;
    a.weights = weights;
    a.weights_are_f32 = weight_type == BMMC_F32;
    a.out = grad_in;
    a.grad_weights = grad_weights;
    a.x_stride = grad_stride;
    a.in_stride = in_stride;
    a.out_stride = grad_in_stride;
    a.tokens = tokens;
    a.capacity = capacity;
    a.dim = dim;
    a.choices = choices;
    return bmmc::launch_expert_combine_backward(a, type, static_cast<hipStream_t>(stream));
}

int bmmc_rotary(const bmmc_heads *x, int count, int64_t batch, int64_t tokens, int head_dim,
                int type, const bmmc_rotation *rotation, void *stream) {
    if (!x || !rotation || count < 1 || count > 2 || batch < 0 || tokens < 0 || head_dim < 1 ||
        head_dim > BMMC_MAX_HEAD_DIM || !data_type(type))
        return BMMC_ERR_INVALID_ARG;
    if (batch > kMaxIndex || (batch && tokens > kMaxIndex / batch)) return BMMC_ERR_INVALID_ARG;
    const int rt = check_rotation(*rotation, head_dim);
    if (rt != BMMC_OK) return rt;
    if (batch == 0 || tokens == 0) return BMMC_OK;
    if (!rotation->positions) return BMMC_ERR_INVALID_ARG;
    HeadsExtent e[2];
    for (int i = 0; i < count; ++i) {
        const int st = check_heads(x[i], batch, tokens, head_dim, type, true, &e[i]);
        if (st != BMMC_OK) return st;
    }
    for (int i = 0; i < count && count == 2; ++i) {
        const bmmc_heads &mine = x[i], &other = x[1 - i];
        if (mine.out != mine.in) {
            if (meet(e[i].out, e[1 - i].in) || meet(e[i].out, e[1 - i].out)) return BMMC_ERR_ALIAS;
            continue;
        }
        // views of one projection turned in place lie between one another, but
        // what one of them writes the other must neither read nor write
        const Steps out = steps_out(mine, batch, tokens, head_dim);
        const int bytes = element_bytes(type);
        if (share(mine.out, out, other.in, steps_in(other, batch, tokens, head_dim), bytes) ||
            share(mine.out, out, other.out, steps_out(other, batch, tokens, head_dim), bytes))
            return BMMC_ERR_ALIAS;
    }
    bmmc::HeadsArgs a{x, count, head_dim, type, batch, tokens};
    return bmmc::launch_rotary(a, *rotation, static_cast<hipStream_t>(stream));
}

int bmmc_cache_append(const bmmc_heads *q, const bmmc_heads *k, const bmmc_heads *v,
                      const bmmc_paged_cache *k_cache, const bmmc_paged_cache *v_cache,
                      int64_t pages, int64_t page_size, const int32_t *table, int64_t batch,
                      int64_t table_width, int64_t table_stride, const int32_t *sequences,
                      const void *positions, int position_type, const bmmc_rotation *rotation,
                      int64_t tokens, int k_dim, int v_dim, int type, void *stream) {
    if (!k || !v || !k_cache || !v_cache || pages < 0 || pages > kMaxIndex || page_size < 1 ||
        page_size > kMaxIndex || batch < 0 || batch > kMaxIndex || table_width < 0 ||
        table_width > kMaxIndex || !stride_ok(table_stride) || tokens < 0 || tokens > kMaxIndex ||
        k_dim < 1 || k_dim > BMMC_MAX_HEAD_DIM || v_dim < 1 || v_dim > BMMC_MAX_HEAD_DIM ||
        !data_type(type) || !index_type_ok(position_type) || (q && !rotation))
        return BMMC_ERR_INVALID_ARG;
    if (rotation) {
        const int rt = check_rotation(*rotation, k_dim);
        if (rt != BMMC_OK) return rt;
        if (!rotation->positions && rotation->axes != 1) return BMMC_ERR_INVALID_ARG;
    }
    if (tokens == 0) return BMMC_OK;
    if (!positions || !aligned(positions, position_type == BMMC_I64 ? 8 : 4) ||
        !aligned(sequences, 4) || !aligned(table, 4) || (batch && table_width && !table))
        return BMMC_ERR_INVALID_ARG;
    if (k->heads != v->heads || k_cache->type != v_cache->type) return BMMC_ERR_INVALID_ARG;
    HeadsExtent qe{}, ke{}, ve{};
    Extent kc, vc;
    int st = check_heads(*k, 1, tokens, k_dim, type, false, &ke);
    if (st == BMMC_OK) st = check_heads(*v, 1, tokens, v_dim, type, false, &ve);
    if (st == BMMC_OK && q) st = check_heads(*q, 1, tokens, k_dim, type, true, &qe);
    if (st == BMMC_OK) st = check_cache(*k_cache, pages, page_size, k->heads, k_dim, type, &kc);
    if (st == BMMC_OK) st = check_cache(*v_cache, pages, page_size, k->heads, v_dim, type, &vc);
    if (st != BMMC_OK) return st;
    // the two caches may lie in one array, with no element in both; nothing that
    // is read may lie in a cache
    if (pages && share(k_cache->data, steps_of(*k_cache, pages, page_size, k->heads, k_dim),
                       v_cache->data, steps_of(*v_cache, pages, page_size, k->heads, v_dim),
                       element_bytes(k_cache->type)))
        return BMMC_ERR_ALIAS;
    for (const Extent &c : {kc, vc})
        if (meet(c, ke.in) || meet(c, ve.in) || (q && (meet(c, qe.in) || meet(c, qe.out))))
            return BMMC_ERR_ALIAS;
    if (q && q->in != q->out && (meet(qe.out, ke.in) || meet(qe.out, ve.in)))
        return BMMC_ERR_ALIAS;
    // queries turned in place may lie between the keys and values, as in bmmc_rotary
    if (q && q->in == q->out) {
        const Steps out = steps_out(*q, 1, tokens, k_dim);
        const int bytes = element_bytes(type);
        if (share(q->out, out, k->in, steps_in(*k, 1, tokens, k_dim), bytes) ||
            share(q->out, out, v->in, steps_in(*v, 1, tokens, v_dim), bytes))
            return BMMC_ERR_ALIAS;
    }
    bmmc::AppendArgs a{};
    if (q) a.q = *q;
    a.k = *k;
    a.v = *v;
    a.k_cache = *k_cache;
    a.v_cache = *v_cache;
    a.where = bmmc::PageTable{table,       sequences, positions, batch, table_width,
                              table_stride, pages,     page_size, position_type == BMMC_I64};
    if (rotation) {
        a.rotation = *rotation;
        if (!rotation->positions) {
            a.rotation.positions = positions;
            a.rotation.position_type = position_type;
            a.rotation.axis_stride = 0;
        }
    }
    a.tokens = tokens;
    a.k_dim = k_dim;
    a.v_dim = v_dim;
    a.type = type;
    return bmmc::launch_cache_append(a, static_cast<hipStream_t>(stream));
}

}  // extern "C"
