// api.cpp -- the extern "C" entry points declared in include/bmmc_layer.h:
// every argument check, before any HIP call, and the kernels' arguments.
#include <hip/hip_runtime.h>

#include <cmath>

#include "../../../include/bmmc_layer.h"
#include "../tokens/checks.h"
#include "layer.h"

using namespace bmmc;

namespace {

struct CacheExtent {
    Extent data, scale;
};

// A cache's type, strides and pointers.  `written`: its elements, and the scales
// that go with them, lie apart.
int check_scaled(const bmmc_scaled_cache &c, int64_t pages, int64_t page_size, int64_t heads,
                 int dim, int type, bool written, CacheExtent *e) {
    if ((c.type != type && c.type != BMMC_E4M3) || !stride_ok(c.page_stride) ||
        !stride_ok(c.place_stride) || !stride_ok(c.head_stride))
        return BMMC_ERR_INVALID_ARG;
    const int bytes = element_bytes(c.type);
    if (pages && (!c.data || !aligned(c.data, bytes))) return BMMC_ERR_INVALID_ARG;
    const int64_t sizes[3] = {pages, page_size, heads};
    const int64_t strides[3] = {c.page_stride, c.place_stride, c.head_stride};
    if (written && !apart(dim, sizes, strides, 3)) return BMMC_ERR_ALIAS;
    e->data = extent(c.data, bytes, dim, sizes, strides, 3);
    e->scale = Extent{0, 0};
    if (c.type != BMMC_E4M3) return c.scale ? BMMC_ERR_INVALID_ARG : BMMC_OK;
    if ((pages && !c.scale) || !aligned(c.scale, 4) || !stride_ok(c.scale_page) ||
        !stride_ok(c.scale_place) || !stride_ok(c.scale_head))
        return BMMC_ERR_INVALID_ARG;
    const int64_t by[3] = {c.scale_page, c.scale_place, c.scale_head};
    if (written && !apart(1, sizes, by, 3)) return BMMC_ERR_ALIAS;
    e->scale = extent(c.scale, 4, 1, sizes, by, 3);
    return BMMC_OK;
}

Steps data_steps(const bmmc_scaled_cache &c, int64_t pages, int64_t page_size, int64_t heads, int dim) {
    const int64_t sizes[3] = {pages, page_size, heads};
    const int64_t strides[3] = {c.page_stride, c.place_stride, c.head_stride};
    return Steps(dim, sizes, strides, 3);
}

Steps scale_steps(const bmmc_scaled_cache &c, int64_t pages, int64_t page_size, int64_t heads) {
    const int64_t sizes[3] = {pages, page_size, heads};
    const int64_t strides[3] = {c.scale_page, c.scale_place, c.scale_head};
    return Steps(1, sizes, strides, 3);
}

// Whether the scales differ by place, and not by head alone.
bool by_place(const bmmc_scaled_cache &c, int64_t pages, int64_t page_size) {
    return c.type == BMMC_E4M3 &&
           ((pages > 1 && c.scale_page) || (page_size > 1 && c.scale_place));
}

// What the calls on a paged cache have in common: sizes, and the table itself.
bool page_sizes_ok(int64_t pages, int64_t page_size, int64_t batch, int64_t table_width,
                   int64_t table_stride) {
    return pages >= 0 && pages <= kMaxIndex && page_size >= 1 && page_size <= kMaxIndex && batch >= 0 &&
           batch <= kMaxIndex && table_width >= 0 && table_width <= kMaxIndex && stride_ok(table_stride);
}
bool table_ok(const int32_t *table, int64_t batch, int64_t table_width) {
    return aligned(table, 4) && (!batch || !table_width || table);
}
int check_pages(int64_t pages, int64_t page_size, const int32_t *table, int64_t batch,
                int64_t table_width, int64_t table_stride) {
    return page_sizes_ok(pages, page_size, batch, table_width, table_stride) &&
                   table_ok(table, batch, table_width)
               ? BMMC_OK
               : BMMC_ERR_INVALID_ARG;
}

int check_places(int64_t tokens, const int32_t *sequences, const void *positions,
                 int position_type) {
    if (tokens < 0 || tokens > kMaxIndex || !index_type_ok(position_type) ||
        (tokens && !positions) || !aligned(positions, position_type == BMMC_I64 ? 8 : 4) ||
        !aligned(sequences, 4))
        return BMMC_ERR_INVALID_ARG;
    return BMMC_OK;
}

// Numbers that a call reads besides rows: `rows` times `bytes` bytes, `stride` bytes apart.
struct Numbers {
    const void *at = nullptr;
    int64_t bytes = 0, rows = 0, stride = 0;
    Extent all{0, 0};
    Numbers() {}
    Numbers(const void *p, int64_t n, int64_t rows_, int64_t stride_)
        : at(p), bytes(p ? n : 0), rows(rows_), stride(stride_) {
        if (bytes > 0) all = extent(p, 1, bytes, &rows, &stride, 1);
    }
};

Numbers flat(const void *p, int64_t bytes) { return Numbers(p, bytes, 1, 0); }

Numbers table_of(const int32_t *table, int64_t batch, int64_t width, int64_t stride) {
    return Numbers(table, 4 * width, batch, 4 * stride);
}

// Whether a written array, of extent e, has a byte of what is read.  Its steps are
// looked at only where the two extents meet, as they seldom do.
template <class F>
bool overwrites(const void *p, const Extent &e, F steps, int element, const Numbers &r) {
    if (!meet(e, r.all)) return false;
    Steps in_bytes = steps();
    in_bytes.inner *= element;
    for (int i = 0; i < in_bytes.dims; ++i) in_bytes.strides[i] *= element;
    return share(p, in_bytes, r.at, Steps(r.bytes, &r.rows, &r.stride, 1), 1);
}

bool dim_ok(int dim, int least) { return dim >= least && dim <= BMMC_MAX_HEAD_DIM; }

// Sizes of an attention alone; of its pointers only whether there are starts.
int check_attention_sizes(const bmmc_attention &a) {
    if (a.tokens < 0 || a.tokens > kMaxIndex || a.heads < 1 || a.q_heads < 1 ||
        a.q_heads > kMaxHeads || a.heads > a.q_heads || a.q_heads % a.heads ||
        !dim_ok(a.k_dim, BMMC_LEAST_ATTENDED) || !dim_ok(a.v_dim, BMMC_LEAST_ATTENDED) ||
        !data_type(a.type) || a.window < 0 ||
        !(a.scale > 0.0f) || !std::isfinite(a.scale) || (!a.starts && a.batch != a.tokens))
        return BMMC_ERR_INVALID_ARG;
    if (a.tokens > kMaxIndex / (a.q_heads / a.heads)) return BMMC_ERR_INVALID_ARG;
    return page_sizes_ok(a.pages, a.page_size, a.batch, a.table_width, a.table_stride)
               ? BMMC_OK
               : BMMC_ERR_INVALID_ARG;
}

int32_t pitch_of(const bmmc_attention &a) { return (a.v_dim + 3) / 4 * 4; }

int64_t workspace_floats(const bmmc_attention &a, const AttendPlan &p) {
    return 2 * (int64_t)p.shares * a.heads * p.rows * pitch_of(a);
}
int64_t workspace_states(const bmmc_attention &a, const AttendPlan &p) {
    return 2 * (int64_t)p.shares * a.heads * p.rows;
}

}  // namespace

extern "C" {

int64_t bmmc_cache_attention_workspace(const bmmc_attention *a) {
    if (!a || check_attention_sizes(*a) != BMMC_OK) return -1;
    if (a->tokens == 0) return 0;
    const AttendPlan p = attend_plan(*a);
    return workspace_floats(*a, p) * 4 + workspace_states(*a, p) * 8 + p.shares * 16;
}

int bmmc_cache_attention(const bmmc_attention *a, const bmmc_scaled_cache *k_cache,
                         const bmmc_scaled_cache *v_cache, void *workspace,
                         int64_t workspace_bytes, void *stream) {
    if (!a || !k_cache || !v_cache) return BMMC_ERR_INVALID_ARG;
    int st = check_attention_sizes(*a);
    if (st != BMMC_OK) return st;
    const int64_t need = bmmc_cache_attention_workspace(a);
    if (!table_ok(a->table, a->batch, a->table_width) || !stride_ok(a->q_token) ||
        !stride_ok(a->q_head) || !stride_ok(a->out_token) || !stride_ok(a->out_head) ||
        !aligned(workspace, 16) || workspace_bytes < 0)
        return BMMC_ERR_INVALID_ARG;
    if (a->tokens == 0) return BMMC_OK;
    const int bytes = element_bytes(a->type);
    if (!a->q || !aligned(a->q, bytes) || !a->out || !aligned(a->out, bytes) ||
        !aligned(a->lengths, 4) || !aligned(a->starts, 4) || (a->batch && !a->lengths) ||
        k_cache->type != v_cache->type || (need && (!workspace || workspace_bytes < need)))
        return BMMC_ERR_INVALID_ARG;
    CacheExtent ke, ve;
    st = check_scaled(*k_cache, a->pages, a->page_size, a->heads, a->k_dim, a->type, false, &ke);
    if (st == BMMC_OK)
        st = check_scaled(*v_cache, a->pages, a->page_size, a->heads, a->v_dim, a->type, false, &ve);
    if (st != BMMC_OK) return st;
    const int64_t sizes[2] = {a->tokens, a->q_heads};
    const int64_t qs[2] = {a->q_token, a->q_head}, os[2] = {a->out_token, a->out_head};
    if (!apart(a->v_dim, sizes, os, 2)) return BMMC_ERR_ALIAS;
    const Extent out = extent(a->out, bytes, a->v_dim, sizes, os, 2);
    const Extent q = extent(a->q, bytes, a->k_dim, sizes, qs, 2);
    const Extent work{(uintptr_t)workspace, (uintptr_t)workspace + (uintptr_t)need};
    if (meet(out, work)) return BMMC_ERR_ALIAS;
    for (const Extent &e : {q, ke.data, ke.scale, ve.data, ve.scale})
        if (meet(out, e) || meet(work, e)) return BMMC_ERR_ALIAS;
    for (const Numbers &r : {table_of(a->table, a->batch, a->table_width, a->table_stride),
                             flat(a->lengths, 4 * a->batch), flat(a->starts, 4 * (a->batch + 1))})
        if (overwrites(a->out, out, [&] { return Steps(a->v_dim, sizes, os, 2); }, bytes, r) ||
            overwrites(workspace, work, [&] { return Steps(need, nullptr, nullptr, 0); }, 1, r))
            return BMMC_ERR_ALIAS;
    AttendArgs x{};
    x.a = *a;
    x.k = *k_cache;
    x.v = *v_cache;
    x.plan = attend_plan(*a);
    x.group = (int32_t)(a->q_heads / a->heads);
    x.by_group = fast_div((uint32_t)x.group);
    x.by_page = fast_div((uint32_t)a->page_size);
    x.rows_scaled = by_place(*k_cache, a->pages, a->page_size) ||
                    by_place(*v_cache, a->pages, a->page_size);
    // places and the tiles behind them stay in 32 bits
    x.reach = std::min(a->table_width * a->page_size, kMaxIndex - 4096);
    x.a.window = std::min(a->window, kMaxIndex);
    x.pitch = pitch_of(*a);
    x.partial = static_cast<float *>(workspace);
    x.state = reinterpret_cast<float2 *>(x.partial + workspace_floats(*a, x.plan));
    x.begun = reinterpret_cast<int4 *>(x.state + workspace_states(*a, x.plan));
    x.by_shares = fast_div((uint32_t)std::max(x.plan.shares, 1));
    // however the sequences lie, none has more tiles than all rows make
    x.few_units = (double)std::max<int64_t>(a->batch, 1) * (double)x.plan.tiles *
                      ((double)x.reach / x.plan.unit + 2) < 2147483648.0;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    st = x.plan.rows > 16 ? launch_attend_many(x, s) : launch_attend_few(x, s);
    return st == BMMC_OK && x.plan.shares ? launch_attend_join(x, s) : st;
}

int bmmc_cache_quantize(const bmmc_heads *q, const bmmc_heads *k, const bmmc_heads *v,
                        const bmmc_scaled_cache *k_cache, const bmmc_scaled_cache *v_cache,
                        int64_t pages, int64_t page_size, const int32_t *table, int64_t batch,
                        int64_t table_width, int64_t table_stride, const int32_t *sequences,
                        const void *positions, int position_type, const bmmc_rotation *rotation,
                        int64_t tokens, int k_dim, int v_dim, int type, void *stream) {
    if (!k || !v || !k_cache || !v_cache || !dim_ok(k_dim, 1) || !dim_ok(v_dim, 1) ||
        !data_type(type) || (q && !rotation) || k->heads != v->heads ||
        k_cache->type != BMMC_E4M3 || v_cache->type != BMMC_E4M3)
        return BMMC_ERR_INVALID_ARG;
    int st = check_pages(pages, page_size, table, batch, table_width, table_stride);
    if (st == BMMC_OK) st = check_places(tokens, sequences, positions, position_type);
    if (st == BMMC_OK && rotation) {
        st = check_rotation(*rotation, k_dim);
        if (st == BMMC_OK && !rotation->positions && rotation->axes != 1) st = BMMC_ERR_INVALID_ARG;
    }
    if (st != BMMC_OK || tokens == 0) return st;
    HeadsExtent qe{}, ke{}, ve{};
    st = check_heads(*k, 1, tokens, k_dim, type, false, &ke);
    if (st == BMMC_OK) st = check_heads(*v, 1, tokens, v_dim, type, false, &ve);
    if (st == BMMC_OK && q) st = check_heads(*q, 1, tokens, k_dim, type, true, &qe);
    CacheExtent kc, vc;
    if (st == BMMC_OK)
        st = check_scaled(*k_cache, pages, page_size, k->heads, k_dim, type, true, &kc);
    if (st == BMMC_OK)
        st = check_scaled(*v_cache, pages, page_size, k->heads, v_dim, type, true, &vc);
    if (st != BMMC_OK) return st;
    // The caches may lie in one array, with no element in both, and so may their
    // scales; scales and caches may not, and nothing that is read lies in either.
    if (pages &&
        (share(k_cache->data, data_steps(*k_cache, pages, page_size, k->heads, k_dim),
               v_cache->data, data_steps(*v_cache, pages, page_size, k->heads, v_dim), 1) ||
         share(k_cache->scale, scale_steps(*k_cache, pages, page_size, k->heads), v_cache->scale,
               scale_steps(*v_cache, pages, page_size, k->heads), 4)))
        return BMMC_ERR_ALIAS;
    for (const Extent &c : {kc.scale, vc.scale})
        if (meet(c, kc.data) || meet(c, vc.data)) return BMMC_ERR_ALIAS;
    for (const Extent &c : {kc.data, kc.scale, vc.data, vc.scale})
        if (meet(c, ke.in) || meet(c, ve.in) || (q && (meet(c, qe.in) || meet(c, qe.out))))
            return BMMC_ERR_ALIAS;
    if (q && q->in != q->out && (meet(qe.out, ke.in) || meet(qe.out, ve.in)))
        return BMMC_ERR_ALIAS;
    // queries turned in place may lie between the keys and values, views of one projection
    if (q && q->in == q->out) {
        const Steps out = steps_out(*q, 1, tokens, k_dim);
        const int bytes = element_bytes(type);
        if (share(q->out, out, k->in, steps_in(*k, 1, tokens, k_dim), bytes) ||
            share(q->out, out, v->in, steps_in(*v, 1, tokens, v_dim), bytes))
            return BMMC_ERR_ALIAS;
    }
    const int64_t each = position_type == BMMC_I64 ? 8 : 4;
    Numbers numbers[6] = {table_of(table, batch, table_width, table_stride),
                          flat(sequences, 4 * tokens), flat(positions, each * tokens)};
    if (rotation) {
        const int64_t turn = rotation->position_type == BMMC_I64 ? 8 : 4;
        numbers[3] = flat(rotation->freqs, rotation->pairs * (rotation->freqs_are_64 ? 8 : 4));
        numbers[4] = flat(rotation->axis_of_pair, rotation->pairs * 4);
        if (rotation->positions)
            numbers[5] = Numbers(rotation->positions, turn * tokens, rotation->axes,
                                 turn * rotation->axis_stride);
    }
    const auto data = [&](const bmmc_scaled_cache &c, int dim) {
        return [&c, dim, pages, page_size, k] { return data_steps(c, pages, page_size, k->heads, dim); };
    };
    const auto scale = [&](const bmmc_scaled_cache &c) {
        return [&c, pages, page_size, k] { return scale_steps(c, pages, page_size, k->heads); };
    };
    for (const Numbers &r : numbers)
        if (overwrites(k_cache->data, kc.data, data(*k_cache, k_dim), 1, r) ||
            overwrites(v_cache->data, vc.data, data(*v_cache, v_dim), 1, r) ||
            overwrites(k_cache->scale, kc.scale, scale(*k_cache), 4, r) ||
            overwrites(v_cache->scale, vc.scale, scale(*v_cache), 4, r) ||
            (q && overwrites(q->out, qe.out, [&] { return steps_out(*q, 1, tokens, k_dim); },
                             element_bytes(type), r)))
            return BMMC_ERR_ALIAS;
    QuantizeArgs a{};
    if (q) a.q = *q;
    a.k = *k;
    a.v = *v;
    a.k_cache = *k_cache;
    a.v_cache = *v_cache;
    a.where = PageTable{table,        sequences, positions, batch, table_width,
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
    return launch_cache_quantize(a, static_cast<hipStream_t>(stream));
}

int bmmc_cache_read(const bmmc_heads *k, const bmmc_heads *v, const bmmc_scaled_cache *k_cache,
                    const bmmc_scaled_cache *v_cache, int64_t pages, int64_t page_size,
                    const int32_t *table, int64_t batch, int64_t table_width,
                    int64_t table_stride, const int32_t *sequences, const void *positions,
                    int position_type, int64_t tokens, int k_dim, int v_dim, int type,
                    void *stream) {
    if (!k || !v || !k_cache || !v_cache || !dim_ok(k_dim, 1) || !dim_ok(v_dim, 1) ||
        !data_type(type) || k->heads != v->heads || k_cache->type != v_cache->type)
        return BMMC_ERR_INVALID_ARG;
    int st = check_pages(pages, page_size, table, batch, table_width, table_stride);
    if (st == BMMC_OK) st = check_places(tokens, sequences, positions, position_type);
    if (st != BMMC_OK || tokens == 0) return st;
    // what is written alone: each out as if it were turned in place
    bmmc_heads kh = *k, vh = *v;
    for (bmmc_heads *h : {&kh, &vh}) {
        h->in = h->out;
        h->in_batch = h->out_batch;
        h->in_token = h->out_token;
        h->in_head = h->out_head;
    }
    HeadsExtent ke{}, ve{};
    CacheExtent kc, vc;
    st = check_heads(kh, 1, tokens, k_dim, type, true, &ke);
    if (st == BMMC_OK) st = check_heads(vh, 1, tokens, v_dim, type, true, &ve);
    if (st == BMMC_OK)
        st = check_scaled(*k_cache, pages, page_size, k->heads, k_dim, type, false, &kc);
    if (st == BMMC_OK)
        st = check_scaled(*v_cache, pages, page_size, k->heads, v_dim, type, false, &vc);
    if (st != BMMC_OK) return st;
    // the two results may lie in one array, with no element in both
    if (share(k->out, steps_out(*k, 1, tokens, k_dim), v->out, steps_out(*v, 1, tokens, v_dim),
              element_bytes(type)))
        return BMMC_ERR_ALIAS;
    for (const Extent &c : {kc.data, kc.scale, vc.data, vc.scale})
        if (meet(c, ke.out) || meet(c, ve.out)) return BMMC_ERR_ALIAS;
    const int bytes = element_bytes(type);
    const int64_t each = position_type == BMMC_I64 ? 8 : 4;
    for (const Numbers &r : {table_of(table, batch, table_width, table_stride),
                             flat(sequences, 4 * tokens), flat(positions, each * tokens)})
        if (overwrites(k->out, ke.out, [&] { return steps_out(*k, 1, tokens, k_dim); }, bytes, r) ||
            overwrites(v->out, ve.out, [&] { return steps_out(*v, 1, tokens, v_dim); }, bytes, r))
            return BMMC_ERR_ALIAS;
    ReadArgs a{};
    a.k = *k;
    a.v = *v;
    a.k_cache = *k_cache;
    a.v_cache = *v_cache;
    a.where = PageTable{table,        sequences, positions, batch, table_width,
                        table_stride, pages,     page_size, position_type == BMMC_I64};
    a.tokens = tokens;
    a.k_dim = k_dim;
    a.v_dim = v_dim;
    a.type = type;
    return launch_cache_read(a, static_cast<hipStream_t>(stream));
}

int64_t bmmc_expert_balance_workspace(int64_t tokens, int num_experts) {
    if (tokens < 0 || tokens > kMaxIndex || num_experts < 1 || num_experts > BMMC_MAX_EXPERTS)
        return -1;
    // sums and counts of each workgroup, then how many have ended and their losses
    const int64_t ends = 1 + (num_experts + kBalanceColumns - 1) / kBalanceColumns;
    return ((int64_t)balance_blocks(tokens, num_experts) * (2 * (int64_t)num_experts + 1) + ends) * 4;
}

int bmmc_expert_balance(const void *logits, int64_t logits_stride, int type, int num_experts,
                        const void *experts, int index_type, int64_t tokens, int choices,
                        const uint8_t *mask, float *loss, int32_t *counts, float *slopes,
                        void *workspace, int64_t workspace_bytes, void *stream) {
    const int64_t need = bmmc_expert_balance_workspace(tokens, num_experts);
    if (need < 0 || choices < 1 || choices > BMMC_MAX_CHOICES || tokens > kMaxIndex / choices ||
        !data_type(type) || !index_type_ok(index_type) || !stride_ok(logits_stride) || !loss ||
        !counts || !slopes || !aligned(loss, 4) || !aligned(counts, 4) || !aligned(slopes, 4) ||
        !workspace || !aligned(workspace, 4) || workspace_bytes < need)
        return BMMC_ERR_INVALID_ARG;
    if (tokens && (!logits || !aligned(logits, element_bytes(type)) || !experts ||
                   !aligned(experts, index_type == BMMC_I64 ? 8 : 4)))
        return BMMC_ERR_INVALID_ARG;
    const auto flat = [](const void *p, int64_t bytes) {
        return Extent{(uintptr_t)p, (uintptr_t)p + (uintptr_t)bytes};
    };
    const Extent written[4] = {flat(loss, 4), flat(counts, 4 * (int64_t)num_experts),
                               flat(slopes, 4 * (int64_t)num_experts), flat(workspace, need)};
    const Extent read[3] = {
        extent(logits, element_bytes(type), num_experts, &tokens, &logits_stride, 1),
        flat(experts, tokens * choices * (index_type == BMMC_I64 ? 8 : 4)),
        flat(mask, mask ? tokens : 0)};
    for (int i = 0; i < 4; ++i) {
        for (const Extent &r : read)
            if (meet(written[i], r)) return BMMC_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (meet(written[i], written[j])) return BMMC_ERR_ALIAS;
    }
    BalanceArgs a{};
    a.logits = logits;
    a.stride = logits_stride;
    a.tokens = tokens;
    a.experts = experts;
    a.mask = mask;
    a.loss = loss;
    a.slopes = slopes;
    a.counts = counts;
    a.blocks = balance_blocks(tokens, num_experts);
    a.sums = static_cast<float *>(workspace);
    a.hits = static_cast<int32_t *>(workspace) + (int64_t)a.blocks * num_experts;
    a.num_experts = num_experts;
    a.choices = choices;
    a.by_choices = fast_div((uint32_t)choices);
    a.is64 = index_type == BMMC_I64;
    a.type = type;
    return launch_expert_balance(a, static_cast<hipStream_t>(stream));
}

int bmmc_expert_balance_backward(const float *grad, const void *logits, int64_t logits_stride,
                                 int type, int num_experts, const float *slopes, int64_t tokens,
                                 const uint8_t *mask, void *grad_logits, int64_t grad_stride,
                                 void *stream) {
    if (tokens < 0 || tokens > kMaxIndex || num_experts < 1 || num_experts > BMMC_MAX_EXPERTS ||
        !data_type(type) || !stride_ok(logits_stride) || !stride_ok(grad_stride))
        return BMMC_ERR_INVALID_ARG;
    if (tokens == 0) return BMMC_OK;
    const int bytes = element_bytes(type);
    if (!grad || !aligned(grad, 4) || !slopes || !aligned(slopes, 4) || !logits ||
        !aligned(logits, bytes) || !grad_logits || !aligned(grad_logits, bytes) ||
        (tokens > 1 && grad_stride < num_experts))
        return BMMC_ERR_INVALID_ARG;
    const Extent out = extent(grad_logits, bytes, num_experts, &tokens, &grad_stride, 1);
    const Extent in = extent(logits, bytes, num_experts, &tokens, &logits_stride, 1);
    const auto flat = [](const void *p, int64_t n) {
        return Extent{(uintptr_t)p, (uintptr_t)p + (uintptr_t)n};
    };
    for (const Extent &e : {in, flat(grad, 4), flat(slopes, 4 * (int64_t)num_experts),
                            flat(mask, mask ? tokens : 0)})
        if (meet(out, e)) return BMMC_ERR_ALIAS;
    BalanceArgs a{};
    a.logits = logits;
    a.stride = logits_stride;
    a.tokens = tokens;
    a.mask = mask;
    a.grad = grad;
    a.slopes = const_cast<float *>(slopes);
    a.grad_logits = grad_logits;
    a.grad_stride = grad_stride;
    a.num_experts = num_experts;
    a.type = type;
    return launch_expert_balance_backward(a, static_cast<hipStream_t>(stream));
}

}  // extern "C"
