/*
 * bmmc_layer.h -- what a decoder layer with experts over a paged cache needs
 * next to its moved rows (gfx950).
 *
 * bmmc_tokens.h moves rows of tokens: to their experts and back, and into a
 * paged cache.  These entry points read that cache and judge that router:
 *
 *   - attention of new tokens, one or a chunk for each sequence, over the cache;
 *   - a cache in 8 bits whose scales are made as it is written, and rows of a
 *     cache read back;
 *   - the balance loss of a router with the counts of its experts, and its
 *     gradient.
 *
 * The rules are those of bmmc_tokens.h: extern "C", device pointers of the
 * current device, a hipStream_t as void*, asynchronous, no allocation, every
 * argument check before the first HIP call, a BMMC_* status, capturable.
 * Strides count elements.  Index arrays are data: a wrong entry is skipped and
 * never reads or writes out of bounds.  What a call writes overlaps nothing
 * else that it reads or writes (BMMC_ERR_ALIAS).
 */
#ifndef BMMC_LAYER_H
#define BMMC_LAYER_H

#include "bmmc_tokens.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A paged cache and the scales of its 8-bit values: element d of head h at
 * place i of page p is data[p * page_stride + i * place_stride + h *
 * head_stride + d], and stands for that times scale[p * scale_page + i *
 * scale_place + h * scale_head].  Scales of each head alone have scale_page =
 * scale_place = 0.  With another type than BMMC_E4M3 scale is NULL. */
typedef struct bmmc_scaled_cache {
    void *data;
    float *scale;
    int64_t page_stride, place_stride, head_stride;
    int64_t scale_page, scale_place, scale_head;
    int type; /* the inputs' type or BMMC_E4M3 */
} bmmc_scaled_cache;

/* ---- attention over a paged cache --------------------------------------- */

#define BMMC_LEAST_ATTENDED 8 /* elements of a head, at least; at most BMMC_MAX_HEAD_DIM */

/* The new tokens of sequence s are rows starts[s] to starts[s + 1] - 1 (row s
 * alone where starts is NULL, batch = tokens then), the last of them at place
 * lengths[s] - 1 of the sequence, each one place after the one before; their
 * keys and values are in the cache already.  Place j of sequence s is page
 * table[s * table_stride + j / page_size], place j % page_size.
 *
 * The token at place p sees the places j <= p, with a window > 0 those with
 * j > p - window only, and of them those whose page is in [0, pages).  With
 * key head h' = h / (q_heads / heads) and a_j = scale <q[t, h], k[j, h']>
 *     out[t, h] = sum of exp(a_j) v[j, h'] / sum of exp(a_j)
 * over them, and zeros where there is none of any weight.  What a place that is
 * not seen holds does not matter, be it a NaN; places from 2^31 - 4097 on are not
 * seen.  A place that is seen counts
 * whatever its weight: an infinity or a NaN in its value shows.
 *
 * Scores, sums and the running maximum are in 32 bits; the weights of one
 * product with values, times their scales where those differ by place, are
 * rounded to `type`, or where that is BMMC_F16 and scales differ by place so that
 * 2^-16 of one is left out at most.  Rows of no sequence are left as
 * they are or, with clear_rest, those before the first and behind the last
 * sequence set to zeros.  starts must not fall; where it does, rows of some
 * sequences are not written. */
typedef struct bmmc_attention {
    const void *q; /* tokens, q_heads of k_dim elements */
    void *out;     /* tokens, q_heads of v_dim elements */
    int64_t q_token, q_head, out_token, out_head;
    int64_t tokens, q_heads, heads; /* q_heads a multiple of heads */
    const int32_t *table;           /* batch rows of table_width pages */
    const int32_t *lengths;         /* batch */
    const int32_t *starts;          /* batch + 1, or NULL */
    int64_t pages, page_size, batch, table_width, table_stride;
    int64_t window; /* 0: no bound */
    float scale;    /* above 0, finite */
    int k_dim, v_dim, type;
    int clear_rest;
} bmmc_attention;

/* Bytes of device workspace that the call needs, which depend on sizes and on
 * whether there are starts alone: other pointers are not looked at (-1 if a size
 * is out of range).  It needs no initial value, nothing is
 * kept in it from one call to the next, and calls that run at the same time
 * need one each. */
int64_t bmmc_cache_attention_workspace(const bmmc_attention *a);

int bmmc_cache_attention(const bmmc_attention *a, const bmmc_scaled_cache *k_cache,
                         const bmmc_scaled_cache *v_cache, void *workspace,
                         int64_t workspace_bytes, void *stream);

/* ---- a cache written in 8 bits, and read back ---------------------------- */

/* bmmc_cache_append into caches of BMMC_E4M3 whose scales are made on the way:
 * each head of each token that is stored has a scale of its own, its largest
 * finite magnitude / 448 (not below 2^-126, and 1 for a head without any but
 * zeros), written to where the cache's scales say, and value / scale is stored,
 * rounded to nearest; infinities become the type's largest value, NaN stays
 * NaN.  Magnitudes are those of the turned keys in 32 bits.  The other
 * arguments are bmmc_cache_append's.  No two scales of a cache share an
 * address, and none lies in a cache or in what is read.  Tokens of one call go
 * to places of their own: where two go to the same, its scale may be one's and
 * its values the other's. */
int bmmc_cache_quantize(const bmmc_heads *q, const bmmc_heads *k, const bmmc_heads *v,
                        const bmmc_scaled_cache *k_cache, const bmmc_scaled_cache *v_cache,
                        int64_t pages, int64_t page_size, const int32_t *table, int64_t batch,
                        int64_t table_width, int64_t table_stride, const int32_t *sequences,
                        const void *positions, int position_type, const bmmc_rotation *rotation,
                        int64_t tokens, int k_dim, int v_dim, int type, void *stream);

/* Rows of the caches brought back: row t of k's and v's out is the place
 * positions[t] of sequence sequences[t] (t where sequences is NULL), times its
 * scale, rounded once to `type`; zeros where there is no such place, as
 * bmmc_cache_append stores nothing there.  k->in, v->in, their strides and the
 * batch strides are not used. */
int bmmc_cache_read(const bmmc_heads *k, const bmmc_heads *v, const bmmc_scaled_cache *k_cache,
                    const bmmc_scaled_cache *v_cache, int64_t pages, int64_t page_size,
                    const int32_t *table, int64_t batch, int64_t table_width,
                    int64_t table_stride, const int32_t *sequences, const void *positions,
                    int position_type, int64_t tokens, int k_dim, int v_dim, int type,
                    void *stream);

/* ---- balance of a router ------------------------------------------------- */

/* With p = softmax of logits[t] (tokens rows of num_experts elements of
 * `type`), N the tokens with mask[t] != 0 (all where mask is NULL) and
 * counts[e] their choices of expert e (experts is tokens * choices; a value
 * outside [0, num_experts) is not counted):
 *     slopes[e] = num_experts counts[e] / (N N choices)
 *     loss      = sum over e of slopes[e] * sum over t of p[t, e]
 * which is num_experts times the sum of each expert's share of the choices
 * times its mean probability, 1 where both are even.  All are zeros for N = 0.
 * Sums are in 32 bits or more in a fixed order. */
int64_t bmmc_expert_balance_workspace(int64_t tokens, int num_experts);

int bmmc_expert_balance(const void *logits, int64_t logits_stride, int type, int num_experts,
                        const void *experts, int index_type, int64_t tokens, int choices,
                        const uint8_t *mask, float *loss, int32_t *counts, float *slopes,
                        void *workspace, int64_t workspace_bytes, void *stream);

/* grad_logits[t, e] = grad * p[t, e] * (slopes[e] - sum over e' of slopes[e']
 * p[t, e']), zeros where the mask is 0; grad is one float32 on the device. */
int bmmc_expert_balance_backward(const float *grad, const void *logits, int64_t logits_stride,
                                 int type, int num_experts, const float *slopes, int64_t tokens,
                                 const uint8_t *mask, void *grad_logits, int64_t grad_stride,
                                 void *stream);

#ifdef __cplusplus
}
#endif

#endif /* BMMC_LAYER_H */
