/*
 * bmmc_tokens.h -- rows of tokens moved to where the data says (gfx950).
 *
 * A plan of bmmc.h knows its map when it is made.  The moves of a language
 * model's layer do not: which expert a token goes to, which page of a cache a
 * key goes to and by which angle a head is turned are data on the device.
 * These entry points make three such moves, each in one pass over its rows
 * with the arithmetic that goes with it:
 *
 *   - tokens sorted by expert, the rows gathered in that order and combined
 *     back with the router's weights, and the gradients of both;
 *   - rotary positions on one or several axes, and their gradient;
 *   - keys and values appended to a paged cache, rotated on the way.
 *
 * As in bmmc.h, every function is extern "C", takes device pointers of the
 * current device, sizes and a hipStream_t as void* (NULL = the default
 * stream), runs asynchronously, allocates nothing, never aborts and returns a
 * BMMC_* status.  Every argument check comes before the first HIP call.  All
 * calls may be captured into a graph.  Strides count elements.  Data pointers
 * are aligned to their element; rows need no other alignment.
 *
 * Index arrays are data: the kernels check every entry they use against the
 * sizes given here and skip what lies outside, so a wrong entry never reads or
 * writes out of bounds.
 *
 * What a call writes overlaps nothing else that it reads or writes, unless a
 * function below allows it; rows, heads and caches that overlap are refused
 * (BMMC_ERR_ALIAS).
 */
#ifndef BMMC_TOKENS_H
#define BMMC_TOKENS_H

#include <stddef.h>
#include <stdint.h>

#include "bmmc.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- element types ------------------------------------------------------ */
#define BMMC_F32 0
#define BMMC_F16 1
#define BMMC_BF16 2
#define BMMC_E4M3 3 /* 8 bits, 4 of exponent, no infinities (caches only) */

/* ---- index types -------------------------------------------------------- */
#define BMMC_I32 0
#define BMMC_I64 1

#define BMMC_MAX_EXPERTS 2048
#define BMMC_MAX_CHOICES 1024
#define BMMC_MAX_HEAD_DIM 512
#define BMMC_MAX_AXES 8

/* ---- tokens by expert --------------------------------------------------- */

/* Rows of the sorted order of n choices among num_experts experts when every
 * expert's rows are padded to a multiple of align: n, and align - 1 for each
 * expert that can hold a choice.  -1 if an argument is out of range
 * (0 <= n < 2^31, 1 <= num_experts <= BMMC_MAX_EXPERTS, align >= 1, the result
 * below 2^31). */
int64_t bmmc_expert_rows(int64_t n, int num_experts, int64_t align);

/* Bytes of device workspace that bmmc_expert_order needs (0 for few choices;
 * -1 if an argument is out of range).  Its contents need no initial value and
 * nothing is kept in it from one call to the next. */
int64_t bmmc_expert_order_workspace(int64_t n, int num_experts);

/* Sort n choices by expert, stable.  experts[i] is the expert of choice i;
 * any value outside [0, num_experts) drops the choice.  With capacity =
 * bmmc_expert_rows(n, num_experts, align):
 *   counts[e]      (num_experts)      choices of expert e
 *   offsets[e]     (num_experts + 1)  first row of expert e, a multiple of
 *                                     align; the last is the end of all rows
 *   rows[i]        (n)                row of choice i, -1 if dropped; an
 *                                     expert's choices keep their order
 *   slots[r]       (capacity)         choice at row r, -1 for padding
 * The result does not depend on timing. */
int bmmc_expert_order(const void *experts, int index_type, int64_t n, int num_experts,
                      int64_t align, int32_t *offsets, int32_t *counts, int32_t *rows,
                      int32_t *slots, void *workspace, int64_t workspace_bytes, void *stream);

/* out[r] = x[slots[r] / choices], zeros where slots[r] < 0: x is tokens rows
 * of dim elements, out capacity rows.  rows (tokens * choices) and slots
 * (capacity) are bmmc_expert_order's for the tokens' choices in order; a row
 * whose choice rows no longer sends there is left as it is.  out must not
 * overlap x.  The gradient of x is bmmc_expert_combine of the gradient of out
 * without weights. */
int bmmc_expert_gather(const void *x, int64_t x_stride, const int32_t *rows,
                       const int32_t *slots, int64_t tokens, int choices, int64_t capacity,
                       int64_t dim, int type, void *out, int64_t out_stride, void *stream);

/* out[t] = sum over k of weights[t, k] * in[rows[t, k]] over the choices that
 * are not dropped, in order of k, held in 32 bits and rounded once; zeros for
 * a token without any.  in is capacity rows, out tokens rows that do not
 * overlap it.  weights is tokens * choices values of weight_type (BMMC_F32 or
 * `type`), or NULL for ones. */
int bmmc_expert_combine(const void *in, int64_t in_stride, const int32_t *rows,
                        const void *weights, int weight_type, int64_t tokens, int choices,
                        int64_t capacity, int64_t dim, int type, void *out, int64_t out_stride,
                        void *stream);

/* Gradients of bmmc_expert_combine with weights:
 *   grad_in[r]         = weights[slots[r]] * grad[slots[r] / choices], zeros
 *                        where slots[r] < 0                (capacity rows)
 *   grad_weights[t, k] = sum over d of grad[t, d] * in[rows[t, k], d], 0 for a
 *                        dropped choice         (tokens * choices, weight_type)
 * in one pass; the sums are held in 32 bits and their order is fixed.  grad_in
 * must not overlap grad or in; as in the gather, a row whose choice rows no
 * longer sends there is left as it is. */
int bmmc_expert_combine_backward(const void *grad, int64_t grad_stride, const void *in,
                                 int64_t in_stride, const int32_t *rows, const int32_t *slots,
                                 const void *weights, int weight_type, int64_t tokens,
                                 int choices, int64_t capacity, int64_t dim, int type,
                                 void *grad_in, int64_t grad_in_stride, void *grad_weights,
                                 void *stream);

/* ---- rotary positions --------------------------------------------------- */

/* Heads of the tokens of a batch: element d of head h of token t of batch
 * entry b is in[b * in_batch + t * in_token + h * in_head + d]. */
typedef struct bmmc_heads {
    const void *in;
    void *out;
    int64_t heads;
    int64_t in_batch, in_token, in_head;
    int64_t out_batch, out_token, out_head;
} bmmc_heads;

/* Pair i of a head (elements i and pairs + i, or 2i and 2i + 1 when
 * interleaved) of token t is turned by the angle
 *     positions[axis(i) * axis_stride + t] * freqs[i]
 * with axis(i) = axis_of_pair[i], or 0 where that is NULL; an axis outside
 * [0, axes) turns by nothing.  The angle is held in 64 bits until it is
 * reduced to a part of a turn.  inverse turns the other way.  Turned pairs
 * are multiplied by scale; elements past the 2 * pairs first are copied.
 * 0 < 2 * pairs <= the head's elements. */
typedef struct bmmc_rotation {
    const void *positions; /* axes arrays of batch * tokens whole numbers */
    const void *freqs;     /* pairs values */
    const int32_t *axis_of_pair;
    int64_t axis_stride;
    int position_type; /* BMMC_I32 or BMMC_I64 */
    int freqs_are_64;  /* 1: double, 0: float */
    int axes;
    int pairs;
    int interleaved;
    int inverse;
    float scale;
} bmmc_rotation;

/* Turn the heads of `count` (1 or 2) tensors of batch * tokens tokens, heads
 * of head_dim elements of `type`.  Each out is its in (same address and
 * strides, turned in place) or does not overlap it.  Of two tensors, one turned
 * in place may lie between the elements of the other (views of one
 * projection) but share none with what the other reads or writes; an out of
 * its own lies clear of the other tensor.  BMMC_ERR_ALIAS otherwise.  The
 * gradient is the same call with inverse. */
int bmmc_rotary(const bmmc_heads *x, int count, int64_t batch, int64_t tokens, int head_dim,
                int type, const bmmc_rotation *rotation, void *stream);

/* ---- paged cache -------------------------------------------------------- */

/* A cache of pages of page_size places: element d of head h at place i of
 * page p is data[p * page_stride + i * place_stride + h * head_stride + d].
 * With type BMMC_E4M3 what is stored is value / scale[h * scale_stride],
 * clamped to the type's largest value (NaN stays NaN); scale is NULL
 * otherwise. */
typedef struct bmmc_paged_cache {
    void *data;
    const float *scale;
    int64_t page_stride, place_stride, head_stride;
    int scale_stride; /* 1, or 0 for one scale for all heads */
    int type;         /* the inputs' type or BMMC_E4M3 */
} bmmc_paged_cache;

/* Append the keys and values of `tokens` tokens.  Token t belongs to sequence
 * s = sequences[t] (t itself where sequences is NULL) and its place there is
 * positions[t]: it goes to page table[s * table_stride + positions[t] /
 * page_size], place positions[t] % page_size, of both caches.  Nothing is
 * stored for a token whose s is not in [0, batch), whose position is negative
 * or past table_width pages, or whose page is not in [0, pages); two tokens
 * with one place leave either's values there.
 *
 * k (k_dim elements a head) is rotated by `rotation` on the way, v (v_dim) is
 * not; q, where given, is rotated into its out in the same pass, for every
 * token.  rotation may be NULL: nothing is turned, and q must be NULL too.
 * rotation->positions may be NULL: the one axis is `positions` then.  k->out
 * and v->out and the batch strides are not used.  Heads of k and v are equal
 * in number.  q may be turned in place, between the elements of k and v (views
 * of one projection) but sharing none; an out of its own lies clear of both.
 * Nothing that is read or turned lies in a cache, and no element is in both
 * caches, which may lie in one array.  BMMC_ERR_ALIAS otherwise. */
int bmmc_cache_append(const bmmc_heads *q, const bmmc_heads *k, const bmmc_heads *v,
                      const bmmc_paged_cache *k_cache, const bmmc_paged_cache *v_cache,
                      int64_t pages, int64_t page_size, const int32_t *table, int64_t batch,
                      int64_t table_width, int64_t table_stride, const int32_t *sequences,
                      const void *positions, int position_type, const bmmc_rotation *rotation,
                      int64_t tokens, int k_dim, int v_dim, int type, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* BMMC_TOKENS_H */
