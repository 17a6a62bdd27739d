// tokens.h -- what the host side (api.cpp) and the kernels of the token-row
// operators share: the launchers and the host-made arguments of the kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../../include/bmmc_tokens.h"
#include "../launch.h"

namespace bmmc {

// `blocks` workgroups in launches of at most kMaxWorkItemsPerLaunch.
template <class F> int in_launches(int64_t blocks, uint32_t threads, F launch) {
    const int64_t per = (int64_t)max_blocks_per_launch(threads);
    for (int64_t b0 = 0; b0 < blocks; b0 += per)
        launch((uint32_t)(blocks - b0 < per ? blocks - b0 : per), b0);
    return hipGetLastError() == hipSuccess ? BMMC_OK : BMMC_ERR_HIP;
}

// Quotients by a fixed divisor of numbers below 2^31: with s = ceil(log2 d)
// and mul = ceil(2^(31+s) / d), floor(n * mul / 2^(31+s)) is exact, since mul
// exceeds 2^(31+s) / d by less than 1 and n < 2^31 <= 2^(31+s) / d.
struct FastDiv {
    uint32_t d, mul, shift;
};

inline FastDiv fast_div(uint32_t d) {
    uint32_t s = 0;
    while ((uint64_t(1) << s) < d) ++s;
    const uint64_t top = uint64_t(1) << (31 + s);
    return FastDiv{d, (uint32_t)((top + d - 1) / d), 31 + s};
}

__host__ __device__ inline uint32_t quotient(const FastDiv &f, uint32_t n) {
    return (uint32_t)(((uint64_t)n * f.mul) >> f.shift);
}

// Where a token's keys and values go: the page, or -1 for nowhere, and the
// place in it.  Every index is checked here, before an address is made of it.
struct PagePlace {
    int32_t page, place;
};

struct PageTable {
    const int32_t *table;
    const int32_t *sequences;
    const void *positions;
    int64_t batch, width, stride, pages, page_size;
    int32_t positions_are_64;
};

__host__ __device__ inline int64_t position_at(const void *p, int is64, int64_t i) {
    return is64 ? static_cast<const int64_t *>(p)[i] : static_cast<const int32_t *>(p)[i];
}

__host__ __device__ inline PagePlace page_place(const PageTable &t, int64_t token) {
    const int64_t s = t.sequences ? (int64_t)t.sequences[token] : token;
    const int64_t pos = position_at(t.positions, t.positions_are_64, token);
    if (s < 0 || s >= t.batch || pos < 0) return PagePlace{-1, 0};
    int64_t column, place;
    if (pos >> 31) {
        column = pos / t.page_size;
        place = pos - column * t.page_size;
    } else {  // page_size is below 2^31
        column = (uint32_t)pos / (uint32_t)t.page_size;
        place = (uint32_t)pos - (uint32_t)column * (uint32_t)t.page_size;
    }
    if (column >= t.width) return PagePlace{-1, 0};
    const int32_t page = t.table[s * t.stride + column];
    if (page < 0 || page >= t.pages) return PagePlace{-1, 0};
    return PagePlace{page, (int32_t)place};
}

// ---- experts ---------------------------------------------------------------

// How bmmc_expert_order cuts its choices: one workgroup up to
// kOrderOneBlockMax choices, which it holds in registers (3000 choices of 64
// experts take it 6.9 us, 4096 8.0 and two launches 7.8, at twice the host's
// time); else at most kOrderMaxBlocks workgroups of `chunk` choices each, which
// first count into the workspace: of kOrderMinChunk choices, or twice as many
// where that makes more than 64 workgroups, whose counts each would have to sum
// (131072 choices of 256 experts 12.2 and 12.7 us, 327680 15.5 and 18.0; 16384
// choices 10.4 and 9.0).
constexpr int64_t kOrderOneBlockMax = 4096;
constexpr int64_t kOrderMaxBlocks = 256;
constexpr int64_t kOrderMinChunk = 1024;

struct OrderCut {
    int64_t chunk;
    int32_t blocks;
};

inline OrderCut order_cut(int64_t n) {
    if (n <= kOrderOneBlockMax) return OrderCut{n, 1};
    int64_t chunk = (n + kOrderMaxBlocks - 1) / kOrderMaxBlocks;
    const int64_t least = n > 64 * kOrderMinChunk ? 2 * kOrderMinChunk : kOrderMinChunk;
    if (chunk < least) chunk = least;
    chunk = (chunk + 63) / 64 * 64;
    return OrderCut{chunk, (int32_t)((n + chunk - 1) / chunk)};
}

struct OrderArgs {
    const void *experts;
    int32_t is64, num_experts;
    int64_t n, align, capacity, chunk;
    int32_t *offsets, *counts, *rows, *slots, *hist;
};
int launch_expert_order(const OrderArgs &a, int blocks, hipStream_t s);

struct MoveArgs {
    const void *x;      // tokens (gather, backward's grad) or rows (combine)
    const void *in;     // backward: the rows
    const int32_t *rows, *slots;
    const void *weights;
    void *out, *grad_weights;
    int64_t x_stride, in_stride, out_stride, tokens, capacity, dim;
    int32_t choices, weights_are_f32;
    int32_t whole_lines;  // rows of out are whole cache lines
    int32_t stream;       // rows by expert are more than the caches keep
};
int launch_expert_gather(const MoveArgs &a, int type, hipStream_t s);
int launch_expert_combine(const MoveArgs &a, int type, hipStream_t s);
int launch_expert_combine_backward(const MoveArgs &a, int type, hipStream_t s);

// ---- rotary positions and the paged cache ------------------------------------

struct HeadsArgs {
    const bmmc_heads *x;
    int32_t count, head_dim, type;
    int64_t batch, tokens;
};
int launch_rotary(const HeadsArgs &a, const bmmc_rotation &r, hipStream_t s);

struct AppendArgs {
    bmmc_heads q, k, v;  // q.heads = 0 without queries
    bmmc_paged_cache k_cache, v_cache;
    PageTable where;
    bmmc_rotation rotation;  // pairs = 0 without a rotation
    int64_t tokens;
    int32_t k_dim, v_dim, type;
};
int launch_cache_append(const AppendArgs &a, hipStream_t s);

}  // namespace bmmc
