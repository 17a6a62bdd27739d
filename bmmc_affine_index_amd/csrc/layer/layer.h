// layer.h -- what the host side (api.cpp) and the kernels of the layer's
// operators share: the launchers, the kernels' arguments and the plan of the
// attention, which the host side makes from the sizes.
#pragma once

#include "../../../include/bmmc_layer.h"
#include "../tokens/tokens.h"

namespace bmmc {

// ---- attention -------------------------------------------------------------

// A sequence's new tokens, times the heads that share a key head, are the rows
// of its products: row r is token r / group, head r % group.  A tile is `rows`
// rows over the keys that any of them sees; a unit is as many keys as a
// workgroup takes at once.
//
// Few tiles leave few workgroups; then the units of all tiles, one after the other,
// are cut into as many equal shares as run at the same time: a workgroup takes
// one of them, be it a part of a tile or several tiles.  Where it ends inside a
// tile, what it has of the tile goes to the workspace, and a second launch joins
// the parts.  The lengths are on the device, and so are the shares: a long
// sequence among short ones is spread over many.  Without shares a tile is one
// workgroup's, however long its sequence is.
struct AttendPlan {
    int32_t rows, unit;   // of a tile; keys of a step
    int32_t shares;       // of a key head; 0: each tile is one workgroup's
    int64_t tiles;        // at most
};

struct AttendArgs {
    bmmc_attention a;
    bmmc_scaled_cache k, v;
    AttendPlan plan;
    FastDiv by_group, by_page, by_shares;
    int32_t group;
    int32_t rows_scaled;  // scales by place, not by head alone
    int32_t few_units;    // their number is below 2^31
    int64_t reach;        // places the table has
    int32_t pitch;        // v_dim in whole vectors of 4
    // Of each share: a tile's end that it begins with, and one's begin that it ends
    // with; [shares, 2, heads, rows, pitch] and [shares, 2, heads, rows]
    float *partial;
    float2 *state;  // maximum and sum
    int4 *begun;    // shares: the tile that each begins and does not end
};

constexpr int kBalanceColumns = 16;  // experts of a workgroup that joins their sums
constexpr int kClearBlocks = 32;  // workgroups that clear rows of no sequence

// How a call is cut; sizes alone tell.
AttendPlan attend_plan(const bmmc_attention &a);
int launch_attend_few(const AttendArgs &a, hipStream_t s);
int launch_attend_many(const AttendArgs &a, hipStream_t s);
int launch_attend_join(const AttendArgs &a, hipStream_t s);

// ---- the cache --------------------------------------------------------------

struct QuantizeArgs {
    bmmc_heads q, k, v;  // q.heads = 0 without queries
    bmmc_scaled_cache k_cache, v_cache;
    PageTable where;
    bmmc_rotation rotation;  // pairs = 0 without a rotation
    int64_t tokens;
    int32_t k_dim, v_dim, type;
};
int launch_cache_quantize(const QuantizeArgs &a, hipStream_t s);

struct ReadArgs {
    bmmc_heads k, v;
    bmmc_scaled_cache k_cache, v_cache;
    PageTable where;
    int64_t tokens;
    int32_t k_dim, v_dim, type;
};
int launch_cache_read(const ReadArgs &a, hipStream_t s);

// ---- balance -----------------------------------------------------------------

struct BalanceArgs {
    const void *logits;
    void *grad_logits;
    int64_t stride, grad_stride, tokens, chunk;
    const void *experts;
    const uint8_t *mask;
    const float *grad;
    float *loss, *slopes;
    int32_t *counts;
    float *sums;      // blocks, num_experts
    int32_t *hits;    // blocks, num_experts + 1: the last is the tokens
    FastDiv by_choices;
    int32_t num_experts, choices, is64, blocks, type;
};
int32_t balance_blocks(int64_t tokens, int num_experts);
int launch_expert_balance(const BalanceArgs &a, hipStream_t s);
int launch_expert_balance_backward(const BalanceArgs &a, hipStream_t s);

}  // namespace bmmc
