// plan.cpp -- how calls of the layer's operators are cut into workgroups, from
// their sizes alone.
#include <algorithm>

#include "layer.h"

namespace bmmc {

namespace {

constexpr int64_t kUnits = 256;  // compute units

}  // namespace

AttendPlan attend_plan(const bmmc_attention &a) {
    const int64_t group = a.q_heads / a.heads;
    const int64_t filled = std::min(a.batch, a.tokens);  // sequences with tokens at most
    const bool wide = a.type == BMMC_F32;
    const int dim = std::max(a.k_dim, a.v_dim);
    AttendPlan p{};
    // tiles of 128 rows where a sequence has more than 48 (64 rows over 32768 keys: 50 us,
    // 66 by tiles of 16; up to 48 rows as many tiles of 16 read no more than one of 128)
    const bool many = !wide && dim <= 256 && a.tokens * group > 48 * filled;
    p.rows = many ? 128 : 16;
    // four waves, of 16 keys each where long rows of 32 bits leave no registers for 32
    p.unit = many || (wide && dim > 96) ? 64 : 128;
    p.tiles = a.starts ? a.tokens * group / p.rows + filled
                       : a.tokens * ((group + p.rows - 1) / p.rows);
    // workgroups of a compute unit, by the registers that a head's elements take
    const int64_t busy = kUnits * (dim <= 64 ? 3 : dim <= 128 ? 2 : 1);
    const int64_t reach = a.table_width * a.page_size;
    if (p.tiles * a.heads < 4 * busy && reach > p.unit)
        p.shares = (int32_t)std::max<int64_t>(busy / a.heads, 1);
    return p;
}

// Workgroups that sum the tokens' probabilities: one, without a second launch, for a
// few rounds of rows (32 tokens of 1024 experts 7.4 us, 11.0 with two launches; 128 of
// 256 9.4 and 10.5; 512 of 64 9.8 and 8.7), otherwise of 16 tokens at least, and no more
// than leave the second launch little to sum.
int32_t balance_blocks(int64_t tokens, int num_experts) {
    if (tokens <= 1024 && tokens * num_experts <= 32768) return 1;
    const int64_t most = std::max<int64_t>(64, std::min<int64_t>(256, 65536 / num_experts));
    return (int32_t)std::max<int64_t>(1, std::min(most, (tokens + 15) / 16));
}

}  // namespace bmmc
