// plan.cpp -- how calls of the layer's operators are cut into workgroups, from
// their sizes alone.
#include <algorithm>

#include "layer.h"

namespace bmmc {

namespace {

// Workgroups that keep the card busy: two or three on each of its 256 compute units.
constexpr int64_t kBusy = 1024;

}  // namespace

AttendPlan attend_plan(const bmmc_attention &a) {
    const int64_t group = a.q_heads / a.heads;
    const int64_t filled = std::min(a.batch, a.tokens);  // sequences with tokens at most
    const bool wide = a.type == BMMC_F32;
    const int dim = std::max(a.k_dim, a.v_dim);
    AttendPlan p{};
    p.rows = 16;
    // four waves, of 16 keys each where long rows of 32 bits leave no registers for 32
    p.unit = wide && dim > 64 ? 64 : 128;
    p.tiles = a.starts ? a.tokens * group / p.rows + filled
                       : a.tokens * ((group + p.rows - 1) / p.rows);
    p.least = 1;
    const int64_t reach = a.table_width * a.page_size;
    if (p.tiles * a.heads < 2 * kBusy && reach > p.unit)
        p.target = (int32_t)std::max<int64_t>(kBusy / a.heads, 1);
    p.parts = p.tiles + p.target;
    return p;
}

// Workgroups that sum the tokens' probabilities: of 16 tokens at least, and no
// more than leave the second launch little to sum.
int32_t balance_blocks(int64_t tokens, int num_experts) {
    const int64_t most = std::max<int64_t>(64, std::min<int64_t>(256, 65536 / num_experts));
    return (int32_t)std::max<int64_t>(1, std::min(most, (tokens + 15) / 16));
}

}  // namespace bmmc
