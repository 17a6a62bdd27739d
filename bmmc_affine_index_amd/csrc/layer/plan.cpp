// plan.cpp -- how calls of the layer's operators are cut into workgroups, from
// their sizes alone.
#include <algorithm>

#include "layer.h"

namespace bmmc {

namespace {

constexpr int64_t kUnits = 256;  // compute units

}  // namespace

// Times below in us, 32 query over 8 key heads of 128 in bf16 where not said otherwise.
AttendPlan attend_plan(const bmmc_attention &a) {
    const int64_t group = a.q_heads / a.heads;
    const int64_t filled = std::max<int64_t>(std::min(a.batch, a.tokens), 1);  // at most
    const bool wide = a.type == BMMC_F32;
    const int dim = std::max(a.k_dim, a.v_dim);
    const int64_t all = a.table_width * a.page_size;
    const int64_t reach = a.window ? std::min(all, std::min(a.window, all) + a.tokens / filled) : all;
    // Tiles of 16 rows read the keys anew for each 16, tiles of 128 keep fewer workgroups
    // busy.  Keys beyond the last cache are read but once: 20 rows over 64 x 2048 places,
    // 537 MB, 109 by tiles of 128, 202 by 16.  Over 134 MB 48 rows take 50 and 75, 32 take
    // 45 and 38; over 33 MB 128 rows 48 and 35, 192 39 and 46.
    const double held = (double)filled * (double)reach * a.heads * (a.k_dim + a.v_dim) * 2;
    const int64_t few = held > 192e6 ? 16 : held > 64e6 ? 40 : 128;
    const bool many = !wide && dim <= 256 && a.tokens * group > few * filled;
    AttendPlan p{};
    p.rows = many ? 128 : 16;
    // four waves, of 16 keys each where long rows of 32 bits leave no registers for 32
    p.unit = many || (wide && dim > 96) ? 64 : 128;
    p.tiles = a.starts ? a.tokens * group / p.rows + filled
                       : a.tokens * ((group + p.rows - 1) / p.rows);
    // workgroups that run at once, by the registers that a head's elements take
    const int64_t busy = kUnits * (dim <= 64 ? 3 : dim <= 128 ? 2 : 1);
    const int64_t work = p.tiles * a.heads, units = reach / p.unit;
    // Equal shares keep all of them busy, for a second launch and parts in memory.
    // Tiles of 128 need them where they are few and long (512 tokens over 32768 places 404
    // in shares, 1182 in tiles; 1024 over 8192 236 and 301) and not otherwise (1536 over
    // 8192 347 and 325, 1024 over themselves 72 and 46, 4096 350 and 217).  Tiles of 16 take
    // less in tiles where there are many of a sequence (2048 tokens over themselves, 8 heads
    // in 32 bits, 170 and 139).  But each tile looks for its sequence among all of them
    // (one token each: 256 x 2048 228 and 224, 1024 x 512 264 and 373, 4096 x 128 510 and 2876).
    const bool shared = many ? (double)units * (double)(5 * busy - 6 * work) > 100.0 * busy
                             : work < 2 * busy && all > p.unit;
    if (shared || filled > 512) p.shares = (int32_t)std::max<int64_t>(busy / a.heads, 1);
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
