// plan.cpp -- how calls of the layer's operators are cut into workgroups, from
// their sizes alone.
#include <algorithm>

#include "layer.h"

namespace bmmc {

namespace {

constexpr int64_t kUnits = 256;  // compute units

}  // namespace

// Times below in us, 32 query over 8 key heads of 128 in bf16 where not said otherwise;
// rows are those of a sequence and key head, "a x b" are a sequences of b places.
AttendPlan attend_plan(const bmmc_attention &a) {
    const int64_t group = a.q_heads / a.heads;
    const int64_t filled = std::max<int64_t>(std::min(a.batch, a.tokens), 1);  // at most
    const bool wide = a.type == BMMC_F32;
    const int dim = std::max(a.k_dim, a.v_dim);
    const int64_t all = a.table_width * a.page_size;
    const int64_t reach = a.window ? std::min(all, std::min(a.window, all) + a.tokens / filled) : all;
    // Tiles of 16 rows read the keys anew for each 16, tiles of 128 keep fewer workgroups
    // busy.  How many elements the table can hold tells, whatever their bytes: in 16 bits
    // they are read from the last cache or from beyond it, from 8 bits they are widened
    // anew.  Tiles of 16 and of 128:
    //   over 64 x 2048 places, 268 M elements (12 rows 107 and 109), 20 rows 135 and 108, 128
    //   rows 375 and 129; from 8 bits with row scales (12 rows 62 and 104), 20 rows 96 and 99,
    //   40 rows 138 and 111, in float16, which takes two products, 98 and 114, 141 and 133
    //   over 32 x 1024, 67 M, 32 rows 32 and 45, 48 rows 40 and 46, 96 rows 69 and 47; from 8
    //   bits 32 and 49, 44 and 51, 78 and 52
    //   over 16 x 512, 17 M, 64 rows 21 and 26, 128 rows 32 and 27, 192 rows 44 and 28; from 8
    //   bits 22 and 29, 35 and 30, 48 and 30
    const double held = (double)filled * (double)reach * a.heads * (a.k_dim + a.v_dim);
    const int64_t few = held > 96e6 ? 16 : held > 32e6 ? 40 : 128;
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
    // Tiles of 128 need them where they are few and long (512 tokens over 32768 places 412
    // in shares, 1196 in tiles; 1024 over 8192 224 and 304) and not otherwise (1536 over
    // 8192 312 and 323, 1024 over themselves 69 and 46, 4096 341 and 204).  Tiles of 16 take
    // less in tiles where there are many of a sequence (2048 tokens over themselves, 8 heads
    // in 32 bits, 166 and 139; 40 rows over 32 x 1024, still in shares, 74 and 40).  But each
    // tile looks for its sequence among all of them (one token each, lengths from 1 on: 64 x
    // 2048 56 and 59, 512 x 1024 241 and 236, 1024 x 512 267 and 380, 4096 x 128 509 and 2894).
    // Both rules go by sequences of one length; a long one among many short ones may be left
    // to one workgroup.
    const bool shared = many ? (double)units * (double)(5 * busy - 6 * work) > 100.0 * busy
                             : work < 2 * busy && all > p.unit;
    if (shared || filled > 512) p.shares = (int32_t)std::max<int64_t>(busy / a.heads, 1);
    return p;
}

// Workgroups that sum the tokens' probabilities: one, without a second launch, for a
// few rounds of rows (32 tokens of 1024 experts 7.5 us, 11.1 with two launches; 128 of
// 256 9.3 and 10.5; 512 of 64 9.3 and 9.7; 1024 of 32 9.7 and 9.9), otherwise of 16 tokens at least, and no more
// than leave the second launch little to sum.
int32_t balance_blocks(int64_t tokens, int num_experts) {
    if (tokens <= 1024 && tokens * num_experts <= 32768) return 1;
    const int64_t most = std::max<int64_t>(64, std::min<int64_t>(256, 65536 / num_experts));
    return (int32_t)std::max<int64_t>(1, std::min(most, (tokens + 15) / 16));
}

}  // namespace bmmc
