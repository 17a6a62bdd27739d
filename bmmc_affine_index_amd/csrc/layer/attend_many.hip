// attend_many.hip -- attention over a paged cache, 128 rows a tile (gfx950).
//
// As in attend_few.hip, with products of 32 x 32 in 16-bit types: S = K Q^T and
// O^T = V^T P^T, so that a lane holds scores of one row, which the second product
// takes from where the first leaves them, keys 8 (i / 4) + 4 (l / 32) + i % 4 of each 32.
// Each of four waves has 32 rows; all of them share tiles of 64 keys, which
// go to LDS one tile ahead: straight from memory where rows are whole vectors
// of the products' type, through registers where they have to be shifted or widened.  Keys are read from LDS as whole
// vectors, values by the transposing read, which brings four keys of one column
// into a lane; the order of a row's vectors in LDS depends on the row, so that
// neither meets a bank twice at a time.
//
// Bound by the matrix units and by the powers of two between the products: two
// workgroups a compute unit let one's products run beside the other's powers.
//
// Measured: 8192 new tokens of 4 sequences, 32 query over 8 key heads of 128 in bf16,
// 342 GFLOP: 490 to 500 us, 690 TFLOP/s (a matrix product of 8192 in the library: 1200);
// the vector unit works for 46% of the time, the matrix unit for 29% of its peak.  From
// 8 bits, 4096 tokens of 4 sequences behind up to 2048 places, 16 over 4 heads of 128, 66
// GFLOP: 138 us in bf16 and 140 in f16 with a scale for each head, 154 and, in two
// products, 181 for each row.
#include "attend.h"

namespace bmmc {

namespace {

using namespace dev;

typedef float f16x __attribute__((ext_vector_type(16)));

constexpr int kManyWaves = 4;
constexpr int kManyThreads = 64 * kManyWaves;
constexpr int kManyRows = 32 * kManyWaves;
constexpr int kKeys = 64;  // of a tile

__device__ __forceinline__ f16x mfma32(Product<f16_t>::vec a, Product<f16_t>::vec b, f16x c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f16x mfma32(Product<bf16_t>::vec a, Product<bf16_t>::vec b, f16x c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// The order of a block's N times PRODUCTS products and EACH reads from LDS for each of
// the N: reads for AHEAD of them come first, so that no product waits for its own.
template <int N, int EACH, int AHEAD, int PRODUCTS = 1> __device__ __forceinline__ void reads_ahead() {
    constexpr int kProduct = 0x8, kRead = 0x100;
    __builtin_amdgcn_sched_group_barrier(kRead, EACH * AHEAD, 0);
#pragma unroll
    for (int i = 0; i < N - AHEAD; ++i) {
        __builtin_amdgcn_sched_group_barrier(kProduct, PRODUCTS, 0);
        __builtin_amdgcn_sched_group_barrier(kRead, EACH, 0);
    }
    __builtin_amdgcn_sched_group_barrier(kProduct, PRODUCTS * AHEAD, 0);
}

// DP: the heads' elements, padded.
template <typename T, int DP> struct Many {
    static constexpr int CR = DP / 8;                    // vectors of a row
    static constexpr int NC = kKeys * CR / kManyThreads;  // vectors of a tile a thread moves
    static constexpr int kRowBytes = DP * 2;
    static constexpr int kTileBytes = kKeys * kRowBytes;

    // Where vector c of a row lies in it.  Keys are read 16 rows at a time in one
    // column, values 4 rows of 64 bytes.
    static __device__ __forceinline__ int key_at(int row, int c) {
        return c ^ (CR == 8 ? row >> 1 & 7 : row & 15);
    }
    static __device__ __forceinline__ int value_at(int row, int c) {
        return c ^ (CR == 8 ? (row >> 1 & 1) << 2 : (row & 3) << 2);
    }

    struct Lds {
        uint8_t k[2][kTileBytes], v[2][kTileBytes];
        const uint8_t *row[2][2][kKeys];  // of a tile's keys, its values
        float scale[2][2][kKeys];
        uint64_t seen[2];  // keys that are there
        uint64_t odd[2];   // keys with a value that is no number
    };
};

// Elements that are no numbers in words of two, as zeros; whether there were any.
template <typename T> __device__ __forceinline__ bool drop_nonfinite(uint32_t &w) {
    constexpr uint32_t m = __is_same(T, f16_t) ? 0x7c00u : 0x7f80u;
    const bool lo = (w & m) == m, hi = (w >> 16 & m) == m;
    if (lo) w &= 0xffff0000u;
    if (hi) w &= 0x0000ffffu;
    return lo || hi;
}

// 16 bytes a lane from memory to 1024 adjacent bytes of LDS.
__device__ __forceinline__ void copy_to_lds(const uint8_t *from, uint8_t *to) {
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)from,
                                     (__attribute__((address_space(3))) void *)to, 16, 0, 0);
}
__device__ __forceinline__ void wait_for_copies() {
    __builtin_amdgcn_s_waitcnt(0x0f70);  // every load of this wave, no other wait
}

// ROWS: 8-bit values have a scale for each row.
template <typename T, typename E, int DP, bool DIRECT, bool ROWS>
__global__ void __launch_bounds__(kManyThreads, DP <= 128 ? 2 : 1)
    bmmc_attend_many_kernel(const AttendArgs x, int64_t block0) {
    using M = Many<T, DP>;
    constexpr int CR = M::CR, NC = M::NC, KS = DP / 16, DB = DP / 32;
    constexpr bool kNarrow = sizeof(E) == 1;
    typedef typename Product<T>::vec vec_t;
    typedef typename Weighed<T, ROWS>::type W;
    typedef typename Product<W>::vec weights_t;
    constexpr bool kTwo = Weighed<T, ROWS>::kTwo;
    extern __shared__ __attribute__((aligned(256))) uint8_t lds_bytes[];
    typename M::Lds &lds = *reinterpret_cast<typename M::Lds *>(lds_bytes);

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n = lane & 31, half = lane >> 5;
    const int64_t block = block0 + blockIdx.x, heads = x.a.heads;
    const int64_t blocks = (x.plan.shares ? x.plan.shares : x.plan.tiles) * heads;
    if (block >= blocks) {
        clear_rest<T>(x, block - blocks, kClearBlocks);
        return;
    }
    const int64_t number = block / heads;
    const int head = (int)(block - number * heads);
    Share share{};
    Tile tile;
    int64_t unit, stop;  // of all: this workgroup's
    if (x.plan.shares) {
        share = find_share(x, (int32_t)number);
        unit = share.from;
        stop = share.to;
        tile = share.tile;
    } else {
        // a sequence's last tiles see most: they come first
        tile = uniform(find_tile(x, x.plan.tiles - 1 - number));
        unit = tile.first;
        stop = tile.first + tile.units;
    }
    // A head's scale of the keys goes into c, by which scores are multiplied behind the
    // mask and the maximum, where that leaves c above 0 and finite; other scales (0,
    // below 0, lost in 32 bits) are multiplied to the scores before those.
    float c = x.a.scale * 1.4426950408889634f, by_key = 1.0f, by_value = 1.0f;
    bool key_apart = false;
    if (kNarrow && !ROWS && x.a.pages) {  // without pages there may be no scales
        by_key = x.k.scale[head * x.k.scale_head];
        by_value = x.v.scale[head * x.v.scale_head];
        key_apart = !(c * by_key > 0.0f && c * by_key < __builtin_inff());
        if (!key_apart) c *= by_key;
    }
    // threads 0 to 63 look after the rows of a tile's keys, 64 to 127 of its values
    const int of_values = wave & 1, key_row = lane;  // the same in a wave: their strides are scalars
    const bool looks = wave < 2;
    const uint8_t *base = static_cast<const uint8_t *>(of_values ? x.v.data : x.k.data);
    const int64_t by_page = of_values ? x.v.page_stride : x.k.page_stride;
    const int64_t by_place = of_values ? x.v.place_stride : x.k.place_stride;
    const int64_t by_head = (of_values ? x.v.head_stride : x.k.head_stride) * head;

    while (tile.found && unit < stop) {
        const int32_t unit0 = (int32_t)(unit - tile.first);
        const int32_t unit1 = (int32_t)min(stop - tile.first, (int64_t)tile.units);
        const Span span = span_of(x, tile, unit0, unit1);
        const int32_t *table = x.a.table + (int64_t)tile.seq * x.a.table_stride;

        // this lane's row, and what its wave's rows see
        const int64_t rows = (int64_t)tile.q.count * x.group;
        const int64_t wave_row = (int64_t)tile.tile * kManyRows + wave * 32;
        const int64_t row = wave_row + n;
        const bool on = row < rows, wave_on = wave_row < rows;
        const int32_t token = (int32_t)quotient(x.by_group, (uint32_t)row);
        const int32_t before = tile.q.length - tile.q.count;
        const int32_t place = before + token;
        const int32_t wave_first = before + (int32_t)quotient(x.by_group, (uint32_t)wave_row);
        const int32_t wave_last =
            before + (int32_t)quotient(x.by_group, (uint32_t)min(wave_row + 31, rows - 1));
        const int64_t q_row = (tile.q.first + (int64_t)token);
        const int64_t q_head = (int64_t)head * x.group + (row - (int64_t)token * x.group);
        vec_t q[KS];
        {
            const uint8_t *in = reinterpret_cast<const uint8_t *>(kZeros);
            if (on)
                in = reinterpret_cast<const uint8_t *>(static_cast<const T *>(x.a.q) +
                                                       q_row * x.a.q_token + q_head * x.a.q_head);
            const int dim = kept(x.a.k_dim), from = kept_lane(half * 8);
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                Raw<T, 8> r = fetch<T, 8>(in, k * 16 + from, dim);
                if (dim & 7) settle(r, k * 16 + from, dim);
                q[k] = product_vec<T>(r);
            }
        }

        const auto look = [&](int32_t t) { return entry_of(x, table, t + key_row, span.to); };
        float scale_next = 0.0f;
        const auto put = [&](int32_t entry, int32_t t, int which) {
            if (!looks) return;
            const int32_t page = page_of(x, entry, t + key_row, span.to);
            const int32_t in =
                t + key_row - (int32_t)quotient(x.by_page, (uint32_t)(t + key_row)) * (int32_t)x.by_page.d;
            lds.row[which][of_values][key_row] =
                page < 0 ? reinterpret_cast<const uint8_t *>(kZeros)
                         : base + (page * by_page + in * by_place + by_head) * (int64_t)sizeof(E);
            const uint64_t seen = __ballot(page >= 0);
            if (tid == 0) {
                lds.seen[which] = seen;
                lds.odd[which] = 0;
            }
            if (ROWS) {
                const bmmc_scaled_cache &cache = of_values ? x.v : x.k;
                scale_next = page < 0 ? 0.0f
                                      : cache.scale[page * cache.scale_page + in * cache.scale_place +
                                                    head * cache.scale_head];
            }
        };
        Raw<E, 8> kr[DIRECT ? 1 : NC], vr[DIRECT ? 1 : NC];
        const auto load = [&](int which) {
            const int k_dim = kept(x.a.k_dim), v_dim = kept(x.a.v_dim);
            if constexpr (DIRECT) {
                const int mine = kept_lane(lane);
#pragma unroll
                for (int i = 0; i < NC; ++i) {
                    const int first = (i * kManyWaves + wave) * 64;  // vector of the tile
                    const int r = (first + mine) / CR, at = (first + mine) % CR;
                    const int kc = M::key_at(r, at), vc = M::value_at(r, at);
                    const uint8_t *zeros = reinterpret_cast<const uint8_t *>(kZeros);
                    copy_to_lds(kc * 8 < k_dim ? lds.row[which][0][r] + kc * 16 : zeros,
                                lds.k[which] + first * 16);
                    copy_to_lds(vc * 8 < v_dim ? lds.row[which][1][r] + vc * 16 : zeros,
                                lds.v[which] + first * 16);
                }
            } else {
                const int my_c = kept_lane(tid) % CR, my_row = kept_lane(tid) / CR;
#pragma unroll
                for (int i = 0; i < NC; ++i) {
                    const int r = my_row + i * (kManyThreads / CR);
                    kr[i] = fetch<E, 8>(lds.row[which][0][r], my_c * 8, k_dim);
                    vr[i] = fetch<E, 8>(lds.row[which][1][r], my_c * 8, v_dim);
                }
            }
        };
        // What a tile's rows hold goes to LDS; a value that is no number must not
        // reach rows that do not see its key, and is put aside where there are such.
        const auto parted_at = [&](int32_t t) {
            return t + kKeys - 1 > span.first || (x.a.window && t <= span.last - x.a.window);
        };
        const auto store = [&](int32_t t, int which) {
            const bool parted = parted_at(t);
            if (ROWS && looks) lds.scale[which][of_values][key_row] = scale_next;
            const auto put_aside = [&](int r, uint32_t (&w)[4]) {
                bool odd = false;
#pragma unroll
                for (int j = 0; j < 4; ++j) odd |= drop_nonfinite<W>(w[j]);
                if (odd) atomicOr(reinterpret_cast<unsigned long long *>(&lds.odd[which]), 1ull << r);
                return odd;
            };
            if constexpr (DIRECT) {
                wait_for_copies();
                if (!parted) return;
                // each thread looks at what it has copied itself
                for (int i = 0; i < NC; ++i) {
                    const int at = (i * kManyWaves + wave) * 64 + lane;
                    u4 *place = reinterpret_cast<u4 *>(lds.v[which] + at * 16);
                    const u4 v = *place;
                    uint32_t w[4] = {v[0], v[1], v[2], v[3]};
                    if (put_aside(at / CR, w)) *place = u4{w[0], w[1], w[2], w[3]};
                }
            } else {
                const int k_dim = kept(x.a.k_dim), v_dim = kept(x.a.v_dim);
                const int my_c = kept_lane(tid) % CR, my_row = kept_lane(tid) / CR;
#pragma unroll
                for (int i = 0; i < NC; ++i) {
                    const int r = my_row + i * (kManyThreads / CR);
                    if (k_dim & 7) settle(kr[i], my_c * 8, k_dim);
                    if (v_dim & 7) settle(vr[i], my_c * 8, v_dim);
                    uint32_t kw[4], vw[4];
                    expand<T>(kr[i], kw);
                    expand<W>(vr[i], vw);
                    if (parted) put_aside(r, vw);
                    *reinterpret_cast<u4 *>(lds.k[which] + r * M::kRowBytes + M::key_at(r, my_c) * 16) =
                        u4{kw[0], kw[1], kw[2], kw[3]};
                    *reinterpret_cast<u4 *>(lds.v[which] + r * M::kRowBytes + M::value_at(r, my_c) * 16) =
                        u4{vw[0], vw[1], vw[2], vw[3]};
                }
            }
        };

        f16x o[DB];
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
            for (int i = 0; i < 16; ++i) o[d][i] = 0.0f;
        float m = kNothing, l = 0.0f;
        int32_t t = span.from;
        int which = 0;
        int32_t entry = -1;  // of the tile after the next
        if (t < span.to) {
            put(look(t), t, 0);
            __syncthreads();
            load(0);
            entry = look(t + kKeys);
            store(t, 0);
            put(entry, t + kKeys, 1);
            entry = look(t + 2 * kKeys);
            __syncthreads();
        }
        // the queries are here before the loop, in which nothing waits for them
#pragma unroll
        for (int k = 0; k < KS; ++k) asm volatile("" : "+v"(q[k]));
        for (; t < span.to; t += kKeys, which ^= 1) {
            const bool more = t + kKeys < span.to;
            if (more) load(which ^ 1);
            const bool busy = wave_on && t <= wave_last &&
                              (!x.a.window || t + kKeys - 1 > wave_first - x.a.window);
            if (busy) {
                f16x s[2];
                const uint8_t *keys = lds.k[which] + n * M::kRowBytes;
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int i = 0; i < 16; ++i) s[b][i] = 0.0f;
#pragma unroll
                for (int k = 0; k < KS; ++k)
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        const vec_t a = *reinterpret_cast<const vec_t *>(
                            keys + b * 32 * M::kRowBytes + M::key_at(n, k * 2 + half) * 16);
                        s[b] = mfma32(a, q[k], s[b]);
                    }
                reads_ahead<2 * KS, 1, 6>();
#pragma unroll
                for (int b = 0; b < 2; ++b) asm volatile("s_nop 15" : "+v"(s[b]));
                if (ROWS) {
#pragma unroll
                    for (int b = 0; b < 2; ++b)
#pragma unroll
                        for (int i = 0; i < 16; i += 4) {
                            const f4 by = *reinterpret_cast<const f4 *>(
                                &lds.scale[which][0][b * 32 + 2 * i + 4 * half]);
#pragma unroll
                            for (int j = 0; j < 4; ++j) s[b][i + j] *= by[j];
                        }
                }
                if (kNarrow && !ROWS && key_apart)
#pragma unroll
                    for (int b = 0; b < 2; ++b)
#pragma unroll
                        for (int i = 0; i < 16; ++i) s[b][i] *= by_key;
                const uint64_t there = uniform(lds.seen[which]);
                const bool parted = t + kKeys - 1 > wave_first ||
                                    (x.a.window && t <= wave_last - x.a.window);
                // this lane's scores of keys that its row does not see
                const auto hide = [&](float as) {
                    const uint64_t mine = (seen_of(place - t, x.a.window) & there) >> 4 * half;
#pragma unroll
                    for (int b = 0; b < 2; ++b)
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            if (!((uint32_t)(mine >> b * 32) & 1u << (8 * (i / 4) + i % 4))) s[b][i] = as;
                };
                if (parted || ~there) hide(kNothing);
                float top = kNothing;
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int i = 0; i < 16; ++i) top = fmaxf(top, s[b][i]);
                top = over_32(top, Largest()) * c;
                // weights may grow to 2^8 before the sums are brought down to a new
                // maximum, which both types hold
                if (__any(top > m + 8.0f)) {
                    const float m_new = fmaxf(m, top);
                    const float down = exp2_of(m - settled(m_new));
                    l *= down;
#pragma unroll
                    for (int d = 0; d < DB; ++d) o[d] *= down;
                    m = m_new;
                }
                const float minus = kLift<W> - settled(m);
                float sum[4] = {};
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        s[b][i] = exp2_of(fmaf(s[b][i], c, minus));
                        sum[i & 3] += s[b][i];
                    }
                l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                if (ROWS) {
#pragma unroll
                    for (int b = 0; b < 2; ++b)
#pragma unroll
                        for (int i = 0; i < 16; i += 4) {
                            const f4 by = *reinterpret_cast<const f4 *>(
                                &lds.scale[which][1][b * 32 + 2 * i + 4 * half]);
#pragma unroll
                            for (int j = 0; j < 4; ++j) s[b][i + j] *= by[j];
                        }
                    // a weight of 0 times a scale that is no number is no number
                    if (parted) hide(0.0f);
                }
                // this lane reads 4 elements of value row 4 half + (l % 16) / 4 of 8
                const int v_row = 4 * half + (lane >> 2 & 3);
                const uint8_t *values = lds.v[which] + v_row * M::kRowBytes + (lane & 1) * 8;
                weights_t p[4], rest[kTwo ? 4 : 1];  // of 16 keys each
#pragma unroll
                for (int k = 0; k < 4; ++k)
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float w = s[k / 2][k % 2 * 8 + j];
                        p[k][j] = (W)w;
                        if constexpr (kTwo) rest[k][j] = (W)(w - (float)p[k][j]);
                    }
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int k = 0; k < 4; ++k)
#pragma unroll
                    for (int d = 0; d < DB; ++d) {
                        const int vec = d * 4 + (lane >> 4 & 1) * 2 + (lane >> 1 & 1);
                        typedef short s4 __attribute__((ext_vector_type(4)));
                        typedef __attribute__((address_space(3))) s4 *lds_s4;
                        const uint8_t *at =
                            values + k * 16 * M::kRowBytes + M::value_at(v_row, vec) * 16;
                        s4 v4[2];
                        v4[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4)at);
                        v4[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4)(at + 8 * M::kRowBytes));
                        weights_t a;
                        __builtin_memcpy(&a, v4, 16);
                        o[d] = mfma32(a, p[k], o[d]);
                        if constexpr (kTwo) o[d] = mfma32(a, rest[k], o[d]);
                    }
                reads_ahead<4 * DB, 2, 4, kTwo ? 2 : 1>();
                // values put aside for any wave, to the rows that see them
                uint64_t odd = parted_at(t) ? uniform(lds.odd[which]) : 0;
                while (odd) {
                    const int key = __ffsll((unsigned long long)odd) - 1;
                    odd &= odd - 1;
                    float w = 0.0f;
#pragma unroll
                    for (int b = 0; b < 2; ++b)
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            if (b * 32 + 8 * (i / 4) + i % 4 == (key & ~4)) w = s[b][i];
                    w = __shfl(w, (key & 4) * 8 + n, 64);
                    if (!(seen_of(place - t, x.a.window) >> key & 1)) continue;
                    const E *in = reinterpret_cast<const E *>(lds.row[which][1][key]);
                    const int dim = kept(x.a.v_dim), from = kept_lane(4 * half);
#pragma unroll
                    for (int d = 0; d < DB; ++d)
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            __builtin_amdgcn_sched_barrier(0);  // one at a time
                            const int at = d * 32 + 8 * (i / 4) + from + i % 4;
                            if (at >= dim) continue;
                            const float v = element_of<T, E>(in + at);
                            if (!(fabsf(v) < __builtin_inff())) o[d][i] += w * v;
                        }
                }
            }
            if (more) {
                store(t + kKeys, which ^ 1);
                if (t + 2 * kKeys < span.to) {
                    // the slot's readers are this tile's loads, odd values and masks
                    __syncthreads();
                    put(entry, t + 2 * kKeys, which);
                    entry = look(t + 3 * kKeys);
                }
            }
            __syncthreads();
        }

        l += __shfl_xor(l, 32, 64);
        if (on) {
            const bool whole = unit0 == 0 && unit1 == tile.units;
            const float inv = l == 0.0f ? 0.0f : by_value / l;
            const int64_t slot =
                ((number * 2 + (unit0 == 0)) * heads + head) * kManyRows + wave * 32 + n;
            if (!whole && half == 0) x.state[slot] = make_float2(m, l);
            T *out = static_cast<T *>(x.a.out) + q_row * x.a.out_token + q_head * x.a.out_head;
            float *part = x.partial + slot * x.pitch;
            const int dim = kept(x.a.v_dim), from = kept_lane(4 * half);
#pragma unroll
            for (int d = 0; d < DB; ++d)
#pragma unroll
                for (int i = 0; i < 16; i += 4) {
                    const int at = d * 32 + 2 * i + from;
                    f4 y{o[d][i], o[d][i + 1], o[d][i + 2], o[d][i + 3]};
                    if (whole) {
                        y = l == 0.0f ? f4{0.0f, 0.0f, 0.0f, 0.0f} : y * inv;
                        if (at + 4 <= dim) {
                            Floats<4> z = y;
                            dev::store<T, 4, false>(out + at, narrow<T, 4>(z));
                        } else {
                            for (int j = 0; j < 4; ++j)
                                if (at + j < dim) out[at + j] = (T)y[j];
                        }
                    } else {
                        if (at < dim) *reinterpret_cast<f4 *>(part + at) = y * by_value;
                    }
                }
        }
        unit = tile.first + unit1;
        if (unit < stop) next_tile(x, tile);
    }
    if (x.plan.shares && head == 0) leave_begun(x, (int32_t)number, share, tile);
}

template <typename T, typename E, int DP, bool DIRECT> int many(const AttendArgs &x, hipStream_t s) {
    const int64_t blocks = (x.plan.shares ? x.plan.shares : x.plan.tiles) * x.a.heads +
                           (x.a.clear_rest && x.a.starts ? kClearBlocks : 0);
    const bool rows = sizeof(E) == 1 && x.rows_scaled;
    const auto kernel = rows ? bmmc_attend_many_kernel<T, E, DP, DIRECT, sizeof(E) == 1>
                             : bmmc_attend_many_kernel<T, E, DP, DIRECT, false>;
    return in_launches(blocks, kManyThreads, [&](uint32_t nb, int64_t b0) {
        hipLaunchKernelGGL(kernel, dim3(nb), dim3(kManyThreads), sizeof(typename Many<T, DP>::Lds), s, x,
                           b0);
    });
}

template <typename T, typename E, bool DIRECT> int many_by_size(const AttendArgs &x, hipStream_t s) {
    const int dim = x.a.k_dim > x.a.v_dim ? x.a.k_dim : x.a.v_dim;
    if (dim <= 64) return many<T, E, 64, DIRECT>(x, s);
    if (dim <= 128) return many<T, E, 128, DIRECT>(x, s);
    return many<T, E, 256, DIRECT>(x, s);
}

// Whether every row of a cache is whole vectors of 16 bytes at whole addresses.
bool whole_vectors(const bmmc_scaled_cache &c, int dim) {
    const int64_t all = c.page_stride | c.place_stride | c.head_stride | dim;
    return (all & 7) == 0 && (reinterpret_cast<uintptr_t>(c.data) & 15) == 0;
}

template <typename T> int many_by_cache(const AttendArgs &x, hipStream_t s) {
    if (x.k.type == BMMC_E4M3) return many_by_size<T, uint8_t, false>(x, s);
    if (whole_vectors(x.k, x.a.k_dim) && whole_vectors(x.v, x.a.v_dim))
        return many_by_size<T, T, true>(x, s);
    return many_by_size<T, T, false>(x, s);
}

}  // namespace

int launch_attend_many(const AttendArgs &x, hipStream_t s) {
    return x.a.type == BMMC_F16 ? many_by_cache<f16_t>(x, s) : many_by_cache<bf16_t>(x, s);
}

}  // namespace bmmc
