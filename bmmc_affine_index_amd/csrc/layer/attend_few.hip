// attend_few.hip -- attention over a paged cache, 16 rows a tile (gfx950).
//
// Rows are a key head's queries: of one token the heads that share it, of a
// chunk those of several tokens.  With K keys by rows and Q queries by rows,
//     S = K Q^T,   O^T = V^T P^T,   P = 2^(S - m)
// so that a lane holds scores of one row only (its column of S): the running
// maximum m and the sum stay in one register each, and what the first product
// leaves in a lane is what the second takes from it, keys 4 (l / 16) + i of each
// 16, without a move between lanes.  The second product's other side wants 8
// keys of one column of V in a lane, where memory has them apart: a lane loads
// a vector of 8 columns of each of its 8 keys, and pairs of keys are put
// together by byte permutes; columns are dealt to the products' rows so that
// its vectors are whole ones.  Nothing goes through LDS but the keys' addresses.
//
// Bound by memory where rows are few: each key and value is read once for all
// rows of a tile.  Four waves of a workgroup take tiles of 32 keys in turn, each
// with a maximum of its own, and are joined through LDS at the end; a tile's
// keys are on their way while the one before is in the products.
//
// Measured (32 query over 8 key heads of 128 in bf16): 64 sequences of up to 8192
// places, 1.09 GB, 209 us and 5 for the join, 5.2 TB/s; reads of this form, 64 bytes
// of 16 rows at once, reach 5.2 to 5.7, whole rows 6.0 to 6.2.  16 sequences of up to
// 1024, 36 MB, 15 us and 4: a chain of waits.  From 8 bits (24 over 4 heads of 96, 128
// sequences of up to 4096, 213 MB) 62 us: widening takes half of the vector unit.
#include <algorithm>

#include "attend.h"

namespace bmmc {

namespace {

using namespace dev;

constexpr int kFewWaves = 4;

// Bits that are all ones in no finite value.
template <typename E> __device__ __forceinline__ bool has_nonfinite(uint32_t w) {
    if constexpr (sizeof(E) == 4) {
        return (w & 0x7f800000u) == 0x7f800000u;
    } else if constexpr (sizeof(E) == 2) {
        constexpr uint32_t m = __is_same(E, f16_t) ? 0x7c00u : 0x7f80u;
        return (w & m) == m || (w >> 16 & m) == m;
    } else {
        bool any = false;
#pragma unroll
        for (int i = 0; i < 4; ++i) any |= (w >> 8 * i & 0x7fu) == 0x7fu;
        return any;
    }
}

// DP: the heads' elements, padded; KB: blocks of 16 keys a wave's tile.  AHEAD: a
// tile's keys are fetched while the one before is worked on, and its values
// while its keys are; longer heads leave no registers for that.
template <typename T, typename E, int DP, int KB, bool AHEAD> struct Few {
    static constexpr int CE = Product<T>::N;      // elements of a vector along a head
    static constexpr int NK = DP / (4 * CE);      // of them a lane has of a key
    // values of a key in a vector, of whole words, and such vectors in a lane
    static constexpr int VE = sizeof(T) == 2 ? (DP == 64 ? 4 : CE) : DP == 96 && sizeof(E) == 4 ? 2 : CE;
    static_assert(VE * sizeof(E) % 4 == 0);
    static constexpr int VG = (DP + 16 * VE - 1) / (16 * VE);
    static constexpr int KT = 16 * KB;            // keys of a tile
    static constexpr int VK = 4 * KB;             // keys in a lane
    static constexpr int KG = AHEAD ? NK : 8;     // vectors of a key fetched at a time
    static constexpr bool kQueriesInLds = DP == 512;
    // + 4: the 16 rows of a joined tile start in different banks
    static constexpr int kPitch = VG * 16 * VE + 4;

    struct PerWave {
        const uint8_t *at[2][2][KT];  // of this tile and the next: keys' and values' rows
        float scale[2][KT];    // of keys, of values
        float p[KT][16];
    };
    struct Joined {
        float o[kFewWaves][16][kPitch];
        float m[kFewWaves][16], l[kFewWaves][16];
    };
    struct Main {
        PerWave wave[kFewWaves];
        uint32_t q[kQueriesInLds ? NK * 64 * 4 : 1];
    };
    static constexpr size_t kLds = sizeof(Main) > sizeof(Joined) ? sizeof(Main) : sizeof(Joined);
};

// ROWS: 8-bit values have a scale for each row.
template <typename T, typename E, int DP, int KB, bool AHEAD, bool ROWS>
__global__ void __launch_bounds__(64 * kFewWaves, (DP <= 128 ? 2 : 1))
    bmmc_attend_few_kernel(const AttendArgs x, int64_t block0) {
    using F = Few<T, E, DP, KB, AHEAD>;
    constexpr int CE = F::CE, NK = F::NK, VE = F::VE, VG = F::VG, KT = F::KT, VK = F::VK, KG = F::KG;
    constexpr bool kNarrow = sizeof(E) == 1;
    typedef typename Product<T>::vec vec_t;
    typedef typename Weighed<T, ROWS>::type W;
    typedef typename Product<W>::vec weights_t;
    constexpr bool kTwo = Weighed<T, ROWS>::kTwo;
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    typename F::Main &main_lds = *reinterpret_cast<typename F::Main *>(lds);
    typename F::Joined &joined = *reinterpret_cast<typename F::Joined *>(lds);

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = lane & 15, g = lane >> 4;
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
        tile = uniform(find_tile(x, number));
        unit = tile.first;
        stop = tile.first + tile.units;
    }
    typename F::PerWave &mine = main_lds.wave[wave];

    while (tile.found && unit < stop) {
        const int32_t unit0 = (int32_t)(unit - tile.first);
        const int32_t unit1 = (int32_t)min(stop - tile.first, (int64_t)tile.units);
        const Span span = span_of(x, tile, unit0, unit1);
        const int32_t *table = x.a.table + (int64_t)tile.seq * x.a.table_stride;

        // this lane's row
        const int64_t row = (int64_t)tile.tile * 16 + n;
        const bool on = row < (int64_t)tile.q.count * x.group;
        const int32_t token = (int32_t)quotient(x.by_group, (uint32_t)row);
        const int32_t place = tile.q.length - tile.q.count + token;
        // lanes 0 to 31 look after the keys, 32 to 63 after the values of a tile
        const int kl = lane & 31, half = lane >> 5;
        const uint8_t *base = static_cast<const uint8_t *>(half ? x.v.data : x.k.data);
        const int64_t by_page = half ? x.v.page_stride : x.k.page_stride;
        const int64_t by_place = half ? x.v.place_stride : x.k.place_stride;
        const int64_t by_head = (half ? x.v.head_stride : x.k.head_stride) * head;
            const auto look = [&](int32_t t) { return entry_of(x, table, t + kl, span.to); };
        float scale_next = 0.0f;
        // Rows of the tile at t into LDS; bits of the keys that are there
        const auto put = [&](int32_t entry, int32_t t, int which) {
            const int32_t page = kl < KT ? page_of(x, entry, t + kl, span.to) : -1;
            const int32_t in = t + kl - (int32_t)quotient(x.by_page, (uint32_t)(t + kl)) * (int32_t)x.by_page.d;
            if (kl < KT)
                mine.at[which][half][kl] =
                    page < 0 ? reinterpret_cast<const uint8_t *>(kZeros)
                             : base + (page * by_page + in * by_place + by_head) * (int64_t)sizeof(E);
            if (ROWS) {
                const bmmc_scaled_cache &c = half ? x.v : x.k;
                scale_next = page < 0 ? 0.0f
                                      : c.scale[page * c.scale_page + in * c.scale_place + head * c.scale_head];
            }
            wave_fence();
            return (uint32_t)__ballot(page >= 0);  // the keys' lanes
        };
        Raw<E, CE> kr[AHEAD ? KB : 1][KG];
        Raw<E, VE> vr[VK][AHEAD ? VG : 1];
        const auto load_keys = [&](int which, int b, int k0) {
            const uint8_t *in = mine.at[which][0][b * 16 + n];
            if (x.a.k_dim == DP) {
#pragma unroll
                for (int k = 0; k < KG; ++k)
                    kr[AHEAD ? b : 0][k] = fetch_whole<E, CE>(in, ((k0 + k) * 4 + g) * CE);
                return;
            }
            const int dim = kept(x.a.k_dim);
#pragma unroll
            for (int k = 0; k < KG; ++k)
                kr[AHEAD ? b : 0][k] = fetch<E, CE>(in, ((k0 + k) * 4 + g) * CE, dim);
        };
        const auto load_values = [&](int which, int v) {
            const int dim = kept(x.a.v_dim);
#pragma unroll
            for (int j = 0; j < VK; ++j) {
                const uint8_t *in = mine.at[which][1][(j >> 2) * 16 + g * 4 + (j & 3)];
                vr[j][AHEAD ? v : 0] = fetch<E, VE>(in, (v * 16 + n) * VE, dim);
            }
        };
        const auto load_all_keys = [&](int which) {
#pragma unroll
            for (int b = 0; b < KB; ++b) load_keys(which, b, 0);
        };
        const auto load_all_values = [&](int which) {
#pragma unroll
            for (int v = 0; v < VG; ++v) load_values(which, v);
        };

        float c = x.a.scale * 1.4426950408889634f, by_value = 1.0f;
        if (kNarrow && !ROWS && x.a.pages) {  // without pages there may be no scales
            c *= x.k.scale[head * x.k.scale_head];
            by_value = x.v.scale[head * x.v.scale_head];
        }
        f4 o[VG][VE];
#pragma unroll
        for (int v = 0; v < VG; ++v)
#pragma unroll
            for (int e = 0; e < VE; ++e) o[v][e] = f4{0.0f, 0.0f, 0.0f, 0.0f};
        float m = kNothing, l = 0.0f;

        const int32_t step = kFewWaves * KT;
        int32_t t = span.from + wave * KT;
        int which = 0;
        const int32_t first = t < span.to ? look(t) : -1;  // on its way while the queries are
        vec_t q[F::kQueriesInLds ? 1 : NK];
        {
            const int64_t h = (int64_t)head * x.group + (row - (int64_t)token * x.group);
            const uint8_t *in = reinterpret_cast<const uint8_t *>(kZeros);
            if (on)
                in = reinterpret_cast<const uint8_t *>(
                    static_cast<const T *>(x.a.q) +
                    (tile.q.first + (int64_t)token) * x.a.q_token + h * x.a.q_head);
            const int dim = kept(x.a.k_dim);
#pragma unroll
            for (int k = 0; k < NK; ++k) {
                if (F::kQueriesInLds && (k & (kFewWaves - 1)) != wave) continue;
                Raw<T, CE> r = fetch<T, CE>(in, (k * 4 + g) * CE, dim);
                if (dim & (CE - 1)) settle(r, (k * 4 + g) * CE, dim);
                if constexpr (F::kQueriesInLds)
                    *reinterpret_cast<u4 *>(&main_lds.q[(k * 64 + lane) * 4]) =
                        u4{r.w[0], r.w[1], r.w[2], r.w[3]};
                else
                    q[k] = product_vec<T>(r);
            }
            if constexpr (F::kQueriesInLds) __syncthreads();
        }
        // What is on its way, in this order: the table's entries for the tile after the
        // next, the next tile's keys, its values.  A wait for the first leaves the others.
        int32_t entry = -1;
        uint32_t seen = 0;
        if (t < span.to) {
            seen = put(first, t, 0);
            entry = look(t + step);
            __builtin_amdgcn_sched_barrier(0);
            if (AHEAD) load_all_keys(0);
            __builtin_amdgcn_sched_barrier(0);
            if (AHEAD) load_all_values(0);
            __builtin_amdgcn_sched_barrier(0);
        }
        // the queries are here before the loop, in which nothing waits for them
        if constexpr (!F::kQueriesInLds)
#pragma unroll
            for (int k = 0; k < NK; ++k) asm volatile("" : "+v"(q[k]));
        for (; t < span.to; t += step) {
            const uint32_t there = seen;
            f4 s[KB];
#pragma unroll
            for (int b = 0; b < KB; ++b) {
                s[b] = f4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int k0 = 0; k0 < NK; k0 += KG) {
                    if (!AHEAD) {
                        __builtin_amdgcn_sched_barrier(0);  // no more than this in registers
                        load_keys(which, b, k0);
                    }
                    Raw<E, CE> *const at = kr[AHEAD ? b : 0];
                    if (x.a.k_dim & (CE - 1)) {
                        const int dim = kept(x.a.k_dim);
#pragma unroll
                        for (int k = 0; k < KG; ++k) settle(at[k], ((k0 + k) * 4 + g) * CE, dim);
                    }
#pragma unroll
                    for (int k = 0; k < KG; ++k) {
                        vec_t qk;
                        if constexpr (F::kQueriesInLds) {
                            const u4 w =
                                *reinterpret_cast<const u4 *>(&main_lds.q[((k0 + k) * 64 + lane) * 4]);
                            __builtin_memcpy(&qk, &w, 16);
                        } else {
                            qk = q[k];
                        }
                        s[b] = mfma16(product_vec<T>(at[k]), qk, s[b]);
                    }
                }
                wait_for(s[b]);
            }
            if (ROWS) {
                if (kl < KT) mine.scale[half][kl] = scale_next;
                wave_fence();
            }
            // behind the last tile there are rows of zeros: a loop without branches
            // around its loads, or the compiler would wait for all of them at once
            seen = put(entry, t + step, which ^ 1);
            entry = look(t + 2 * step);
            __builtin_amdgcn_sched_barrier(0);
            if (AHEAD) load_all_keys(which ^ 1);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int b = 0; b < KB; ++b) {
                f4 by{c, c, c, c};
                if (ROWS) by *= *reinterpret_cast<const f4 *>(&mine.scale[0][b * 16 + g * 4]);
                s[b] *= by;
            }
            // the tile has keys that are not there, or that some rows do not see
            const bool parted = t + KT - 1 > span.first ||
                                (x.a.window && t <= span.last - x.a.window);
            uint32_t see = there;
            if (parted || ~there << (32 - KT)) {
                see &= (uint32_t)seen_of(place - t, x.a.window);
                const uint32_t lane_sees = see >> 4 * g;
#pragma unroll
                for (int b = 0; b < KB; ++b)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (!(lane_sees & 1u << (b * 16 + i))) s[b][i] = kNothing;
            }
            float top = kNothing;
#pragma unroll
            for (int b = 0; b < KB; ++b)
#pragma unroll
                for (int i = 0; i < 4; ++i) top = fmaxf(top, s[b][i]);
            top = over_32(over_16(top, Largest()), Largest());
            const float m_new = fmaxf(m, top);
            if (__any(m_new != m)) {
                const float down = exp2_of(m - settled(m_new));
                l *= down;
#pragma unroll
                for (int v = 0; v < VG; ++v)
#pragma unroll
                    for (int e = 0; e < VE; ++e) o[v][e] *= down;
                m = m_new;
            }
            const float base = settled(m) - kLift<W>;
            float p[VK];
#pragma unroll
            for (int b = 0; b < KB; ++b) {
                f4 by{1.0f, 1.0f, 1.0f, 1.0f};
                if (ROWS) by = *reinterpret_cast<const f4 *>(&mine.scale[1][b * 16 + g * 4]);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float w = exp2_of(s[b][i] - base);
                    l += w;
                    p[b * 4 + i] = ROWS ? w * by[i] : w;
                }
            }
            // a weight of 0 times a scale that is no number would reach rows that do not see its key
            if (ROWS && parted)
#pragma unroll
                for (int j = 0; j < VK; ++j)
                    if (!(see >> 4 * g & 1u << (j / 4 * 16 + j % 4))) p[j] = 0.0f;
            // a value that is no number must not reach rows that do not see its key
            bool odd = false;
            if (parted) {
#pragma unroll
                for (int v = 0; v < VG; ++v) {
                    if (!AHEAD) load_values(which, v);
#pragma unroll
                    for (int j = 0; j < VK; ++j)
#pragma unroll
                        for (int i = 0; i < Raw<E, VE>::kWords; ++i)
                            odd |= has_nonfinite<E>(vr[j][AHEAD ? v : 0].w[i]);
                }
                odd = __any(odd);
            }
            if (odd) {
#pragma unroll
                for (int b = 0; b < KB; ++b)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int key = b * 16 + g * 4 + i;
                        mine.p[key][n] = p[b * 4 + i];
                    }
                wave_fence();
                for (int key = 0; key < KT; ++key) {
                    if (!(see >> key & 1u)) continue;  // this lane's row, as the weights'
                    const float w = mine.p[key][n];
                    const int dim = kept(x.a.v_dim);
                    const E *in = reinterpret_cast<const E *>(mine.at[which][1][key]);
#pragma unroll
                    for (int v = 0; v < VG; ++v)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
#pragma unroll
                            for (int e = 0; e < VE; ++e) {
                                const int d = (v * 16 + 4 * g + i) * VE + e;
                                if (d < dim) o[v][e][i] += w * element_of<T, E>(in + d);
                            }
                }
                wave_fence();
            } else {
                weights_t pv, rest;  // rounded once here, and what that leaves out
                if constexpr (sizeof(T) == 2)
#pragma unroll
                    for (int j = 0; j < VK; ++j) pv[j] = (W)p[j];
                if constexpr (kTwo)
#pragma unroll
                    for (int j = 0; j < VK; ++j) rest[j] = (W)(p[j] - (float)pv[j]);
#pragma unroll
                for (int v = 0; v < VG; ++v) {
                    constexpr int kWords = VE * (int)sizeof(T) / 4;
                    const int at = AHEAD ? v : 0;
                    if (!AHEAD) {
                        __builtin_amdgcn_sched_barrier(0);
                        load_values(which, v);
                    }
                    if (x.a.v_dim & (VE - 1)) {
                        const int dim = kept(x.a.v_dim);
#pragma unroll
                        for (int j = 0; j < VK; ++j) settle(vr[j][at], (v * 16 + n) * VE, dim);
                    }
                    uint32_t w[VK][kWords];
#pragma unroll
                    for (int j = 0; j < VK; ++j) expand<W>(vr[j][at], w[j]);
#pragma unroll
                    for (int e = 0; e < VE; ++e) {
                        if constexpr (sizeof(T) == 4) {
#pragma unroll
                            for (int j = 0; j < VK; ++j)
                                o[v][e] = mfma16(__builtin_bit_cast(float, w[j][e]), p[j], o[v][e]);
                        } else {
                            uint32_t keys[4];
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                keys[j] = __builtin_amdgcn_perm(w[2 * j + 1][e / 2], w[2 * j][e / 2],
                                                                e & 1 ? 0x07060302u : 0x05040100u);
                            weights_t a;
                            __builtin_memcpy(&a, keys, 16);
                            o[v][e] = mfma16(a, pv, o[v][e]);
                            if constexpr (kTwo) o[v][e] = mfma16(a, rest, o[v][e]);
                        }
                    }
                }
            }
            which ^= 1;
            if (AHEAD) load_all_values(which);
        }

        // the waves joined
        l += __shfl_xor(l, 16, 64);
        l += __shfl_xor(l, 32, 64);
        __syncthreads();  // the addresses' part of LDS is free
        if (g == 0) {
            joined.m[wave][n] = m;
            joined.l[wave][n] = l;
        }
#pragma unroll
        for (int v = 0; v < VG; ++v)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int e = 0; e < VE; e += VE < 4 ? VE : 4) {
                    float *to = &joined.o[wave][n][(v * 16 + 4 * g + i) * VE + e];
                    if constexpr (VE == 2)
                        *reinterpret_cast<float2 *>(to) = make_float2(o[v][0][i], o[v][1][i]);
                    else
                        *reinterpret_cast<f4 *>(to) =
                            f4{o[v][e][i], o[v][e + 1][i], o[v][e + 2][i], o[v][e + 3][i]};
                }
        __syncthreads();
        const int r = threadIdx.x >> 4, col = threadIdx.x & 15;
        const int64_t out_row = (int64_t)tile.tile * 16 + r;
        if (out_row < (int64_t)tile.q.count * x.group) {
            float top = kNothing;
#pragma unroll
            for (int w = 0; w < kFewWaves; ++w) top = fmaxf(top, joined.m[w][r]);
            float by[kFewWaves], sum = 0.0f;
#pragma unroll
            for (int w = 0; w < kFewWaves; ++w) {
                by[w] = exp2_of(joined.m[w][r] - settled(top));
                sum += joined.l[w][r] * by[w];
                by[w] *= by_value;
            }
            const bool whole = unit0 == 0 && unit1 == tile.units;
            const int64_t slot = ((number * 2 + (unit0 == 0)) * heads + head) * 16 + r;
            const int32_t tok = (int32_t)quotient(x.by_group, (uint32_t)out_row);
            T *out = static_cast<T *>(x.a.out) + (tile.q.first + (int64_t)tok) * x.a.out_token +
                     ((int64_t)head * x.group + (out_row - (int64_t)tok * x.group)) * x.a.out_head;
            if (!whole && col == 0) x.state[slot] = make_float2(top, sum);
            const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
            for (int d = col * 4; d < x.a.v_dim; d += 64) {
                f4 y{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int w = 0; w < kFewWaves; ++w)
                    y += by[w] * *reinterpret_cast<const f4 *>(&joined.o[w][r][d]);
                if (whole) {
                    y = sum == 0.0f ? f4{0.0f, 0.0f, 0.0f, 0.0f} : y * inv;
                    if (d + 4 <= x.a.v_dim) {
                        Floats<4> z = y;
                        store<T, 4, false>(out + d, narrow<T, 4>(z));
                    } else {
                        for (int i = 0; i < x.a.v_dim - d; ++i) out[d + i] = (T)y[i];
                    }
                } else {
                    *reinterpret_cast<f4 *>(x.partial + slot * x.pitch + d) = y;
                }
            }
        }
        unit = tile.first + unit1;
        if (unit < stop) next_tile(x, tile);
        __syncthreads();  // LDS is used again
    }
    if (x.plan.shares && head == 0) leave_begun(x, (int32_t)number, share, tile);
}

// The parts of a tile joined, by the share that began it; a wave takes a row at a
// time, LANES lanes a part with 4 C elements each.
template <typename T, int LANES, int C>
__global__ void __launch_bounds__(256) bmmc_attend_join_kernel(const AttendArgs x, int64_t block0) {
    constexpr int kParts = 64 / LANES;       // that a wave loads at once
    constexpr int kAhead = C == 1 ? 8 : 4;   // such loads on their way
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t block = block0 + blockIdx.x, heads = x.a.heads;
    const int32_t share0 = (int32_t)(block / heads);
    const int head = (int)(block - share0 * heads);
    const int4 begun = x.begun[share0];
    const int32_t share1 = uniform(begun.x);
    if (share1 < 0) return;
    const int64_t row0 = (int64_t)uniform(begun.w) * x.plan.rows;
    const int rows = (int)min((int64_t)uniform(begun.z) * x.group - row0, (int64_t)x.plan.rows);
    const int32_t count = share1 - share0 + 1;
    const int dim = x.a.v_dim, pitch = x.pitch, at = lane % LANES * 4, mine = lane / LANES;
    for (int r = blockIdx.y * 4 + wave; r < rows; r += gridDim.y * 4) {
        // the first share holds the tile's begin
        const auto slot_of = [&](int32_t p) {
            return (((int64_t)(share0 + p) * 2 + (p == 0)) * heads + head) * x.plan.rows + r;
        };
        const auto state_of = [&](int32_t p) {
            return p < count ? x.state[slot_of(p)] : make_float2(kNothing, 0.0f);
        };
        float2 state = state_of(lane);
        f4 in[kAhead][C];
        const auto fetch_parts = [&](int32_t p0) {
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const float *from = x.partial + slot_of(min(p0 + k * kParts + mine, count - 1)) * pitch;
#pragma unroll
                for (int j = 0; j < C; ++j)
                    in[k][j] = *reinterpret_cast<const f4 *>(from + min(at + j * LANES * 4, pitch - 4));
            }
        };
        // the first parts are fetched before their weights are known
        fetch_parts(0);
        float top = state.x;
        for (int32_t p = 64; p < count; p += 64) top = fmaxf(top, state_of(p + lane).x);
        top = over_32(over_16(top, Largest()), Largest());
#pragma unroll
        for (int d = 8; d; d >>= 1) top = fmaxf(top, __shfl_xor(top, d, 64));
        float sum = 0.0f;
        f4 y[C];
#pragma unroll
        for (int j = 0; j < C; ++j) y[j] = f4{0.0f, 0.0f, 0.0f, 0.0f};
        for (int32_t p0 = 0; p0 < count; p0 += 64) {
            if (p0) state = state_of(p0 + lane);
            const float by = exp2_of(state.x - settled(top));
            sum += state.y * by;
            for (int32_t p = p0; p < min(p0 + 64, count); p += kAhead * kParts) {
                f4 now[kAhead][C];
#pragma unroll
                for (int k = 0; k < kAhead; ++k)
#pragma unroll
                    for (int j = 0; j < C; ++j) now[k][j] = in[k][j];
                if (p + kAhead * kParts < count) fetch_parts(p + kAhead * kParts);
#pragma unroll
                for (int k = 0; k < kAhead; ++k) {
                    const int part = p + k * kParts + mine;
                    const float weight = __shfl(by, (part - p0) & 63, 64);
                    if (part < count)
#pragma unroll
                        for (int j = 0; j < C; ++j) y[j] += weight * now[k][j];
                }
            }
        }
        sum = wave_sum(sum);
#pragma unroll
        for (int j = 0; j < C; ++j)
#pragma unroll
            for (int d = LANES; d < 64; d <<= 1)
#pragma unroll
                for (int i = 0; i < 4; ++i) y[j][i] += __shfl_xor(y[j][i], d, 64);
        const int32_t token = (int32_t)quotient(x.by_group, (uint32_t)(row0 + r));
        T *out = static_cast<T *>(x.a.out) + (begun.y + (int64_t)token) * x.a.out_token +
                 ((int64_t)head * x.group + (row0 + r - (int64_t)token * x.group)) * x.a.out_head;
        if (mine) continue;
#pragma unroll
        for (int j = 0; j < C; ++j) {
            const int to = at + j * LANES * 4;
            const f4 z = sum == 0.0f ? f4{0.0f, 0.0f, 0.0f, 0.0f} : y[j] / sum;
            if (to + 4 <= dim) {
                Floats<4> w = z;
                store<T, 4, false>(out + to, narrow<T, 4>(w));
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (to + i < dim) out[to + i] = (T)z[i];
            }
        }
    }
}

template <typename T, typename E, int DP, int KB, bool AHEAD>
int few(const AttendArgs &x, hipStream_t s) {
    using F = Few<T, E, DP, KB, AHEAD>;
    const bool rows = sizeof(E) == 1 && x.rows_scaled;
    const auto kernel = rows ? bmmc_attend_few_kernel<T, E, DP, KB, AHEAD, sizeof(E) == 1>
                             : bmmc_attend_few_kernel<T, E, DP, KB, AHEAD, false>;
    const int64_t blocks = (x.plan.shares ? x.plan.shares : x.plan.tiles) * x.a.heads +
                           (x.a.clear_rest && x.a.starts ? kClearBlocks : 0);
    return in_launches(blocks, 64 * kFewWaves, [&](uint32_t nb, int64_t b0) {
        hipLaunchKernelGGL(kernel, dim3(nb), dim3(64 * kFewWaves), F::kLds, s, x, b0);
    });
}

template <typename T, typename E> int few_by_size(const AttendArgs &x, hipStream_t s) {
    constexpr bool kWide = sizeof(T) == 4;
    const int dim = x.a.k_dim > x.a.v_dim ? x.a.k_dim : x.a.v_dim;
    // Padding costs products and, from 8 bits, widening of zeros: heads of 96 from 8 bits
    // padded to 128 take 67 us, to 96 62; 80 and 72 elements in 32 bits 95 and 91.
    // Tiles of 64 keys a wave: 84 us for the former, with twice the keys on their way.
    if (dim <= 64) return few<T, E, 64, 2, true>(x, s);
    if (dim <= 96) return few<T, E, 96, 2, true>(x, s);
    if (dim <= 128) return few<T, E, 128, kWide ? 1 : 2, true>(x, s);
    if (dim <= 256) return few<T, E, 256, kWide ? 1 : 2, true>(x, s);
    return few<T, E, 512, kWide ? 1 : 2, false>(x, s);
}

template <typename T> int few_by_cache(const AttendArgs &x, hipStream_t s) {
    return x.k.type == BMMC_E4M3 ? few_by_size<T, uint8_t>(x, s) : few_by_size<T, T>(x, s);
}

template <typename T, int LANES, int C> int join(const AttendArgs &x, hipStream_t s) {
    // a wave for each row that a tile has on average; 4096 workgroups that find
    // nothing to do take 4 us
    const int64_t filled = std::max<int64_t>(std::min(x.a.batch, x.a.tokens), 1);
    const int64_t rows = std::min<int64_t>((x.a.tokens * x.group + filled - 1) / filled, x.plan.rows);
    const int64_t blocks = x.plan.shares * x.a.heads;
    const uint32_t groups = (uint32_t)std::max<int64_t>(std::min((rows + 3) / 4, 4096 / blocks), 1);
    return in_launches(blocks, 256 * groups, [&](uint32_t nb, int64_t b0) {
        hipLaunchKernelGGL((bmmc_attend_join_kernel<T, LANES, C>), dim3(nb, groups), dim3(256), 0, s, x, b0);
    });
}

template <typename T> int join_by_size(const AttendArgs &x, hipStream_t s) {
    if (x.pitch <= 64) return join<T, 16, 1>(x, s);
    if (x.pitch <= 128) return join<T, 32, 1>(x, s);
    return x.pitch <= 256 ? join<T, 64, 1>(x, s) : join<T, 64, 2>(x, s);
}

}  // namespace

int launch_attend_few(const AttendArgs &x, hipStream_t s) {
    switch (x.a.type) {
    case BMMC_F32: return few_by_cache<float>(x, s);
    case BMMC_F16: return few_by_cache<f16_t>(x, s);
    default: return few_by_cache<bf16_t>(x, s);
    }
}

int launch_attend_join(const AttendArgs &x, hipStream_t s) {
    switch (x.a.type) {
    case BMMC_F32: return join_by_size<float>(x, s);
    case BMMC_F16: return join_by_size<f16_t>(x, s);
    default: return join_by_size<bf16_t>(x, s);
    }
}

}  // namespace bmmc
