// attend.h -- what the kernels of the attention over a paged cache share: the
// sequences and their parts, rows of the cache, and the products' types.
#pragma once

#include "../tokens/device.h"
#include "lanes.h"
#include "layer.h"

namespace bmmc {
namespace dev {

constexpr float kNothing = -__builtin_inff();  // the maximum of no score

typedef float f4 __attribute__((ext_vector_type(4)));
typedef uint32_t u2 __attribute__((ext_vector_type(2)));
typedef uint32_t u4 __attribute__((ext_vector_type(4)));

// What all lanes of a wave know to be the same, in scalar registers.
__device__ __forceinline__ int32_t uniform(int32_t v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ uint64_t uniform(uint64_t v) {
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)v);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
    return (uint64_t)hi << 32 | lo;
}
__device__ __forceinline__ int64_t uniform(int64_t v) { return (int64_t)uniform((uint64_t)v); }

// ---- sequences, tiles and parts ------------------------------------------------

// A sequence's new tokens: rows first .. first + count - 1 of q, the last at
// place length - 1.  Every number from the arrays is bounded here.
struct Sequence {
    int32_t first, count, length, end;  // end: places that are there to be seen
};

__device__ __forceinline__ Sequence sequence_at(const AttendArgs &x, int32_t s) {
    const int32_t tokens = (int32_t)x.a.tokens;
    int32_t from = s, to = s + 1;
    if (x.a.starts) {
        from = min(max(x.a.starts[s], 0), tokens);
        to = min(max(x.a.starts[s + 1], 0), tokens);
    }
    const int32_t length = max(x.a.lengths[s], 0);
    return Sequence{from, max(to - from, 0), length, (int32_t)min((int64_t)length, x.reach)};
}

__device__ __forceinline__ int32_t ceil_div(int32_t a, int32_t b) {
    return (int32_t)(((int64_t)a + b - 1) / b);
}

__device__ __forceinline__ int32_t tiles_of(const AttendArgs &x, const Sequence &q) {
    return (int32_t)(((int64_t)q.count * x.group + x.plan.rows - 1) / x.plan.rows);
}

// The places [from, to) that the tokens at first to last see, from a multiple
// of 64 on.
struct Range {
    int32_t from, to;
};
__device__ __forceinline__ Range range_of(const AttendArgs &x, const Sequence &q, int32_t first,
                                          int32_t last) {
    Range r{0, min(q.end, last + 1)};
    if (x.a.window) r.from = (int32_t)max((int64_t)first - x.a.window + 1, (int64_t)0) & ~63;
    if (r.to < r.from) r.to = r.from;
    return r;
}

// Units of a sequence's tiles, each taken for as long as its last.
__device__ __forceinline__ int32_t units_of(const AttendArgs &x, const Sequence &q) {
    const Range r = range_of(x, q, q.length - q.count, q.length - 1);
    return max(ceil_div(r.to - r.from, x.plan.unit), 1);
}

// A tile of a sequence, and its first unit among all.
struct Tile {
    bool found;
    int32_t seq, tile, units;
    int64_t first;
    Sequence q;
};

// Sums over the lanes before this one and, of all, in *total.
template <typename W> __device__ __forceinline__ W sum_before(W v, W *total) {
    const int lane = threadIdx.x & 63;
    W upto = v;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const W o = __shfl_up(upto, d, 64);
        if (lane >= d) upto += o;
    }
    *total = uniform(__shfl(upto, 63, 64));
    return upto - v;
}

// 64 sequences, one a lane.
struct Sequences {
    Sequence q;
    int32_t tiles, units;
};
__device__ __forceinline__ Sequences sequences_from(const AttendArgs &x, int32_t s) {
    Sequences r{};
    r.units = 1;
    if (s < (int32_t)x.a.batch) {
        r.q = sequence_at(x, s);
        r.tiles = tiles_of(x, r.q);
        r.units = units_of(x, r.q);
    }
    return r;
}

// The tile that is number `in` of lane l's, or holds its unit `in`.
template <bool BY_TILE>
__device__ __forceinline__ Tile tile_in(const Sequences &r, int l, int32_t s0, int64_t start, int64_t in) {
    Tile t;
    t.found = true;
    t.seq = s0 + l;
    t.units = __builtin_amdgcn_readlane(r.units, l);
    t.q.first = __builtin_amdgcn_readlane(r.q.first, l);
    t.q.count = __builtin_amdgcn_readlane(r.q.count, l);
    t.q.length = __builtin_amdgcn_readlane(r.q.length, l);
    t.q.end = __builtin_amdgcn_readlane(r.q.end, l);
    if (BY_TILE)
        t.tile = (int32_t)in;
    else if (in >> 31)
        t.tile = uniform((int32_t)(in / t.units));
    else
        t.tile = uniform((int32_t)((uint32_t)in / (uint32_t)t.units));
    t.first = start + (int64_t)t.tile * t.units;
    return t;
}

// The want'th tile of all.  Every wave looks for itself, 64 sequences at a time: a
// prefix sum over the lanes tells which of them holds it.
__device__ __forceinline__ Tile find_tile(const AttendArgs &x, int64_t want) {
    for (int32_t s0 = 0; s0 < (int32_t)x.a.batch; s0 += 64) {
        const Sequences r = sequences_from(x, s0 + (threadIdx.x & 63));
        int64_t all;
        const int64_t before = sum_before((int64_t)r.tiles, &all);
        const uint64_t here = __ballot(want >= before && want < before + r.tiles);
        if (here) {
            const int l = __ffsll((unsigned long long)here) - 1;
            // its units are its own: it is no part of a share
            return tile_in<true>(r, l, s0, 0, want - uniform(__shfl(before, l, 64)));
        }
        want -= all;
    }
    return Tile{};
}

// A share's units of all, [from, to), and the tile that it begins in.
struct Share {
    int64_t each, over;  // shares below `over` have one unit more than the others
    int64_t from, to;
    Tile tile;
    __device__ __forceinline__ int64_t first_of(int64_t w) const { return w * each + min(w, over); }
    // The share that has unit u.
    __device__ __forceinline__ int32_t of(int64_t u) const {
        const int64_t more = over * (each + 1);
        if (u < more) return (int32_t)(u / (each + 1));
        return (int32_t)(over + (u - more) / each);
    }
};

// W: what holds the number of all units.
template <typename W> __device__ __forceinline__ Share find_share(const AttendArgs &x, int32_t number) {
    const int lane = threadIdx.x & 63;
    const int32_t batch = (int32_t)x.a.batch;
    Sequences r = sequences_from(x, lane);
    W all, before = sum_before((W)((W)r.tiles * r.units), &all);
    for (int32_t s0 = 64; s0 < batch; s0 += 64) {
        const Sequences more = sequences_from(x, s0 + lane);
        W sum;
        sum_before((W)((W)more.tiles * more.units), &sum);
        all += sum;
    }
    Share p;
    p.each = sizeof(W) == 4 ? (int64_t)quotient(x.by_shares, (uint32_t)all) : (int64_t)(all / x.plan.shares);
    p.over = all - p.each * x.plan.shares;
    p.from = p.first_of(number);
    p.to = p.first_of(number + 1);
    p.tile = Tile{};
    W start = 0;
    for (int32_t s0 = 0; p.from < p.to && s0 < batch; s0 += 64) {
        if (s0) {
            r = sequences_from(x, s0 + lane);
            W sum;
            before = sum_before((W)((W)r.tiles * r.units), &sum) + start;
            start += sum;
        } else {
            start = uniform(__shfl((W)(before + (W)r.tiles * r.units), 63, 64));
        }
        const W want = (W)p.from;
        const uint64_t here = __ballot(want >= before && want < before + (W)r.tiles * r.units);
        if (here) {
            const int l = __ffsll((unsigned long long)here) - 1;
            const int64_t first = uniform(__shfl(before, l, 64));
            p.tile = tile_in<false>(r, l, s0, first, p.from - first);
            return p;
        }
    }
    p.to = p.from;
    return p;
}
__device__ __forceinline__ Tile uniform(const Tile &t) {
    return Tile{t.found,
                uniform(t.seq),
                uniform(t.tile),
                uniform(t.units),
                uniform(t.first),
                Sequence{uniform(t.q.first), uniform(t.q.count), uniform(t.q.length), uniform(t.q.end)}};
}
__device__ __forceinline__ Share find_share(const AttendArgs &x, int32_t number) {
    Share p = x.few_units ? find_share<int32_t>(x, number) : find_share<int64_t>(x, number);
    p.each = uniform(p.each);
    p.over = uniform(p.over);
    p.from = uniform(p.from);
    p.to = uniform(p.to);
    p.tile = uniform(p.tile);
    return p;
}

// What a share leaves for the join of the tile that it began and did not end.
struct Begun {
    int32_t last_share;  // the tile's; -1: there is no such tile
    int32_t first, count, tile;
};
__device__ __forceinline__ void leave_begun(const AttendArgs &x, int32_t number, const Share &p,
                                            const Tile &t) {
    // t: the share's last tile, p.to its end
    const bool begun = t.found && t.first >= p.from && t.first + t.units > p.to;
    if (threadIdx.x == 0)
        x.begun[number] = begun ? int4{p.of(t.first + t.units - 1), t.q.first, t.q.count, t.tile}
                                : int4{-1, 0, 0, 0};
}

// The tile after t; not found behind the last.
__device__ __forceinline__ void next_tile(const AttendArgs &x, Tile &t) {
    t.first += t.units;
    if (++t.tile < tiles_of(x, t.q)) return;
    t.tile = 0;
    for (++t.seq; t.seq < (int32_t)x.a.batch; ++t.seq) {
        const Sequence q = sequence_at(x, t.seq);
        t.q = Sequence{uniform(q.first), uniform(q.count), uniform(q.length), uniform(q.end)};
        if (t.q.count) {
            t.units = units_of(x, t.q);
            return;
        }
    }
    t.found = false;
}

// The tokens of a tile, and the places that units [from, to) of it look at.
struct Span {
    int32_t first, last;  // places of the first and the last token
    int32_t from, to;
};
__device__ __forceinline__ Span span_of(const AttendArgs &x, const Tile &t, int32_t from, int32_t to) {
    const int64_t row0 = (int64_t)t.tile * x.plan.rows;
    const int64_t row1 = min(row0 + x.plan.rows, (int64_t)t.q.count * x.group) - 1;
    const int32_t base = t.q.length - t.q.count;
    Span s;
    s.first = base + (int32_t)quotient(x.by_group, (uint32_t)row0);
    s.last = base + (int32_t)quotient(x.by_group, (uint32_t)row1);
    const Range r = range_of(x, t.q, s.first, s.last);
    s.from = (int32_t)min(r.from + (int64_t)from * x.plan.unit, (int64_t)r.to);
    s.to = (int32_t)min(r.from + (int64_t)to * x.plan.unit, (int64_t)r.to);
    return s;
}

// Rows of no sequence, those before the first and behind the last, as zeros; by
// workgroups of their own.
template <typename T>
__device__ __forceinline__ void clear_rest(const AttendArgs &x, int64_t block, int64_t blocks) {
    if (!x.a.starts) return;
    const int32_t tokens = (int32_t)x.a.tokens;
    const int64_t head = min(max(x.a.starts[0], 0), tokens);
    const int64_t tail = max((int64_t)min(max(x.a.starts[x.a.batch], 0), tokens), head);
    const int64_t rows = head + tokens - tail;
    for (int64_t r = block; r < rows * x.a.q_heads; r += blocks) {
        const int64_t t = r / x.a.q_heads, h = r - t * x.a.q_heads;
        T *out = static_cast<T *>(x.a.out) + (t < head ? t : t - head + tail) * x.a.out_token +
                 h * x.a.out_head;
        for (int i = threadIdx.x; i < x.a.v_dim; i += blockDim.x) out[i] = (T)0.0f;
    }
}

// ---- elements --------------------------------------------------------------------

// What stands for a row that is not there: zeros, as long as the longest head.
__device__ const uint32_t __attribute__((aligned(16))) kZeros[BMMC_MAX_HEAD_DIM] = {};

// Rows are in global memory, which the compiler is told: their addresses come from
// LDS, and loads through generic addresses would wait for LDS as well.
//
// N elements of a row from element `at` on, zeros past its end.  Rows have N
// elements at least; the last vector of a row that is no whole number of them
// ends with the row, and `settle` shifts it into its place when the elements are
// used, and not before, when they are still on their way.
template <typename E, int N> struct Raw {
    static constexpr int kBytes = N * (int)sizeof(E);
    static constexpr int kWords = kBytes / 4;
    uint32_t w[kWords];
};
template <typename E, int N>
__device__ __forceinline__ Raw<E, N> fetch(const uint8_t *row, int at, int dim) {
    typedef typename Vec<uint8_t, Raw<E, N>::kBytes>::raw bytes_t;
    typedef bytes_t packed_t __attribute__((aligned(sizeof(E))));
    const uint8_t *from = row + min(at, dim - N) * (int)sizeof(E);
    if (at >= dim) from = reinterpret_cast<const uint8_t *>(kZeros);
    const bytes_t v = *(const __attribute__((address_space(1))) packed_t *)from;
    Raw<E, N> r;
    __builtin_memcpy(r.w, &v, sizeof(r.w));
    return r;
}
// The same of a row that reaches past the vector.
template <typename E, int N>
__device__ __forceinline__ Raw<E, N> fetch_whole(const uint8_t *row, int at) {
    typedef typename Vec<uint8_t, Raw<E, N>::kBytes>::raw bytes_t;
    typedef bytes_t packed_t __attribute__((aligned(sizeof(E))));
    const bytes_t v = *(const __attribute__((address_space(1))) packed_t *)(row + at * (int)sizeof(E));
    Raw<E, N> r;
    __builtin_memcpy(r.w, &v, sizeof(r.w));
    return r;
}
template <typename E, int N>
__device__ __forceinline__ void settle(Raw<E, N> &r, int at, int dim) {
    constexpr int W = Raw<E, N>::kWords;
    if (at + N <= dim || at >= dim) return;
    const int bits = (N - (dim & (N - 1))) * 8 * (int)sizeof(E);  // the same in all lanes
    if constexpr (W == 4)
        if (bits & 64) {
            r.w[0] = r.w[2];
            r.w[1] = r.w[3];
            r.w[2] = r.w[3] = 0;
        }
    if (W >= 2 && (bits & 32)) {
#pragma unroll
        for (int i = 0; i + 1 < W; ++i) r.w[i] = r.w[i + 1];
        r.w[W - 1] = 0;
    }
#pragma unroll
    for (int i = 0; i < W; ++i)
        r.w[i] = __builtin_amdgcn_alignbit(i + 1 < W ? r.w[i + 1] : 0u, r.w[i], bits & 31);
}

// A number that the compiler does not know to be the same each time: what hangs
// on it is made where it is used, and not kept in registers from tile to tile.
__device__ __forceinline__ int kept(int v) {
    asm volatile("" : "+s"(v));
    return v;
}
__device__ __forceinline__ int kept_lane(int v) {
    asm volatile("" : "+v"(v));
    return v;
}

// The inputs' type: vectors of 8 for the products of 16-bit types, of 4 in 32 bits.
template <typename T> struct Product {
    static constexpr int N = 8;
    typedef T vec __attribute__((ext_vector_type(8)));
};
template <> struct Product<float> {
    static constexpr int N = 4;
    typedef f4 vec;
};

// Words of two elements of T (one of float) from a row's raw words.
template <typename T, typename E, int N>
__device__ __forceinline__ void expand(const Raw<E, N> &r, uint32_t *w) {
    if constexpr (sizeof(E) > 1) {
#pragma unroll
        for (int i = 0; i < Raw<E, N>::kWords; ++i) w[i] = r.w[i];
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            typedef float f2 __attribute__((ext_vector_type(2)));
            const f2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)r.w[i], false);
            const f2 hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)r.w[i], true);
            const float v[4] = {lo[0], lo[1], hi[0], hi[1]};
            __builtin_memcpy(w + 4 * i, v, 16);
        }
    } else {  // e4m3's values are all values of both 16-bit types
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            if constexpr (__is_same(T, f16_t)) {
                const auto lo = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(r.w[i], 1.0f, false);
                const auto hi = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(r.w[i], 1.0f, true);
                __builtin_memcpy(w + 2 * i, &lo, 4);
                __builtin_memcpy(w + 2 * i + 1, &hi, 4);
            } else {
                const auto lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(r.w[i], 1.0f, false);
                const auto hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(r.w[i], 1.0f, true);
                __builtin_memcpy(w + 2 * i, &lo, 4);
                __builtin_memcpy(w + 2 * i + 1, &hi, 4);
            }
        }
    }
}

template <typename T, typename E>
__device__ __forceinline__ typename Product<T>::vec product_vec(const Raw<E, Product<T>::N> &r) {
    uint32_t w[Product<T>::N * sizeof(T) / 4];
    expand<T>(r, w);
    typename Product<T>::vec v;
    __builtin_memcpy(&v, w, sizeof(v));
    return v;
}

// Bit i: whether the token at place p sees place t + i, by p - t.
__device__ __forceinline__ uint64_t seen_of(int32_t ahead, int64_t window) {
    uint64_t see = ahead < 0 ? 0 : ahead >= 63 ? ~uint64_t(0) : (uint64_t(2) << ahead) - 1;
    const int64_t from = (int64_t)ahead - window + 1;
    if (window && from > 0) see = from > 63 ? 0 : see & ~((uint64_t(1) << from) - 1);
    return see;
}

// One element of a row.
template <typename T, typename E> __device__ __forceinline__ float element_of(const E *p) {
    const auto *q = (const __attribute__((address_space(1))) E *)p;
    if constexpr (sizeof(E) == 1)
        return __builtin_amdgcn_cvt_f32_fp8((int)*q, 0);
    else
        return (float)*q;
}

// c += a b of 16 x 16: lane l holds row (a) or column (b) l % 16 and 8 (32 bits:
// 1) of the inner elements, l / 16 the eighth; c's column is l % 16, its rows 4 (l / 16) + i.
__device__ __forceinline__ f4 mfma16(Product<f16_t>::vec a, Product<f16_t>::vec b, f4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f4 mfma16(Product<bf16_t>::vec a, Product<bf16_t>::vec b, f4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f4 mfma16(float a, float b, f4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f4 mfma16(Product<float>::vec a, Product<float>::vec b, f4 c) {
#pragma unroll
    for (int i = 0; i < 4; ++i) c = mfma16(a[i], b[i], c);
    return c;
}

// The results of matrix products that a branch parts from their use.  The compiler
// has been seen to count too few cycles between the two there, so that a result
// was read before it was written; this waits for all of them.
__device__ __forceinline__ void wait_for(f4 &x) { asm volatile("s_nop 15" : "+v"(x)); }

// What weights and values are in their product: the inputs' type, but bfloat16 for
// float16 inputs whose values have a scale for each row (ROWS).  There a weight is
// multiplied by its value's scale, and 5 exponent bits do not hold both: a row of zeros
// has the scale 1, one of small values 2^-20, and either may weigh 2^-14 of the other.
// So that no bits are lost for the exponent's, the weight goes into two products, as its
// rounding and as the rounding of what that leaves out, which is 2^-16 of it at most
// (float16: 2^-11).  e4m3's values are all values of both types.  One product and two:
// 4096 tokens of 4 sequences behind up to 2048 places, 16 over 4 heads of 128, 154 us
// (bfloat16) and 181; one token of 128 sequences of up to 4096, 24 over 4 heads of 96,
// 67.0 us and 67.7.
template <typename T, bool ROWS> struct Weighed {
    typedef T type;
    static constexpr bool kTwo = false;
};
template <> struct Weighed<f16_t, true> {
    typedef bf16_t type;
    static constexpr bool kTwo = true;
};

// Weights of type W are made as 2^(score - maximum + kLift).  In 16 bits of 5 exponent
// bits small ones would be lost below 2^-25 of the largest; lifted, below 2^-32.
template <typename W> constexpr float kLift = __is_same(W, f16_t) ? 7.0f : 0.0f;

__device__ __forceinline__ float exp2_of(float x) { return __builtin_amdgcn_exp2f(x); }

// An unseen maximum counts as 0, so that 2^(-inf - it) is 0 and not NaN.
__device__ __forceinline__ float settled(float m) { return m == kNothing ? 0.0f : m; }

__device__ __forceinline__ void wave_fence() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// The table's entry for a place before `end` (the last one for those behind it), as
// it is: looked at later, by page_of, so that nothing waits for it here.
__device__ __forceinline__ int32_t entry_of(const AttendArgs &x, const int32_t *table, int32_t place,
                                            int32_t end) {
    return table[quotient(x.by_page, (uint32_t)min(place, end - 1))];
}
// The page of a place, -1 where there is none.
__device__ __forceinline__ int32_t page_of(const AttendArgs &x, int32_t entry, int32_t place,
                                           int32_t end) {
    return place < end && entry >= 0 && entry < x.a.pages ? entry : -1;
}

}  // namespace dev
}  // namespace bmmc
