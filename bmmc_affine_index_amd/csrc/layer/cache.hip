// cache.hip -- a paged cache written in 8 bits with scales made on the way, and
// rows of a cache read back (gfx950).
//
// A head of a token is a row with a scale of its own: its largest finite
// magnitude / 448.  The largest is known only when all of the row has been
// turned, so a row lies in one wave, 16 elements a lane, and never leaves its
// registers: loaded, turned (both halves of a pair are in one lane), its largest
// magnitude found by moves among the row's lanes, divided and stored.
//
// Bound by memory: each element is read once and written once, keys and values in 1
// byte.  Turns are made once a token, in LDS, as for rotary positions.
//
// Measured: 16384 tokens of 24 + 8 heads of 128 and 8 of 96 in bf16, 291 MB: 64 us, 4.6
// TB/s (96 with 8 elements a lane, halves exchanged and true divisions); 64 tokens 4 us
// on the device.  Read back: 40001 tokens of 8 + 8 heads of 128, 8 bits to bf16, 249 MB:
// 51.5 us, 4.8 TB/s.
#include "../tokens/turns.h"
#include "lanes.h"
#include "layer.h"

namespace bmmc {

namespace {

constexpr int kPer = 8;  // elements of a vector; to quantize, a lane has two of its row

// Where a row's lanes are: `lanes` a row, a power of two, and 64 / lanes rows a wave.
struct RowCut {
    int32_t shift;  // log2 of lanes
    __device__ int row() const { return (threadIdx.x & 63) >> shift; }
    __device__ int lane() const { return threadIdx.x & ((1 << shift) - 1); }
    __host__ __device__ int rows_a_wave() const { return 64 >> shift; }
};

RowCut row_cut(int dim, int each) {
    RowCut c{0};
    while (each << c.shift < dim) ++c.shift;
    return c;
}

template <typename T, bool NT = false>
__device__ __forceinline__ dev::Vec<T, kPer> load_part(const T *row, int at, int dim) {
    if (at + kPer <= dim) return dev::load<T, kPer, NT>(row + at);
    dev::Vec<T, kPer> r;
#pragma unroll
    for (int i = 0; i < kPer; ++i) r.v[i] = at + i < dim ? row[at + i] : (T)0;
    return r;
}

template <typename T, bool NT = false>
__device__ __forceinline__ void store_part(T *row, int at, int dim, const dev::Vec<T, kPer> &x) {
    if (at + kPer <= dim) {
        dev::store<T, kPer, NT>(row + at, x);
        return;
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i)
        if (at + i < dim) row[at + i] = x.v[i];
}

// Tensors of a token's rows: q's heads, then k's, then v's.
struct Rows {
    const void *in;
    int64_t token, head;
};

struct Scaled {
    uint8_t *data;
    float *scale;
    int64_t page, place, head, scale_page, scale_place, scale_head;
};

Scaled scaled_of(const bmmc_scaled_cache &c) {
    return Scaled{static_cast<uint8_t *>(c.data), c.scale,       c.page_stride, c.place_stride,
                  c.head_stride,                  c.scale_page, c.scale_place, c.scale_head};
}

struct Quantize {
    Rows q, k, v;
    void *q_out;
    int64_t q_out_token, q_out_head;
    Scaled k_cache, v_cache;
    PageTable where;
    FastDiv by_tasks;
    int64_t tokens;
    RowCut cut;
    int32_t q_heads, heads, k_dim, v_dim, tokens_a_block;
    int32_t q_tasks, k_tasks;  // waves' tasks a token for q and for k
};

// 8 bits of value / scale.  The quotient is the product with by = 1 / scale, put right
// by what it leaves of x; it passes 448 by its rounding at most, which 8 bits round off.
__device__ __forceinline__ dev::Vec<uint8_t, kPer> quotients_of(const float (&x)[kPer], float scale,
                                                                float by) {
    uint32_t word[kPer / 4];
#pragma unroll
    for (int k = 0; k < kPer / 4; ++k) {
        float y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float q = x[4 * k + i] * by;
            y[i] = fmaf(fmaf(-q, scale, x[4 * k + i]), by, q);
        }
        const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
        word[k] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], lo, true);
    }
    dev::Vec<uint8_t, kPer> r;
    __builtin_memcpy(&r.v, word, kPer);
    return r;
}

// A part of a row: its elements, in 32 bits, and where in the row they are.
struct Part {
    float x[kPer];
    int at;
};

// Turned elements of a part whose pairs are its neighbours, or whose other halves are
// read from the row.
template <typename T, bool PAIRED>
__device__ __forceinline__ void turn_part(Part &p, const T *row, bool on, int pairs, const float2 *cs) {
#pragma unroll
    for (int i = 0; i < kPer; i += PAIRED ? 2 : 1) {
        const int e = p.at + i;
        if (e >= 2 * pairs) continue;
        if constexpr (PAIRED) {
            const float2 u = cs[e / 2];
            const float a = p.x[i], b = p.x[i + 1];
            p.x[i] = a * u.x - b * u.y;
            p.x[i + 1] = b * u.x + a * u.y;
        } else {
            const float2 u = cs[e < pairs ? e : e - pairs];
            const float other = on ? (float)row[e < pairs ? e + pairs : e - pairs] : 0.0f;
            p.x[i] = p.x[i] * u.x + (e < pairs ? -other : other) * u.y;
        }
    }
}

// WHOLE: rows, and halves of pairs, are whole vectors of a lane.
template <typename T, bool PAIRED, bool WHOLE>
__global__ void __launch_bounds__(kTurnThreads)
    bmmc_cache_quantize_kernel(const Quantize a, const Turn r, int64_t block0) {
    __shared__ float2 cs[kTurnPairs];
    __shared__ PagePlace places[kTurnTokens];
    const int64_t token0 = (block0 + blockIdx.x) * a.tokens_a_block;
    const int tokens = (int)min((int64_t)a.tokens_a_block, a.tokens - token0);
    const int per = (int)a.by_tasks.d, tasks = tokens * per, waves = blockDim.x >> 6;
    const int first = (int)(blockIdx.y * waves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6));
    const int step = (int)gridDim.y * waves;
    const int lane = a.cut.lane(), lane_row = a.cut.row(), rows = a.cut.rows_a_wave();

    // A lane has two vectors of its row: both halves of the same pairs, where those are
    // whole vectors, and of the rest one of each half, so that lanes side by side load and
    // store side by side.
    const int halves = !PAIRED && WHOLE ? r.pairs / kPer : 0;
    struct Row {
        const T *in;
        int t, kind, head;  // kind: 0 q, 1 k, 2 v
        bool on;
    } row{};
    dev::Vec<T, kPer> next[2];
    const auto at_of = [&](int kind, int half) {
        const int turned = kind == 2 ? 0 : halves;
        const int all = ((kind == 2 ? a.v_dim : a.k_dim) + kPer - 1) / kPer;
        const int rest = (all + 1) / 2 - turned;  // lanes of the rest
        const int by = lane < turned ? half * turned : lane < turned + rest ? turned + half * rest : all;
        return (lane + by) * kPer;
    };
    const auto fetch = [&](int task) {
        const int t = (int)quotient(a.by_tasks, (uint32_t)task);
        int number = task - t * per;
        const int kind = number < a.q_tasks ? 0 : number < a.q_tasks + a.k_tasks ? 1 : 2;
        number -= kind == 0 ? 0 : kind == 1 ? a.q_tasks : a.q_tasks + a.k_tasks;
        const Rows &x = kind == 0 ? a.q : kind == 1 ? a.k : a.v;
        const int head = number * rows + lane_row;
        row = Row{static_cast<const T *>(x.in) + (token0 + t) * x.token + head * x.head, t, kind,
                  head, head < (kind == 0 ? a.q_heads : a.heads)};
        const int dim = kind == 2 ? a.v_dim : a.k_dim;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int at = at_of(kind, h);
            next[h] = dev::Vec<T, kPer>{};
            if (row.on && at < dim) next[h] = load_part<T>(row.in + at, 0, WHOLE ? kPer : dim - at);
        }
    };
    const int looker = (int)threadIdx.x - ((int)blockDim.x - 64);
    if (looker >= 0 && looker < tokens) places[looker] = page_place(a.where, token0 + looker);
    make_turns(r, token0, r.pairs ? tokens : 0, cs, [&] {
        if (first < tasks) fetch(first);
    });
    __syncthreads();
    for (int task = first; task < tasks; task += step) {
        const Row w = row;
        Part p[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const dev::Floats<kPer> wide = dev::widen<T, kPer>(next[h]);
            p[h].at = at_of(w.kind, h);
#pragma unroll
            for (int i = 0; i < kPer; ++i) p[h].x[i] = wide[i];
        }
        if (task + step < tasks) fetch(task + step);
        const int dim = w.kind == 2 ? a.v_dim : a.k_dim;
        if (w.kind != 2 && r.pairs) {
            const float2 *turns = cs + w.t * r.pairs;
            if constexpr (!PAIRED && WHOLE) {
                if (lane < halves)
#pragma unroll
                    for (int i = 0; i < kPer; ++i) {
                        const float2 u = turns[p[0].at + i];
                        const float x = p[0].x[i], y = p[1].x[i];
                        p[0].x[i] = x * u.x + -y * u.y;
                        p[1].x[i] = y * u.x + x * u.y;
                    }
            } else {
#pragma unroll
                for (int h = 0; h < 2; ++h) turn_part<T, PAIRED>(p[h], w.in, w.on, r.pairs, turns);
            }
        }
        if (w.kind == 0) {
            if (!w.on) continue;
            T *out = static_cast<T *>(a.q_out) + (token0 + w.t) * a.q_out_token + w.head * a.q_out_head;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (p[h].at >= dim) continue;
                dev::Floats<kPer> y;
#pragma unroll
                for (int i = 0; i < kPer; ++i) y[i] = p[h].x[i];
                store_part<T>(out + p[h].at, 0, WHOLE ? kPer : dim - p[h].at, dev::narrow<T, kPer>(y));
            }
            continue;
        }
        // magnitudes are in the order of their bits, infinities and NaN behind the others
        uint32_t bits = 0;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                bits = max(bits, __builtin_bit_cast(uint32_t, p[h].x[i]) & 0x7fffffffu);
        const bool odd = __any(bits >= 0x7f800000u);
        float most = __builtin_bit_cast(float, bits);
        if (odd) {
            most = 0.0f;
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < kPer; ++i) {
                    const float m = fabsf(p[h].x[i]);
                    if (m < __builtin_inff()) most = fmaxf(most, m);
                }
        }
        most = dev::over_lanes(most, a.cut.shift, dev::Largest());
        const float scale = most == 0.0f ? 1.0f : fmaxf(most / 448.0f, 0x1p-126f);
        const float by = 1.0f / scale;
        if (odd) {  // infinities become what is stored as the type's largest; NaN stays
            const float largest = fminf(448.0f * scale, 0x1.fffffep127f);
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < kPer; ++i)
                    if (fabsf(p[h].x[i]) == __builtin_inff())
                        p[h].x[i] = __builtin_copysignf(largest, p[h].x[i]);
        }
        const PagePlace home{__builtin_amdgcn_readfirstlane(places[w.t].page),
                             __builtin_amdgcn_readfirstlane(places[w.t].place)};
        if (home.page < 0 || !w.on) continue;
        const Scaled &c = w.kind == 1 ? a.k_cache : a.v_cache;
        uint8_t *out = c.data + home.page * c.page + home.place * c.place + w.head * c.head;
        if (lane == 0)
            c.scale[home.page * c.scale_page + home.place * c.scale_place + w.head * c.scale_head] =
                scale;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (p[h].at >= dim) continue;
            store_part<uint8_t>(out + p[h].at, 0, WHOLE ? kPer : dim - p[h].at,
                                quotients_of(p[h].x, scale, by));
        }
    }
}

template <typename T, bool PAIRED> int quantize(const QuantizeArgs &h, hipStream_t s) {
    const Turn r = turn_of<1>(h.rotation);
    Quantize a{};
    a.q = Rows{h.q.in, h.q.in_token, h.q.in_head};
    a.k = Rows{h.k.in, h.k.in_token, h.k.in_head};
    a.v = Rows{h.v.in, h.v.in_token, h.v.in_head};
    a.q_out = h.q.out;
    a.q_out_token = h.q.out_token;
    a.q_out_head = h.q.out_head;
    a.k_cache = scaled_of(h.k_cache);
    a.v_cache = scaled_of(h.v_cache);
    a.where = h.where;
    a.tokens = h.tokens;
    a.cut = row_cut(std::max(h.k_dim, h.v_dim), 2 * kPer);
    a.q_heads = (int32_t)h.q.heads;
    a.heads = (int32_t)h.k.heads;
    a.k_dim = h.k_dim;
    a.v_dim = h.v_dim;
    const int rows = a.cut.rows_a_wave();
    a.q_tasks = (a.q_heads + rows - 1) / rows;
    a.k_tasks = (a.heads + rows - 1) / rows;
    const int64_t tasks = a.q_tasks + 2 * a.k_tasks;
    a.by_tasks = fast_div((uint32_t)tasks);
    // Many tokens go four to a workgroup, whose waves then have as many tasks each
    // (16384 tokens of 5 tasks: 1 token 75 us, 2 65.2, 3 64.1, 4 65.0, 6 68.7, 8 71.0).
    // Streamed loads and stores: 70, rows being written in parts of lines.
    TurnCut cut = turn_cut(a.tokens, r.pairs, tasks);
    const int n = std::min(kTurnTokens, r.pairs ? kTurnPairs / r.pairs : kTurnTokens);
    if (a.tokens / n >= kTurnBlocks) cut = TurnCut{n, kTurnWaves, (a.tokens + n - 1) / n, 1};
    a.tokens_a_block = cut.tokens_a_block;
    const bool whole = h.k_dim % kPer == 0 && h.v_dim % kPer == 0 && (PAIRED || r.pairs % kPer == 0);
    const auto kernel = whole ? bmmc_cache_quantize_kernel<T, PAIRED, true>
                              : bmmc_cache_quantize_kernel<T, PAIRED, false>;
    return in_launches(cut.blocks, kTurnThreads, [&](uint32_t nb, int64_t b0) {
        hipLaunchKernelGGL(kernel, dim3(nb, cut.shares), dim3(64 * cut.waves), 0, s, a, r, b0);
    });
}

template <typename T> int quantize_t(const QuantizeArgs &h, hipStream_t s) {
    return h.rotation.interleaved ? quantize<T, true>(h, s) : quantize<T, false>(h, s);
}

// ---- rows read back ------------------------------------------------------------------

constexpr int kReadTokens = 64;  // most of a workgroup
constexpr int kReadBlocks = 2048;
constexpr int kReadAhead = 4;    // rows a lane has on their way

// Keys or values: one grid's half each, so that all of it is the same in a workgroup.
struct ReadHalf {
    void *out;
    int64_t out_token, out_head;
    Scaled cache;
    int32_t dim;
};

struct Read {
    ReadHalf half[2];
    PageTable where;
    FastDiv by_heads;
    int64_t tokens;
    RowCut cut;
    int32_t heads, tokens_a_block;
};

// Where a token's rows and their scales begin, in elements; `in` is below 0 if nowhere.
struct ReadPlace {
    int64_t in, scale;
};

template <typename E> __device__ __forceinline__ dev::Floats<kPer> widened(const dev::Vec<E, kPer> &x) {
    if constexpr (sizeof(E) == 1) {
        uint32_t w[2];
        __builtin_memcpy(w, &x.v, 8);
        dev::Floats<kPer> y;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], false);
            const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], true);
            y[4 * i] = lo[0];
            y[4 * i + 1] = lo[1];
            y[4 * i + 2] = hi[0];
            y[4 * i + 3] = hi[1];
        }
        return y;
    } else {
        return dev::widen<E, kPer>(x);
    }
}

// WHOLE: rows are whole vectors of a lane.
template <typename T, typename E, bool WHOLE, bool NT>
__global__ void __launch_bounds__(256) bmmc_cache_read_kernel(const Read a, int64_t block0) {
    __shared__ ReadPlace places[kReadTokens];
    const ReadHalf &x = a.half[blockIdx.z];
    const int64_t token0 = (block0 + blockIdx.x) * a.tokens_a_block;
    const int tokens = (int)min((int64_t)a.tokens_a_block, a.tokens - token0);
    if ((int)threadIdx.x < tokens) {
        const PagePlace p = page_place(a.where, token0 + threadIdx.x);
        places[threadIdx.x] =
            ReadPlace{p.page < 0 ? -1 : p.page * x.cache.page + p.place * x.cache.place,
                      p.page * x.cache.scale_page + p.place * x.cache.scale_place};
    }
    __syncthreads();
    const int at = a.cut.lane() * kPer, each = a.cut.rows_a_wave() * 4;  // rows of a workgroup at once
    if (at >= x.dim) return;
    const int mine = (int)(threadIdx.x >> 6) * a.cut.rows_a_wave() + a.cut.row();
    const int rows = tokens * a.heads;
    const E *const in = reinterpret_cast<const E *>(x.cache.data) + at;
    T *const out = static_cast<T *>(x.out) + token0 * x.out_token + at;
    const int size = WHOLE ? kPer : x.dim - at;
    for (int base = (int)blockIdx.y * each * kReadAhead; base < rows;
         base += (int)gridDim.y * each * kReadAhead) {
        dev::Vec<E, kPer> raw[kReadAhead];
        float scale[kReadAhead];
        int64_t to[kReadAhead];
#pragma unroll
        for (int j = 0; j < kReadAhead; ++j) {
            // rows behind the last are read as the last, and not written
            const uint32_t row = (uint32_t)min(base + j * each + mine, rows - 1);
            const uint32_t t = quotient(a.by_heads, row), head = row - t * (uint32_t)a.heads;
            to[j] = t * x.out_token + head * x.out_head;
            raw[j] = dev::Vec<E, kPer>{};
            scale[j] = 1.0f;
            const ReadPlace home = places[t];
            if (home.in < 0) continue;
            raw[j] = load_part<E, NT>(in + home.in + head * x.cache.head, 0, size);
            if (sizeof(E) == 1) scale[j] = x.cache.scale[home.scale + head * x.cache.scale_head];
        }
#pragma unroll
        for (int j = 0; j < kReadAhead; ++j) {
            if (base + j * each + mine >= rows) continue;
            if constexpr (sizeof(E) == 1)
                store_part<T, NT>(out + to[j], 0, size, dev::narrow<T, kPer>(widened<E>(raw[j]) * scale[j]));
            else
                store_part<T, NT>(out + to[j], 0, size, raw[j]);
        }
    }
}

template <typename T, typename E> int read(const ReadArgs &h, hipStream_t s) {
    Read a{};
    a.half[0] = ReadHalf{h.k.out, h.k.out_token, h.k.out_head, scaled_of(h.k_cache), h.k_dim};
    a.half[1] = ReadHalf{h.v.out, h.v.out_token, h.v.out_head, scaled_of(h.v_cache), h.v_dim};
    a.where = h.where;
    a.tokens = h.tokens;
    a.cut = row_cut(std::max(h.k_dim, h.v_dim), kPer);
    a.heads = (int32_t)h.k.heads;
    a.by_heads = fast_div((uint32_t)h.k.heads);
    a.tokens_a_block =
        (int32_t)std::min<int64_t>(kReadTokens, (2 * h.tokens + kReadBlocks - 1) / kReadBlocks);
    const int64_t blocks = (a.tokens + a.tokens_a_block - 1) / a.tokens_a_block;
    // a token's rows are shared by workgroups where there are few tokens
    const int64_t passes =
        (a.tokens_a_block * h.k.heads - 1) / (a.cut.rows_a_wave() * 4 * kReadAhead) + 1;
    const uint32_t shares =
        (uint32_t)std::max<int64_t>(1, std::min(passes, kReadBlocks / (2 * blocks)));
    const bool whole = h.k_dim % kPer == 0 && h.v_dim % kPer == 0;
    // 164 MB of results: 51.5 us streamed, 56 through the caches
    const bool streamed = whole && streams(a.tokens * a.heads * (h.k_dim + h.v_dim), sizeof(T));
    const auto kernel = streamed ? bmmc_cache_read_kernel<T, E, true, true>
                        : whole  ? bmmc_cache_read_kernel<T, E, true, false>
                                 : bmmc_cache_read_kernel<T, E, false, false>;
    return in_launches(blocks, 512 * shares, [&](uint32_t nb, int64_t b0) {
        hipLaunchKernelGGL(kernel, dim3(nb, shares, 2), dim3(256), 0, s, a, b0);
    });
}

template <typename T> int read_t(const ReadArgs &h, hipStream_t s) {
    return h.k_cache.type == BMMC_E4M3 ? read<T, uint8_t>(h, s) : read<T, T>(h, s);
}

}  // namespace

int launch_cache_quantize(const QuantizeArgs &a, hipStream_t s) {
    switch (a.type) {
    case BMMC_F32: return quantize_t<float>(a, s);
    case BMMC_F16: return quantize_t<dev::f16_t>(a, s);
    default: return quantize_t<dev::bf16_t>(a, s);
    }
}

int launch_cache_read(const ReadArgs &a, hipStream_t s) {
    switch (a.type) {
    case BMMC_F32: return read_t<float>(a, s);
    case BMMC_F16: return read_t<dev::f16_t>(a, s);
    default: return read_t<dev::bf16_t>(a, s);
    }
}

}  // namespace bmmc
