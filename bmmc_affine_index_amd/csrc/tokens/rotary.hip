// rotary.hip -- heads turned by their positions, and keys and values put into
// a paged cache (gfx950).
//
// A pair (x, y) turned by the angle p f becomes (x cos - y sin, y cos + x sin).
// The angle of a far position loses its fraction in 32 bits, so the part of a
// turn, p f / 2 pi, is made and reduced to an eighth of a turn in 64 bits;
// what is left goes through the Taylor series in 32.  One pair of cosine and
// sine serves every head of the token: a workgroup makes those of its tokens
// once, in LDS, and then streams the heads past them.  Its first heads are on
// their way from memory while it does.
//
// Bound by memory: each element of the heads is read and written once.  A
// workgroup takes as few tokens as keep its waves busy, usually one: what runs
// at the same time then lies close together in memory (plain copies of 40 heads
// of 256 bytes a token: 6.2 TB/s by workgroups of one token, 5.9 of two, 5.8 of
// four, 5.4 of eight).
#include "turns.h"

namespace bmmc {

namespace {

// Heads to turn, and what of them is only copied.  A wave's task is
// heads_a_wave heads of one token, or 64 vectors of what is copied of them.
struct Heads {
    const void *in;
    void *out;
    int64_t in_batch, in_token, in_head, out_batch, out_token, out_head;
    int32_t heads;
    int32_t turns, copies;  // tasks a token
};

// Vector j of a head's pairs, turned: the first and second elements' N values
// from a and b (interleaved: the 2N elements in order are a's, then b's).
template <typename T, int N, bool PAIRED>
__device__ __forceinline__ void turn_vector(const dev::Vec<T, N> &a, const dev::Vec<T, N> &b,
                                            const float2 *cs, dev::Floats<N> &x,
                                            dev::Floats<N> &y) {
    const dev::Floats<N> fa = dev::widen<T, N>(a), fb = dev::widen<T, N>(b);
    if constexpr (!PAIRED) {
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const float2 u = cs[k];
            x[k] = fa[k] * u.x - fb[k] * u.y;
            y[k] = fb[k] * u.x + fa[k] * u.y;
        }
    } else if constexpr (N == 1) {
        const float2 u = cs[0];
        x[0] = fa[0] * u.x - fb[0] * u.y;
        y[0] = fb[0] * u.x + fa[0] * u.y;
    } else {
#pragma unroll
        for (int k = 0; k < N / 2; ++k) {
            const float2 u = cs[k], w = cs[N / 2 + k];
            x[2 * k] = fa[2 * k] * u.x - fa[2 * k + 1] * u.y;
            x[2 * k + 1] = fa[2 * k + 1] * u.x + fa[2 * k] * u.y;
            y[2 * k] = fb[2 * k] * w.x - fb[2 * k + 1] * w.y;
            y[2 * k + 1] = fb[2 * k + 1] * w.x + fb[2 * k] * w.y;
        }
    }
}

// A lane's head and first pair among a wave's heads_a_wave heads.  All
// vectors of a head are one wave's, so that the last, which overlaps the one
// before where the pairs are not whole vectors, is read before that one is
// written even when the head is turned in place.
struct Lane {
    int head, at;  // at: its first vector; the second is `gap` elements on
    bool on;
};
template <int N, bool PAIRED> __device__ __forceinline__ Lane lane_of(const Turn &r) {
    const int lane = threadIdx.x & 63;
    const int g = (int)quotient(r.by_units, (uint32_t)lane);
    const int pair = min((lane - g * r.units) * N, r.pairs - N);
    return Lane{g, PAIRED ? 2 * pair : pair, g < r.heads_a_wave};
}
template <int N, bool PAIRED> __device__ __forceinline__ int gap_of(const Turn &r) {
    return PAIRED ? N : r.pairs;
}
template <bool PAIRED> __device__ __forceinline__ int pair_of(const Lane &l) {
    return PAIRED ? l.at / 2 : l.at;
}

// `len` elements of each head that are moved as they are, in whole vectors
// (the last may overlap the one before; both write the same) or, of less than
// a vector, single elements by one lane.
struct Part {
    FastDiv by_units;
    int32_t from, len, units;  // of a head; units: vectors
};
template <typename T> Part part_of(int from, int len) {
    constexpr int N = dev::Lanes<T>::N;
    const int units = (len + N - 1) / N;
    return Part{fast_div((uint32_t)(units ? units : 1)), from, len, units};
}
int copies_of(const Part &p, int64_t heads) { return (int)((heads * p.units + 63) / 64); }

// Task `task` of a part of one token's heads: put(h, element, vector) moves
// one vector or element of head h.
template <int N> struct Count {
    constexpr operator int() const { return N; }
};
template <typename T, class F>
__device__ __forceinline__ void copy_task(const Part &p, int heads, int task, const T *in,
                                          int64_t in_head, F put) {
    constexpr int N = dev::Lanes<T>::N;
    const int u = task * 64 + (threadIdx.x & 63);
    if (u >= heads * p.units) return;
    const int h = (int)quotient(p.by_units, (uint32_t)u);
    in += h * in_head;
    if (p.len >= N) {
        const int at = p.from + min((u - h * p.units) * N, p.len - N);
        put(h, at, dev::load<T, N>(in + at));
    } else {
        for (int at = p.from; at < p.from + p.len; ++at) put(h, at, dev::load<T, 1>(in + at));
    }
}

struct TurnHeads {
    Heads x[2];
    Part rest;
    int64_t tokens;  // of all batch entries
    FastDiv by_tokens, by_tasks;
    int32_t batch, tokens_a_block, stream;
};

// This wave's first task and the waves of the workgroups that share its tokens.
struct Waves {
    int first, count;
};
__device__ __forceinline__ Waves waves_of() {
    const int n = blockDim.x >> 6;
    return Waves{(int)(blockIdx.y * n + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6)),
                 (int)(gridDim.y * n)};
}

// A task's numbers are the same in all lanes, and so are its token's place in
// memory and in the cache: they are made in scalar registers, and a lane adds
// its own offset.
template <typename T, int N, bool PAIRED>
__global__ void __launch_bounds__(kTurnThreads)
    bmmc_rotary_kernel(const TurnHeads a, const Turn r, int64_t block0) {
    __shared__ float2 cs[kTurnPairs];
    const int64_t token0 = (block0 + blockIdx.x) * a.tokens_a_block;
    const int tokens = (int)min((int64_t)a.tokens_a_block, a.tokens - token0);
    const int per = (int)a.by_tasks.d, tasks = tokens * per;
    const int turns0 = a.x[0].turns, turns = turns0 + a.x[1].turns;
    const Waves waves = waves_of();
    const Lane l = lane_of<N, PAIRED>(r);
    const int gap = gap_of<N, PAIRED>(r);
    const int64_t lane_in[2] = {l.head * a.x[0].in_head + l.at, l.head * a.x[1].in_head + l.at};
    const int64_t lane_out[2] = {l.head * a.x[0].out_head + l.at, l.head * a.x[1].out_head + l.at};

    struct Task {
        int token, number;  // of the workgroup's tokens, of its token's tasks
        int64_t in_batch, in_token;
    };
    const auto locate = [&](int task) {
        const int t = (int)quotient(a.by_tasks, (uint32_t)task);
        const int64_t tok = token0 + t;
        const int64_t b = a.batch > 1 ? quotient(a.by_tokens, (uint32_t)tok) : 0;
        return Task{t, task - t * per, b, tok - b * a.by_tokens.d};
    };
    dev::Vec<T, N> va, vb;
    const auto fetch = [&](int task) {
        const Task k = locate(task);
        if (k.number >= turns) return;
        const bool second = k.number >= turns0;
        const Heads &x = a.x[second];
        const int head = (k.number - (second ? turns0 : 0)) * r.heads_a_wave;
        if (!l.on || head + l.head >= x.heads) return;
        const T *in = static_cast<const T *>(x.in) + k.in_batch * x.in_batch +
                      k.in_token * x.in_token + head * x.in_head + lane_in[second];
        dev::by_hint(a.stream, [&](auto nt) {
            va = dev::load<T, N, nt.value>(in);
            vb = dev::load<T, N, nt.value>(in + gap);
        });
    };
    make_turns(r, token0, tokens, cs, [&] {
        if (waves.first < tasks) fetch(waves.first);
    });
    __syncthreads();
    for (int task = waves.first; task < tasks; task += waves.count) {
        const Task k = locate(task);
        const dev::Vec<T, N> a0 = va, b0 = vb;
        // the next heads are others: what is read here is not written below
        if (task + waves.count < tasks) fetch(task + waves.count);
        if (k.number < turns) {
            const bool second = k.number >= turns0;
            const Heads &x = a.x[second];
            const int head = (k.number - (second ? turns0 : 0)) * r.heads_a_wave;
            if (!l.on || head + l.head >= x.heads) continue;
            T *out = static_cast<T *>(x.out) + k.in_batch * x.out_batch +
                     k.in_token * x.out_token + head * x.out_head + lane_out[second];
            dev::Floats<N> fx, fy;
            turn_vector<T, N, PAIRED>(a0, b0, cs + k.token * r.pairs + pair_of<PAIRED>(l), fx, fy);
            dev::store<T, N>(out, dev::narrow<T, N>(fx));
            dev::store<T, N>(out + gap, dev::narrow<T, N>(fy));
        } else {
            const int c = k.number - turns;
            const bool second = c >= a.x[0].copies;
            const Heads &x = a.x[second];
            T *out = static_cast<T *>(x.out) + k.in_batch * x.out_batch + k.in_token * x.out_token;
            copy_task<T>(a.rest, x.heads, c - (second ? a.x[0].copies : 0),
                         static_cast<const T *>(x.in) + k.in_batch * x.in_batch +
                             k.in_token * x.in_token,
                         x.in_head, [&](int h, int at, auto v) {
                             dev::store(out + h * x.out_head + at, v);
                         });
        }
    }
}

// ---- the paged cache -----------------------------------------------------------

struct Append {
    Heads q, k, v;
    uint8_t *k_cache, *v_cache;
    const float *k_scale, *v_scale;
    int64_t k_page, k_place, k_head, v_page, v_place, v_head;
    PageTable where;
    Part rest, values;
    int64_t tokens;
    FastDiv by_tasks;
    int32_t k_scale_stride, v_scale_stride, tokens_a_block, stream;
};

// N elements to a cache of T or, E4M3, of 8 bits.
template <typename T, int N, bool E4M3>
__device__ __forceinline__ void put(uint8_t *cache, int64_t at, const dev::Floats<N> &x,
                                    const float *scale, int64_t which) {
    if constexpr (E4M3)
        store_e4m3<N>(cache + at, x, scale[which]);
    else
        dev::store<T, N>(reinterpret_cast<T *>(cache) + at, dev::narrow<T, N>(x));
}
template <bool E4M3, typename T, int N>
__device__ __forceinline__ void put_as_is(uint8_t *cache, int64_t at, const dev::Vec<T, N> &x,
                                          const float *scale, int64_t which) {
    if constexpr (E4M3)
        store_e4m3<N>(cache + at, dev::widen<T, N>(x), scale[which]);
    else
        dev::store<T, N>(reinterpret_cast<T *>(cache) + at, x);
}

// A token's tasks: q's and k's heads to turn, what of q, of k and of v is copied.
template <typename T, int N, bool PAIRED, bool E4M3>
__global__ void __launch_bounds__(kTurnThreads)
    bmmc_cache_append_kernel(const Append a, const Turn r, int64_t block0) {
    __shared__ float2 cs[kTurnPairs];
    __shared__ PagePlace places[kTurnTokens];
    constexpr int VN = dev::Lanes<T>::N;
    const int64_t token0 = (block0 + blockIdx.x) * a.tokens_a_block;
    const int tokens = (int)min((int64_t)a.tokens_a_block, a.tokens - token0);
    const int per = (int)a.by_tasks.d, tasks = tokens * per;
    const int turns = a.q.turns + a.k.turns, values = turns + a.q.copies + a.k.copies;
    const Waves waves = waves_of();
    const Lane l = r.pairs ? lane_of<N, PAIRED>(r) : Lane{0, 0, false};
    const int gap = gap_of<N, PAIRED>(r);
    const int64_t q_in = l.head * a.q.in_head + l.at, q_out = l.head * a.q.out_head + l.at;
    const int64_t k_in = l.head * a.k.in_head + l.at, k_out = l.head * a.k_head + l.at;

    const auto source = [](const Heads &x, int64_t token) {
        return static_cast<const T *>(x.in) + token * x.in_token;
    };
    // This lane's vector of v in task `number`.
    struct Value {
        int head, at;
        bool on;
    };
    const auto value = [&](int number) {
        const int u = (number - values) * 64 + (threadIdx.x & 63);
        const int h = (int)quotient(a.values.by_units, (uint32_t)u);
        return Value{h, min((u - h * a.values.units) * VN, a.values.len - VN),
                     u < a.v.heads * a.values.units};
    };
    const bool whole = a.values.len >= VN;
    dev::Vec<T, N> va, vb;  // a turn's
    dev::Vec<T, VN> vc;     // of v
    const auto fetch = [&](int task) {
        const int t = (int)quotient(a.by_tasks, (uint32_t)task), number = task - t * per;
        if (number >= values && whole) {
            const Value f = value(number);
            if (f.on)
                dev::by_hint(a.stream, [&](auto nt) {
                    vc = dev::load<T, VN, nt.value>(source(a.v, token0 + t) +
                                                    f.head * a.v.in_head + f.at);
                });
        }
        if (number >= turns) return;
        const bool key = number >= a.q.turns;
        const Heads &x = key ? a.k : a.q;
        const int head = (number - (key ? a.q.turns : 0)) * r.heads_a_wave;
        if (!l.on || head + l.head >= x.heads) return;
        const T *in = source(x, token0 + t) + head * x.in_head + (key ? k_in : q_in);
        dev::by_hint(a.stream, [&](auto nt) {
            va = dev::load<T, N, nt.value>(in);
            vb = dev::load<T, N, nt.value>(in + gap);
        });
    };
    const auto copy = [&](int64_t token, const PagePlace &home, int number) {
        if (number < a.q.copies) {
            T *out = static_cast<T *>(a.q.out) + token * a.q.out_token;
            copy_task<T>(a.rest, a.q.heads, number, source(a.q, token), a.q.in_head,
                         [&](int h, int at, auto v) { dev::store(out + h * a.q.out_head + at, v); });
            return;
        }
        number -= a.q.copies;
        if (home.page < 0) return;
        const bool key = number < a.k.copies;
        const int64_t base = key ? home.page * a.k_page + home.place * a.k_place
                                 : home.page * a.v_page + home.place * a.v_place;
        const Heads &x = key ? a.k : a.v;
        copy_task<T>(key ? a.rest : a.values, x.heads, number - (key ? 0 : a.k.copies),
                     source(x, token), x.in_head, [&](int h, int at, auto v) {
                         put_as_is<E4M3>(key ? a.k_cache : a.v_cache,
                                         base + h * (key ? a.k_head : a.v_head) + at, v,
                                         key ? a.k_scale : a.v_scale,
                                         h * (key ? a.k_scale_stride : a.v_scale_stride));
                     });
    };
    // the last wave looks the places up while the first make cosines
    const int looker = (int)threadIdx.x - ((int)blockDim.x - 64);
    if (looker >= 0 && looker < tokens) places[looker] = page_place(a.where, token0 + looker);
    make_turns(r, token0, r.pairs ? tokens : 0, cs, [&] {
        if (waves.first < tasks) fetch(waves.first);
    });
    __syncthreads();
    for (int task = waves.first; task < tasks; task += waves.count) {
        const int t = (int)quotient(a.by_tasks, (uint32_t)task), number = task - t * per;
        const int64_t token = token0 + t;
        const dev::Vec<T, N> a0 = va, b0 = vb;
        const dev::Vec<T, VN> c0 = vc;
        // the next heads are others: what is read here is not written below
        if (task + waves.count < tasks) fetch(task + waves.count);
        const PagePlace home = places[t];
        if (number >= values && whole) {
            const Value f = value(number);
            if (home.page < 0 || !f.on) continue;
            put_as_is<E4M3>(a.v_cache,
                            home.page * a.v_page + home.place * a.v_place + f.head * a.v_head + f.at,
                            c0, a.v_scale, f.head * a.v_scale_stride);
            continue;
        }
        if (number >= turns) {
            copy(token, home, number - turns);
            continue;
        }
        const bool key = number >= a.q.turns;
        const int head = (number - (key ? a.q.turns : 0)) * r.heads_a_wave;
        const bool on = l.on && head + l.head < (key ? a.k : a.q).heads;
        dev::Floats<N> x, y;
        turn_vector<T, N, PAIRED>(a0, b0, cs + t * r.pairs + pair_of<PAIRED>(l), x, y);
        if (!key) {
            T *out = static_cast<T *>(a.q.out) + token * a.q.out_token + head * a.q.out_head + q_out;
            if (!on) continue;
            dev::store<T, N>(out, dev::narrow<T, N>(x));
            dev::store<T, N>(out + gap, dev::narrow<T, N>(y));
        } else {
            if (home.page < 0 || !on) continue;
            const int64_t at = home.page * a.k_page + home.place * a.k_place + head * a.k_head + k_out;
            const int64_t which = (head + l.head) * a.k_scale_stride;
            put<T, N, E4M3>(a.k_cache, at, x, a.k_scale, which);
            put<T, N, E4M3>(a.k_cache, at + gap, y, a.k_scale, which);
        }
    }
}

// ---- launches --------------------------------------------------------------------

// `rest`: what past the pairs is copied, unless the heads stay where they are.
Heads heads_of(const bmmc_heads &x, const Turn &r, const Part &rest) {
    const int32_t heads = (int32_t)x.heads;
    return Heads{x.in, x.out, x.in_batch, x.in_token, x.in_head, x.out_batch, x.out_token,
                 x.out_head, heads,
                 r.pairs ? (heads + r.heads_a_wave - 1) / r.heads_a_wave : 0,
                 x.in == x.out ? 0 : copies_of(rest, heads)};
}

template <typename T, int N, bool PAIRED>
int rotary_n(const HeadsArgs &h, const bmmc_rotation &x, hipStream_t s) {
    const Turn r = turn_of<N>(x);
    TurnHeads a{};
    a.rest = part_of<T>(2 * x.pairs, h.head_dim - 2 * x.pairs);
    int64_t tasks = 0;
    for (int i = 0; i < h.count; ++i) {
        a.x[i] = heads_of(h.x[i], r, a.rest);
        tasks += a.x[i].turns + a.x[i].copies;
    }
    a.tokens = h.batch * h.tokens;
    a.batch = (int32_t)h.batch;
    a.by_tokens = fast_div((uint32_t)h.tokens);
    a.by_tasks = fast_div((uint32_t)tasks);
    const TurnCut cut = turn_cut(a.tokens, x.pairs, tasks);
    a.tokens_a_block = cut.tokens_a_block;
    a.stream = streams(a.tokens * (a.x[0].heads + a.x[1].heads) * h.head_dim, sizeof(T));
    return in_launches(cut.blocks, kTurnThreads, [&](uint32_t nb, int64_t b0) {
        hipLaunchKernelGGL((bmmc_rotary_kernel<T, N, PAIRED>), dim3(nb, cut.shares),
                           dim3(64 * cut.waves), 0, s, a, r, b0);
    });
}

template <typename T, int N, bool PAIRED, bool E4M3>
int append_n(const AppendArgs &h, hipStream_t s) {
    const Turn r = turn_of<N>(h.rotation);
    Append a{};
    a.rest = part_of<T>(2 * r.pairs, h.k_dim - 2 * r.pairs);
    a.values = part_of<T>(0, h.v_dim);
    if (h.q.heads) a.q = heads_of(h.q, r, a.rest);
    a.k = heads_of(h.k, r, a.rest);
    a.v = heads_of(h.v, Turn{}, a.values);
    a.k.copies = copies_of(a.rest, h.k.heads);  // k and v have no out of their own
    a.v.copies = copies_of(a.values, h.v.heads);
    a.k_cache = static_cast<uint8_t *>(h.k_cache.data);
    a.v_cache = static_cast<uint8_t *>(h.v_cache.data);
    a.k_scale = h.k_cache.scale;
    a.v_scale = h.v_cache.scale;
    a.k_page = h.k_cache.page_stride;
    a.k_place = h.k_cache.place_stride;
    a.k_head = h.k_cache.head_stride;
    a.v_page = h.v_cache.page_stride;
    a.v_place = h.v_cache.place_stride;
    a.v_head = h.v_cache.head_stride;
    a.k_scale_stride = h.k_cache.scale_stride;
    a.v_scale_stride = h.v_cache.scale_stride;
    a.where = h.where;
    a.tokens = h.tokens;
    const int64_t tasks = (int64_t)a.q.turns + a.q.copies + a.k.turns + a.k.copies + a.v.copies;
    a.by_tasks = fast_div((uint32_t)tasks);
    const TurnCut cut = turn_cut(a.tokens, r.pairs, tasks);
    a.tokens_a_block = cut.tokens_a_block;
    a.stream = streams(a.tokens * ((a.q.heads + a.k.heads) * (int64_t)h.k_dim +
                                   a.v.heads * (int64_t)h.v_dim), sizeof(T));
    return in_launches(cut.blocks, kTurnThreads, [&](uint32_t nb, int64_t b0) {
        hipLaunchKernelGGL((bmmc_cache_append_kernel<T, N, PAIRED, E4M3>), dim3(nb, cut.shares),
                           dim3(64 * cut.waves), 0, s, a, r, b0);
    });
}

template <typename T> int rotary_t(const HeadsArgs &h, const bmmc_rotation &x, hipStream_t s) {
    constexpr int N = dev::Lanes<T>::N;
    if (x.pairs < N)
        return x.interleaved ? rotary_n<T, 1, true>(h, x, s) : rotary_n<T, 1, false>(h, x, s);
    return x.interleaved ? rotary_n<T, N, true>(h, x, s) : rotary_n<T, N, false>(h, x, s);
}

template <typename T, int N> int append_t(const AppendArgs &h, hipStream_t s) {
    const bool narrow = h.k_cache.type == BMMC_E4M3;
    if (h.rotation.interleaved)
        return narrow ? append_n<T, N, true, true>(h, s) : append_n<T, N, true, false>(h, s);
    return narrow ? append_n<T, N, false, true>(h, s) : append_n<T, N, false, false>(h, s);
}

template <typename T> int append_w(const AppendArgs &h, hipStream_t s) {
    constexpr int N = dev::Lanes<T>::N;
    return h.rotation.pairs && h.rotation.pairs < N ? append_t<T, 1>(h, s) : append_t<T, N>(h, s);
}

}  // namespace

int launch_rotary(const HeadsArgs &a, const bmmc_rotation &r, hipStream_t s) {
    switch (a.type) {
    case BMMC_F32: return rotary_t<float>(a, r, s);
    case BMMC_F16: return rotary_t<dev::f16_t>(a, r, s);
    default: return rotary_t<dev::bf16_t>(a, r, s);
    }
}

int launch_cache_append(const AppendArgs &a, hipStream_t s) {
    switch (a.type) {
    case BMMC_F32: return append_w<float>(a, s);
    case BMMC_F16: return append_w<dev::f16_t>(a, s);
    default: return append_w<dev::bf16_t>(a, s);
    }
}

}  // namespace bmmc
