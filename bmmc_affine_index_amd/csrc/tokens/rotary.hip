// rotary.hip -- heads turned by their positions, and keys and values put into
// a paged cache (gfx950).
//
// A pair (x, y) turned by the angle p f becomes (x cos - y sin, y cos + x sin).
// The angle of a far position loses its fraction in 32 bits, so the part of a
// turn, p f / 2 pi, is made and reduced to an eighth of a turn in 64 bits;
// what is left goes through the Taylor series in 32.  One pair of cosine and
// sine serves every head of the token: a workgroup makes those of its tokens
// once, in LDS, and then streams the heads past them.
//
// Bound by memory: each element of the heads is read and written once.
#include "device.h"
#include "tokens.h"

namespace bmmc {

namespace {

constexpr int kTurnThreads = 256;
constexpr int kTurnWaves = kTurnThreads / 64;
constexpr int kTurnPairs = 256;  // pairs of LDS a workgroup: BMMC_MAX_HEAD_DIM / 2
constexpr int kTurnTokens = 8;   // most tokens a workgroup takes

struct Turn {
    const void *positions, *freqs;
    const int32_t *axis_of_pair;
    int64_t axis_stride;
    FastDiv by_pairs, by_units, by_heads;
    int32_t positions_are_64, freqs_are_64, axes, pairs;
    int32_t units;  // vectors of pairs a head, at most 64
    int32_t heads_a_wave;
    float scale, sign;
};

struct Heads {
    const void *in;
    void *out;
    int64_t in_batch, in_token, in_head, out_batch, out_token, out_head;
    int32_t heads, in_place;
};

// Cosine and sine, times scale, of a whole number of turns' fraction.
__device__ __forceinline__ float2 cos_sin(double turns) {
    constexpr float kTwoPi = 6.283185307179586f;
    const double eighths = __builtin_rint(turns * 4.0);
    const float x = (float)(turns - eighths * 0.25) * kTwoPi;  // |x| <= pi / 4
    const float x2 = x * x;
    // Taylor: what is left out is below 2e-9 of the sine, 1e-9 of the cosine
    float s = fmaf(x2, 1.0f / 362880.0f, -1.0f / 5040.0f);
    s = fmaf(x2, s, 1.0f / 120.0f);
    s = fmaf(x2, s, -1.0f / 6.0f);
    s = fmaf(x * x2, s, x);
    float c = fmaf(x2, -1.0f / 3628800.0f, 1.0f / 40320.0f);
    c = fmaf(x2, c, -1.0f / 720.0f);
    c = fmaf(x2, c, 1.0f / 24.0f);
    c = fmaf(x2, c, -0.5f);
    c = fmaf(x2, c, 1.0f);
    // whole quarters, modulo 4 (exact: eighths is a whole number)
    const int q = (int)(eighths - 4.0 * __builtin_floor(eighths * 0.25));
    const float a = (q & 1) ? s : c, b = (q & 1) ? c : s;
    return make_float2((q == 1 || q == 2) ? -a : a, q >= 2 ? -b : b);
}

// The workgroup's cosines and sines: cs[t * pairs + i] for its tokens t.
__device__ __forceinline__ void make_turns(const Turn &r, int64_t token0, int tokens,
                                           float2 *cs) {
    constexpr double kInvTwoPi = 0.15915494309189535;
    for (int n = threadIdx.x; n < tokens * r.pairs; n += kTurnThreads) {
        const int t = (int)quotient(r.by_pairs, (uint32_t)n);
        const int i = n - t * r.pairs;
        const int axis = r.axis_of_pair ? r.axis_of_pair[i] : 0;
        const double f = r.freqs_are_64 ? static_cast<const double *>(r.freqs)[i]
                                        : (double)static_cast<const float *>(r.freqs)[i];
        double p = 0.0;
        if (axis >= 0 && axis < r.axes)
            p = (double)position_at(r.positions, r.positions_are_64,
                                    axis * r.axis_stride + token0 + t);
        const float2 u = cos_sin(p * (f * kInvTwoPi));
        cs[n] = make_float2(u.x * r.scale, u.y * r.scale * r.sign);
    }
}

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

// Where the two vectors of pairs [i, i + N) of a head start.
template <int N, bool PAIRED> __device__ __forceinline__ int second_at(int i, int pairs) {
    return PAIRED ? 2 * i + N : pairs + i;
}
template <bool PAIRED> __device__ __forceinline__ int first_at(int i) {
    return PAIRED ? 2 * i : i;
}

// A lane's head and first pair among a wave's heads_a_wave heads.  All
// vectors of a head are one wave's, so that the last, which overlaps the one
// before where the pairs are not whole vectors, is read before that one is
// written even when the head is turned in place.
struct Lane {
    int head, pair;
    bool on;
};
template <int N> __device__ __forceinline__ Lane lane_of(const Turn &r) {
    const int lane = threadIdx.x & 63;
    const int g = (int)quotient(r.by_units, (uint32_t)lane);
    const int j = lane - g * r.units;
    return Lane{g, min(j * N, r.pairs - N), g < r.heads_a_wave};
}

struct TurnHeads {
    Heads x[2];
    int64_t tokens;  // of all batch entries
    FastDiv by_tokens;
    FastDiv by_rest;
    int32_t batch, tokens_a_block;
    int32_t rest, rest_units;  // elements past the pairs, their vectors a head; 0 if all is in place
};

__device__ __forceinline__ void split_token(const FastDiv &by, int batch, int64_t token,
                                            int64_t *b, int64_t *t) {
    *b = batch > 1 ? quotient(by, (uint32_t)token) : 0;
    *t = token - *b * by.d;
}

// Part j of `len` elements that are moved as they are: move(n, at) moves the n
// elements at `at`, a whole vector (the last may overlap the one before; both
// write the same) or, of less than a vector, single elements by one lane.
template <int N> struct Count {
    constexpr operator int() const { return N; }
};
template <typename T, class F> __device__ __forceinline__ void copy_part(int len, int j, F move) {
    constexpr int N = dev::Lanes<T>::N;
    if (len >= N)
        move(Count<N>(), min(j * N, len - N));
    else
        for (int at = 0; at < len; ++at) move(Count<1>(), at);
}
template <typename T> int copy_parts(int len) {
    constexpr int N = dev::Lanes<T>::N;
    return (len + N - 1) / N;
}

template <typename T, int N, bool PAIRED>
__global__ void __launch_bounds__(kTurnThreads)
    bmmc_rotary_kernel(const TurnHeads a, const Turn r, int64_t block0) {
    __shared__ float2 cs[kTurnPairs];
    const int64_t token0 = (block0 + blockIdx.x) * a.tokens_a_block;
    const int tokens = (int)min((int64_t)a.tokens_a_block, a.tokens - token0);
    make_turns(r, token0, tokens, cs);
    __syncthreads();

    const int wave = blockIdx.y * kTurnWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int waves = gridDim.y * kTurnWaves;
    const int heads = (int)r.by_heads.d;
    const Lane l = lane_of<N>(r);
    for (int i0 = wave * r.heads_a_wave; i0 < tokens * heads; i0 += waves * r.heads_a_wave) {
        const int i = i0 + l.head;
        if (!l.on || i >= tokens * heads) continue;
        const int t = (int)quotient(r.by_heads, (uint32_t)i);
        int h = i - t * heads;
        const bool second = h >= a.x[0].heads;
        const Heads &x = a.x[second ? 1 : 0];
        h -= second ? a.x[0].heads : 0;
        int64_t b, tok;
        split_token(a.by_tokens, a.batch, token0 + t, &b, &tok);
        const T *in = static_cast<const T *>(x.in) + b * x.in_batch + tok * x.in_token +
                      h * x.in_head;
        T *out = static_cast<T *>(x.out) + b * x.out_batch + tok * x.out_token + h * x.out_head;
        const int at = first_at<PAIRED>(l.pair), to = second_at<N, PAIRED>(l.pair, r.pairs);
        const dev::Vec<T, N> va = dev::load<T, N>(in + at), vb = dev::load<T, N>(in + to);
        dev::Floats<N> fx, fy;
        turn_vector<T, N, PAIRED>(va, vb, cs + t * r.pairs + l.pair, fx, fy);
        dev::store<T, N>(out + at, dev::narrow<T, N>(fx));
        dev::store<T, N>(out + to, dev::narrow<T, N>(fy));
    }

    // elements past the pairs
    if (!a.rest) return;
    const int n = tokens * heads * a.rest_units;
    for (int i = blockIdx.y * kTurnThreads + threadIdx.x; i < n;
         i += gridDim.y * kTurnThreads) {
        const int th = (int)quotient(a.by_rest, (uint32_t)i);
        const int t = (int)quotient(r.by_heads, (uint32_t)th);
        int h = th - t * heads;
        const bool second = h >= a.x[0].heads;
        const Heads &x = a.x[second ? 1 : 0];
        if (x.in_place) continue;
        h -= second ? a.x[0].heads : 0;
        int64_t b, tok;
        split_token(a.by_tokens, a.batch, token0 + t, &b, &tok);
        const T *in = static_cast<const T *>(x.in) + b * x.in_batch + tok * x.in_token +
                      h * x.in_head + 2 * r.pairs;
        T *out = static_cast<T *>(x.out) + b * x.out_batch + tok * x.out_token + h * x.out_head +
                 2 * r.pairs;
        copy_part<T>(a.rest, i - th * a.rest_units,
                     [&](auto n, int at) { dev::store<T, n>(out + at, dev::load<T, n>(in + at)); });
    }
}

// ---- the paged cache -----------------------------------------------------------

struct Append {
    Heads q, k, v;
    uint8_t *k_cache, *v_cache;
    const float *k_scale, *v_scale;
    int64_t k_page, k_place, k_head, v_page, v_place, v_head;
    PageTable where;
    int64_t tokens;
    FastDiv by_rest, by_v, by_v_heads;
    int32_t rest, rest_units, v_dim, v_units, k_scale_stride, v_scale_stride;
    int32_t tokens_a_block;
};

// Stored 8-bit values: clamped, NaN kept, rounded to nearest, ties to even.
template <int N>
__device__ __forceinline__ void store_e4m3(uint8_t *p, const dev::Floats<N> &x, float scale) {
    constexpr float kMax = 448.0f;
    float y[N];
#pragma unroll
    for (int k = 0; k < N; ++k) {
        const float q = x[k] / scale;
        y[k] = q > kMax ? kMax : q < -kMax ? -kMax : q;
    }
    if constexpr (N == 1) {
        *p = (uint8_t)__builtin_amdgcn_cvt_pk_fp8_f32(y[0], 0.0f, 0, false);
    } else {
        dev::Vec<uint8_t, N> out;
        uint32_t w[N / 4];
#pragma unroll
        for (int k = 0; k < N / 4; ++k) {
            const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * k], y[4 * k + 1], 0, false);
            w[k] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(y[4 * k + 2], y[4 * k + 3], lo, true);
        }
        __builtin_memcpy(&out.v, w, N);
        dev::store<uint8_t, N>(p, out);
    }
}

// N elements to a cache of T or, E4M3, of 8 bits.
template <typename T, int N, bool E4M3>
__device__ __forceinline__ void put(uint8_t *cache, int64_t at, const dev::Floats<N> &x,
                                    const float *scale, int64_t which) {
    if constexpr (E4M3)
        store_e4m3<N>(cache + at, x, scale[which]);
    else
        dev::store<T, N>(reinterpret_cast<T *>(cache) + at, dev::narrow<T, N>(x));
}
template <typename T, int N, bool E4M3>
__device__ __forceinline__ void put_as_is(uint8_t *cache, int64_t at, const dev::Vec<T, N> &x,
                                          const float *scale, int64_t which) {
    if constexpr (E4M3)
        store_e4m3<N>(cache + at, dev::widen<T, N>(x), scale[which]);
    else
        dev::store<T, N>(reinterpret_cast<T *>(cache) + at, x);
}

template <typename T, int N, bool PAIRED, bool E4M3>
__global__ void __launch_bounds__(kTurnThreads)
    bmmc_cache_append_kernel(const Append a, const Turn r, int64_t block0) {
    __shared__ float2 cs[kTurnPairs];
    __shared__ PagePlace places[kTurnTokens];
    const int64_t token0 = (block0 + blockIdx.x) * a.tokens_a_block;
    const int tokens = (int)min((int64_t)a.tokens_a_block, a.tokens - token0);
    if ((int)threadIdx.x < tokens) places[threadIdx.x] = page_place(a.where, token0 + threadIdx.x);
    if (r.pairs) make_turns(r, token0, tokens, cs);
    __syncthreads();

    // A wave's tasks: heads_a_wave heads of q and k to turn, or 64 vectors of v.
    const int wave = blockIdx.y * kTurnWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int waves = gridDim.y * kTurnWaves;
    const int heads = (int)r.by_heads.d;
    const int turns = r.pairs ? (tokens * heads + r.heads_a_wave - 1) / r.heads_a_wave : 0;
    const int vectors = tokens * a.v.heads * a.v_units;
    const int copies = (vectors + 63) / 64;
    const Lane l = r.pairs ? lane_of<N>(r) : Lane{0, 0, false};
    for (int task = wave; task < turns + copies; task += waves) {
        if (task < turns) {
            const int i = task * r.heads_a_wave + l.head;
            if (!l.on || i >= tokens * heads) continue;
            const int t = (int)quotient(r.by_heads, (uint32_t)i);
            const int h = i - t * heads;
            const int at = first_at<PAIRED>(l.pair), to = second_at<N, PAIRED>(l.pair, r.pairs);
            const float2 *u = cs + t * r.pairs + l.pair;
            const int64_t tok = token0 + t;
            dev::Floats<N> x, y;
            if (h < a.q.heads) {
                const T *in = static_cast<const T *>(a.q.in) + tok * a.q.in_token + h * a.q.in_head;
                T *out = static_cast<T *>(a.q.out) + tok * a.q.out_token + h * a.q.out_head;
                turn_vector<T, N, PAIRED>(dev::load<T, N>(in + at), dev::load<T, N>(in + to), u,
                                          x, y);
                dev::store<T, N>(out + at, dev::narrow<T, N>(x));
                dev::store<T, N>(out + to, dev::narrow<T, N>(y));
            } else {
                const int kh = h - a.q.heads;
                const PagePlace p = places[t];
                if (p.page < 0) continue;
                const T *in =
                    static_cast<const T *>(a.k.in) + tok * a.k.in_token + kh * a.k.in_head;
                const int64_t base = p.page * a.k_page + p.place * a.k_place + kh * a.k_head;
                turn_vector<T, N, PAIRED>(dev::load<T, N>(in + at), dev::load<T, N>(in + to), u,
                                          x, y);
                put<T, N, E4M3>(a.k_cache, base + at, x, a.k_scale, kh * a.k_scale_stride);
                put<T, N, E4M3>(a.k_cache, base + to, y, a.k_scale, kh * a.k_scale_stride);
            }
        } else {
            const int i = (task - turns) * 64 + (threadIdx.x & 63);
            if (i >= vectors) continue;
            const int th = (int)quotient(a.by_v, (uint32_t)i);
            const int t = (int)quotient(a.by_v_heads, (uint32_t)th);
            const int h = th - t * a.v.heads;
            const PagePlace p = places[t];
            if (p.page < 0) continue;
            const T *in = static_cast<const T *>(a.v.in) + (token0 + t) * a.v.in_token +
                          h * a.v.in_head;
            const int64_t base = p.page * a.v_page + p.place * a.v_place + h * a.v_head;
            copy_part<T>(a.v_dim, i - th * a.v_units, [&](auto n, int at) {
                put_as_is<T, n, E4M3>(a.v_cache, base + at, dev::load<T, n>(in + at), a.v_scale,
                                      h * a.v_scale_stride);
            });
        }
    }

    // elements of q and k past the pairs
    if (!a.rest) return;
    const int n = tokens * heads * a.rest_units;
    for (int i = blockIdx.y * kTurnThreads + threadIdx.x; i < n;
         i += gridDim.y * kTurnThreads) {
        const int th = (int)quotient(a.by_rest, (uint32_t)i);
        const int j = i - th * a.rest_units;
        const int t = (int)quotient(r.by_heads, (uint32_t)th);
        const int h = th - t * heads;
        const int64_t tok = token0 + t;
        if (h < a.q.heads) {
            if (a.q.in_place) continue;
            const T *in = static_cast<const T *>(a.q.in) + tok * a.q.in_token +
                          h * a.q.in_head + 2 * r.pairs;
            T *out = static_cast<T *>(a.q.out) + tok * a.q.out_token + h * a.q.out_head +
                     2 * r.pairs;
            copy_part<T>(a.rest, j, [&](auto n, int at) {
                dev::store<T, n>(out + at, dev::load<T, n>(in + at));
            });
        } else {
            const int kh = h - a.q.heads;
            const PagePlace p = places[t];
            if (p.page < 0) continue;
            const T *in = static_cast<const T *>(a.k.in) + tok * a.k.in_token +
                          kh * a.k.in_head + 2 * r.pairs;
            const int64_t base =
                p.page * a.k_page + p.place * a.k_place + kh * a.k_head + 2 * r.pairs;
            copy_part<T>(a.rest, j, [&](auto n, int at) {
                put_as_is<T, n, E4M3>(a.k_cache, base + at, dev::load<T, n>(in + at), a.k_scale,
                                      kh * a.k_scale_stride);
            });
        }
    }
}

// ---- launches --------------------------------------------------------------------

template <int N> Turn turn_of(const bmmc_rotation &x, int heads) {
    Turn r{};
    r.by_heads = fast_div((uint32_t)(heads > 0 ? heads : 1));
    if (x.pairs == 0) {
        r.by_pairs = r.by_units = fast_div(1);
        return r;
    }
    r.positions = x.positions;
    r.freqs = x.freqs;
    r.axis_of_pair = x.axis_of_pair;
    r.axis_stride = x.axis_stride;
    r.positions_are_64 = x.position_type == BMMC_I64;
    r.freqs_are_64 = x.freqs_are_64;
    r.axes = x.axes;
    r.pairs = x.pairs;
    r.units = (x.pairs + N - 1) / N;
    r.heads_a_wave = 64 / r.units;
    r.by_pairs = fast_div((uint32_t)x.pairs);
    r.by_units = fast_div((uint32_t)r.units);
    r.scale = x.scale;
    r.sign = x.inverse ? -1.0f : 1.0f;
    return r;
}

Heads heads_of(const bmmc_heads &x) {
    return Heads{x.in, x.out, x.in_batch, x.in_token, x.in_head, x.out_batch, x.out_token,
                 x.out_head, (int32_t)x.heads,
                 x.in == x.out};
}

// Tokens a workgroup takes, and workgroups that share a block's tasks: about
// as many tokens as LDS holds where that leaves at least four workgroups for
// each of the 256 compute units, else one token, its heads over several
// workgroups up to that many.
constexpr int64_t kTurnBlocks = 1024;

int tokens_a_block(int64_t tokens, int pairs) {
    int n = pairs ? kTurnPairs / pairs : 4;
    n = n > kTurnTokens ? kTurnTokens : n < 1 ? 1 : n;
    return tokens / n >= kTurnBlocks ? n : 1;
}

uint32_t shares(int64_t blocks, int64_t tasks) {
    int64_t most = (tasks + kTurnWaves - 1) / kTurnWaves, want = kTurnBlocks / blocks;
    if (most > want) most = want;
    return most < 1 ? 1 : (uint32_t)most;
}

template <typename T, int N, bool PAIRED>
int rotary_n(const HeadsArgs &h, const bmmc_rotation &x, hipStream_t s) {
    TurnHeads a{};
    int64_t heads = 0;
    bool place = true;
    for (int i = 0; i < h.count; ++i) {
        a.x[i] = heads_of(h.x[i]);
        heads += h.x[i].heads;
        place &= a.x[i].in_place != 0;
    }
    a.tokens = h.batch * h.tokens;
    a.batch = (int32_t)h.batch;
    a.by_tokens = fast_div((uint32_t)h.tokens);
    a.rest = place ? 0 : h.head_dim - 2 * x.pairs;
    a.rest_units = copy_parts<T>(a.rest);
    a.by_rest = fast_div((uint32_t)(a.rest ? a.rest_units : 1));
    a.tokens_a_block = tokens_a_block(a.tokens, x.pairs);
    const Turn r = turn_of<N>(x, (int)heads);
    const int64_t blocks = (a.tokens + a.tokens_a_block - 1) / a.tokens_a_block;
    const int64_t tasks = (a.tokens_a_block * heads + r.heads_a_wave - 1) / r.heads_a_wave;
    return in_launches(blocks, kTurnThreads, [&](uint32_t nb, int64_t b0) {
        hipLaunchKernelGGL((bmmc_rotary_kernel<T, N, PAIRED>), dim3(nb, shares(blocks, tasks)),
                           dim3(kTurnThreads), 0, s, a, r, b0);
    });
}

template <typename T, int N, bool PAIRED, bool E4M3>
int append_n(const AppendArgs &h, hipStream_t s) {
    Append a{};
    a.q = heads_of(h.q);
    a.k = heads_of(h.k);
    a.v = heads_of(h.v);
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
    a.v_dim = h.v_dim;
    a.v_units = copy_parts<T>(h.v_dim);
    a.rest = h.k_dim - 2 * h.rotation.pairs;
    a.rest_units = copy_parts<T>(a.rest);
    a.by_rest = fast_div((uint32_t)(a.rest ? a.rest_units : 1));
    a.by_v = fast_div((uint32_t)a.v_units);
    a.by_v_heads = fast_div((uint32_t)h.v.heads);
    a.tokens_a_block = tokens_a_block(a.tokens, h.rotation.pairs);
    const int64_t heads = h.q.heads + h.k.heads;
    const Turn r = turn_of<N>(h.rotation, (int)heads);
    const int64_t blocks = (a.tokens + a.tokens_a_block - 1) / a.tokens_a_block;
    const int64_t turns =
        r.pairs ? (a.tokens_a_block * heads + r.heads_a_wave - 1) / r.heads_a_wave : 0;
    const int64_t copies = ((int64_t)a.tokens_a_block * h.v.heads * a.v_units + 63) / 64;
    return in_launches(blocks, kTurnThreads, [&](uint32_t nb, int64_t b0) {
        hipLaunchKernelGGL((bmmc_cache_append_kernel<T, N, PAIRED, E4M3>),
                           dim3(nb, shares(blocks, turns + copies)), dim3(kTurnThreads), 0, s, a,
                           r, b0);
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
