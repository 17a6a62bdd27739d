// turns.h -- what the kernels that turn heads share: the turns of a workgroup's
// tokens, 8-bit values, and how tokens are cut into workgroups (gfx950).
#pragma once

#include <algorithm>

#include "device.h"
#include "tokens.h"

namespace bmmc {

namespace {

constexpr int kTurnWaves = 4;  // most waves a workgroup
constexpr int kTurnThreads = 64 * kTurnWaves;
constexpr int kTurnTokens = 4;   // most tokens a workgroup
constexpr int kTurnPairs = 256;  // pairs of LDS a workgroup: BMMC_MAX_HEAD_DIM / 2

struct Turn {
    const void *positions, *freqs;
    const int32_t *axis_of_pair;
    int64_t axis_stride;
    FastDiv by_pairs, by_units;
    int32_t positions_are_64, freqs_are_64, axes, pairs;
    int32_t units;         // vectors of pairs a head, at most 64
    int32_t heads_a_wave;  // 64 / units
    float scale, sign;
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
// `meanwhile` runs once, in every thread, after the first loads for them have
// been issued.
template <class F>
__device__ __forceinline__ void make_turns(const Turn &r, int64_t token0, int tokens, float2 *cs,
                                           F meanwhile) {
    constexpr double kInvTwoPi = 0.15915494309189535;
    bool first = true;
    for (int n = threadIdx.x; first || n < tokens * r.pairs; n += blockDim.x) {
        const bool on = n < tokens * r.pairs;
        const int t = (int)quotient(r.by_pairs, (uint32_t)n);
        const int i = n - t * r.pairs;
        double p = 0.0, f = 0.0;
        if (on) {
            const int axis = r.axis_of_pair ? r.axis_of_pair[i] : 0;
            f = r.freqs_are_64 ? static_cast<const double *>(r.freqs)[i]
                               : (double)static_cast<const float *>(r.freqs)[i];
            if (axis >= 0 && axis < r.axes)
                p = (double)position_at(r.positions, r.positions_are_64,
                                        axis * r.axis_stride + token0 + t);
        }
        if (first) meanwhile();
        first = false;
        if (!on) break;
        const float2 u = cos_sin(p * (f * kInvTwoPi));
        cs[n] = make_float2(u.x * r.scale, u.y * r.scale * r.sign);
    }
}

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

// ---- launches --------------------------------------------------------------------

template <int N> Turn turn_of(const bmmc_rotation &x) {
    Turn r{};
    r.by_pairs = r.by_units = fast_div(1);
    if (x.pairs == 0) return r;
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

// How the tokens are cut: a workgroup takes one token, or as many as its four
// waves have one task each for and LDS holds cosines for, if that leaves four
// workgroups for each of the 256 compute units.  32768 tokens of 40 heads of 256
// bytes (5 tasks): 109 us with one token and four waves, 113 with two tokens,
// 117 with four; 133 with eight waves, which wait for one another's cosines.
// Few tokens have their tasks spread over several workgroups, up to as many (with
// twice as many, 1024 tokens of 40 heads and 8 of values take 8.2 us, not 7.0, and
// 512 tokens 4.9, not 4.8).
constexpr int64_t kTurnBlocks = 1024;

struct TurnCut {
    int tokens_a_block, waves;
    int64_t blocks;
    uint32_t shares;
};

TurnCut turn_cut(int64_t tokens, int pairs, int64_t tasks) {
    int64_t n = std::min<int64_t>(kTurnTokens, kTurnWaves / tasks);
    if (pairs) n = std::min<int64_t>(n, kTurnPairs / pairs);
    if (n < 1 || tokens / n < kTurnBlocks) n = 1;
    TurnCut c;
    c.tokens_a_block = (int)n;
    c.waves = (int)std::min<int64_t>(n * tasks, kTurnWaves);
    c.blocks = (tokens + n - 1) / n;
    const int64_t most = (n * tasks + c.waves - 1) / c.waves, want = kTurnBlocks / c.blocks;
    c.shares = (uint32_t)std::max<int64_t>(std::min(most, want), 1);
    return c;
}

// Heads are a projection's output just written, and are read through the caches
// where they and what becomes of them fit, streamed beyond (98 MB: 17.7 us, 23.2
// streamed; 168 to 500 MB: the same within 3%; 672 MB: 115 us, 111 streamed).
constexpr int64_t kTurnCached = int64_t(128) << 20;

bool streams(int64_t elements, size_t bytes) {
    return elements * 2 > kTurnCached / (int64_t)bytes;
}

}  // namespace

}  // namespace bmmc
