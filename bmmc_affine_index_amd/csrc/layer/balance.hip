// balance.hip -- the balance loss of a router, and its gradient (gfx950).
//
// The loss sums p = softmax(logits) over the tokens for each expert, the
// gradient needs each token's p again: one pass over the logits each, in which
// a token's row lies in 16 lanes of a wave or, if long, more, and its maximum and
// sums go through moves among them.  A lane holds the same
// experts of all its rows, so that the sums over tokens stay in registers until
// the end; they leave the workgroup once and are summed by a second launch, in
// a fixed order.  Choices are counted in LDS by whole numbers, whose order
// does not matter.
//
// Bound by memory: the logits are read once for the loss, once for the gradient.
// 65536 tokens of 256 experts in fp32: 17 us and 7 for the join (36 and 10 with a row in
// 64 lanes and 8 waves a workgroup), the gradient 22.5, 6.0 TB/s.
#include <algorithm>

#include "../tokens/device.h"
#include "lanes.h"
#include "layer.h"

namespace bmmc {

namespace {

// Waves of a workgroup that sums rows: as many as have registers for a lane's vectors.
template <typename T, int C> constexpr int kBalanceWaves = C * dev::Lanes<T>::N > 16 ? 8 : 16;
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kColumns = kBalanceColumns;

// C vectors of a row in each of 1 << shift lanes; past its end what weighs nothing.
template <typename T, int C>
__device__ __forceinline__ void load_row(const T *row, int lane, int shift, int experts,
                                         dev::Vec<T, dev::Lanes<T>::N> (&raw)[C]) {
    constexpr int N = dev::Lanes<T>::N;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int at = ((c << shift) + lane) * N;
        if (at + N <= experts) {
            raw[c] = dev::load<T, N, false>(row + at);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i)
                raw[c].v[i] = at + i < experts ? row[at + i] : (T)-__builtin_inff();
        }
    }
}

// p = softmax of a row.  A maximum that is no number leaves NaN in all of it.
template <typename T, int C>
__device__ __forceinline__ void softmax_row(const dev::Vec<T, dev::Lanes<T>::N> (&raw)[C], int shift,
                                            float (&p)[C * dev::Lanes<T>::N]) {
    constexpr int N = dev::Lanes<T>::N;
    float top = -__builtin_inff();
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const dev::Floats<N> x = dev::widen<T, N>(raw[c]);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            p[c * N + i] = x[i];
            top = fmaxf(top, x[i]);
        }
    }
    top = dev::over_lanes(top, shift, dev::Largest());
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < C * N; ++i) {
        p[i] = __builtin_amdgcn_exp2f((p[i] - top) * kLog2e);
        sum += p[i];
    }
    sum = dev::over_lanes(sum, shift, dev::Sum());
    const float by = 1.0f / sum;
#pragma unroll
    for (int i = 0; i < C * N; ++i) p[i] *= by;
}

// An expert's count and slope, and its part of the loss.
__device__ __forceinline__ double end_expert(const BalanceArgs &a, int e, int32_t count,
                                             int32_t tokens, double sum) {
    const double counted = (double)tokens;
    const float slope =
        tokens ? (float)((double)count * a.num_experts / (counted * counted * a.choices)) : 0.0f;
    a.counts[e] = count;
    a.slopes[e] = slope;
    return (double)slope * sum;
}

template <typename T, int C>
__global__ void __launch_bounds__((64 * kBalanceWaves<T, C>))
    bmmc_balance_rows_kernel(const BalanceArgs a, int shift) {
    constexpr int N = dev::Lanes<T>::N, WAVES = kBalanceWaves<T, C>;
    extern __shared__ float part[];  // WAVES, num_experts; then the counts and the tokens'
    const int E = a.num_experts, tid = threadIdx.x;
    int32_t *hits = reinterpret_cast<int32_t *>(part + WAVES * E);
    const int64_t from = blockIdx.x * a.chunk, to = min(from + a.chunk, a.tokens);
    const int lane = tid & 63, in_row = lane & ((1 << shift) - 1), wave = tid >> 6;
    const int rows = 64 >> shift;
    float sums[C * N] = {};
    dev::Vec<T, N> next[C];
    const int64_t step = (int64_t)rows * WAVES;
    const T *logits = static_cast<const T *>(a.logits);
    bool on = false;
    // a row that is not counted is read all the same, not to wait for its mask first
    const auto fetch = [&](int64_t t) {
        on = t < to;
        if (!on) return;
        if (a.mask) on = a.mask[t] != 0;
        load_row<T, C>(logits + t * a.stride, in_row, shift, E, next);
    };
    int64_t t = from + (int64_t)wave * rows + (lane >> shift);
    fetch(t);  // on its way while the choices are counted
    for (int e = tid; e <= E; e += blockDim.x) hits[e] = 0;
    if (blockIdx.x == 0 && tid == 0) *reinterpret_cast<uint32_t *>(a.hits + (int64_t)a.blocks * (E + 1)) = 0;
    __syncthreads();
    // a choice, and with a token's first the token
    for (int64_t i = from * a.choices + tid; i < to * a.choices; i += blockDim.x) {
        const int64_t t = quotient(a.by_choices, (uint32_t)i);
        if (a.mask && !a.mask[t]) continue;
        const int64_t e = a.is64 ? static_cast<const int64_t *>(a.experts)[i]
                                 : (int64_t)static_cast<const int32_t *>(a.experts)[i];
        if (e >= 0 && e < E) atomicAdd(&hits[e], 1);
        if (i == t * a.choices) atomicAdd(&hits[E], 1);
    }
    // every lane of a wave goes round as often as any: rows of a wave are in step
    for (int64_t t0 = from + (int64_t)wave * rows; t0 < to; t0 += step, t += step) {
        dev::Vec<T, N> raw[C];
        const bool now = on;
#pragma unroll
        for (int c = 0; c < C; ++c) raw[c] = next[c];
        fetch(t + step);
        float p[C * N];
        softmax_row<T, C>(raw, shift, p);
#pragma unroll
        for (int i = 0; i < C * N; ++i) sums[i] += now ? p[i] : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < C * N; ++i)
        for (int d = 1 << shift; d < 64; d <<= 1) sums[i] += __shfl_xor(sums[i], d, 64);
    if (lane < 1 << shift)
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int e = ((c << shift) + lane) * N + i;
                if (e < E) part[wave * E + e] = sums[c * N + i];
            }
    __syncthreads();
    double all = 0.0;
    for (int e = tid; e < E; e += blockDim.x) {
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) s += part[w * E + e];
        if (gridDim.x > 1) {
            a.sums[(int64_t)blockIdx.x * E + e] = s;
            a.hits[(int64_t)blockIdx.x * (E + 1) + e] = hits[e];
        } else {
            all += end_expert(a, e, hits[e], hits[E], (double)s);
        }
    }
    if (gridDim.x > 1) {
        if (tid == 0) a.hits[(int64_t)blockIdx.x * (E + 1) + E] = hits[E];
        return;
    }
    // alone: the loss is the sum of its terms
#pragma unroll
    for (int d = 32; d; d >>= 1) all += __shfl_xor(all, d, 64);
    __shared__ double ends[WAVES];
    if (lane == 0) ends[wave] = all;
    __syncthreads();
    if (tid == 0) {
        for (int w = 1; w < WAVES; ++w) all += ends[w];
        *a.loss = (float)all;
    }
}

// The workgroups' sums joined, kColumns experts a workgroup, in an order that is
// always the same; the last one to end sums the loss, in the experts' order.
__global__ void __launch_bounds__(1024) bmmc_balance_join_kernel(const BalanceArgs a) {
    constexpr int R = 1024 / kColumns;  // threads of an expert
    __shared__ double sums[R][kColumns];
    __shared__ int32_t hits[R][kColumns];
    __shared__ int32_t tokens;
    const int E = a.num_experts, col = threadIdx.x % kColumns, row = threadIdx.x / kColumns;
    const int e = blockIdx.x * kColumns + col;
    if (threadIdx.x == 0) tokens = 0;
    __syncthreads();
    int32_t n = 0;
    for (int b = threadIdx.x; b < a.blocks; b += blockDim.x) n += a.hits[(int64_t)b * (E + 1) + E];
    double s = 0.0;
    int32_t h = 0;
    if (e < E)
#pragma unroll 4
        for (int b = row; b < a.blocks; b += R) {
            s += (double)a.sums[(int64_t)b * E + e];
            h += a.hits[(int64_t)b * (E + 1) + e];
        }
    if (n) atomicAdd(&tokens, n);
    sums[row][col] = s;
    hits[row][col] = h;
    for (int half = R / 2; half; half >>= 1) {
        __syncthreads();
        if (row < half) {
            sums[row][col] += sums[row + half][col];
            hits[row][col] += hits[row + half][col];
        }
    }
    uint32_t *done = reinterpret_cast<uint32_t *>(a.hits + (int64_t)a.blocks * (E + 1));
    float *losses = reinterpret_cast<float *>(done + 1);
    if (row == 0) {
        double term = 0.0;
        if (e < E) term = end_expert(a, e, hits[0][col], tokens, sums[0][col]);
#pragma unroll
        for (int d = kColumns / 2; d; d >>= 1) term += __shfl_xor(term, d, kColumns);
        int32_t last = 0;
        if (col == 0) {
            __hip_atomic_store(&losses[blockIdx.x], (float)term, __ATOMIC_RELAXED,
                               __HIP_MEMORY_SCOPE_AGENT);
            last = __hip_atomic_fetch_add(done, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) ==
                   gridDim.x - 1;
        }
        if (__shfl(last, 0, kColumns)) {
            double all = 0.0;
            for (uint32_t b = col; b < gridDim.x; b += kColumns)
                all += (double)__hip_atomic_load(&losses[b], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
            for (int d = kColumns / 2; d; d >>= 1) all += __shfl_xor(all, d, kColumns);
            if (col == 0) *a.loss = (float)all;
        }
    }
}

template <typename T, int C>
__global__ void __launch_bounds__(256) bmmc_balance_backward_kernel(const BalanceArgs a, int shift,
                                                                    int64_t block0) {
    constexpr int N = dev::Lanes<T>::N;
    const int lane = threadIdx.x & 63, in_row = lane & ((1 << shift) - 1), rows = 64 >> shift;
    const int64_t first = ((block0 + blockIdx.x) * 4 + (threadIdx.x >> 6)) * a.chunk * rows;
    const int E = a.num_experts;
    float slope[C * N];
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int e = ((c << shift) + in_row) * N + i;
            slope[c * N + i] = e < E ? a.slopes[e] : 0.0f;
        }
    const float g = *a.grad;
    const T *logits = static_cast<const T *>(a.logits);
    dev::Vec<T, N> next[C];
    bool on = false;
    const auto fetch = [&](int64_t t) {
        on = t < a.tokens;
        if (!on) return;
        if (a.mask) on = a.mask[t] != 0;
        load_row<T, C>(logits + t * a.stride, in_row, shift, E, next);
    };
    int64_t t = first + (lane >> shift);
    fetch(t);
    for (int64_t k = 0; k < a.chunk && first + k * rows < a.tokens; ++k, t += rows) {
        dev::Vec<T, N> raw[C];
        const bool now = on;
#pragma unroll
        for (int c = 0; c < C; ++c) raw[c] = next[c];
        on = false;
        if (k + 1 < a.chunk) fetch(t + rows);
        float p[C * N];
        softmax_row<T, C>(raw, shift, p);
        float dot = 0.0f;
#pragma unroll
        for (int i = 0; i < C * N; ++i) dot += slope[i] * p[i];
        dot = dev::over_lanes(dot, shift, dev::Sum());
        if (t >= a.tokens) continue;
        T *out = static_cast<T *>(a.grad_logits) + t * a.grad_stride;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int at = ((c << shift) + in_row) * N;
            dev::Floats<N> y;
#pragma unroll
            for (int i = 0; i < N; ++i)
                y[i] = now ? g * (p[c * N + i] * (slope[c * N + i] - dot)) : 0.0f;
            const dev::Vec<T, N> z = dev::narrow<T, N>(y);
            if (at + N <= E) {
                dev::store<T, N, false>(out + at, z);
            } else {
#pragma unroll
                for (int i = 0; i < N; ++i)
                    if (at + i < E) out[at + i] = z.v[i];
            }
        }
    }
}

// Lanes and vectors a lane of a row: 16 lanes, which exchange at the least cost and
// leave a wave several rows to work on, and more of them beyond four vectors each.
struct Cut {
    int shift, vectors;
};
template <typename T> Cut cut_of(int experts) {
    constexpr int N = dev::Lanes<T>::N;
    const int all = (experts + N - 1) / N;
    Cut c{0, 1};
    while (c.shift < 4 && 1 << c.shift < all) ++c.shift;
    while (c.vectors < 4 && c.vectors << c.shift < all) c.vectors *= 2;
    while (c.shift < 6 && c.vectors << c.shift < all) ++c.shift;
    while (c.vectors << c.shift < all) c.vectors *= 2;
    return c;
}

template <typename T, int C> int forward(const BalanceArgs &x, int shift, hipStream_t s) {
    BalanceArgs a = x;
    a.chunk = (a.tokens + a.blocks - 1) / a.blocks;
    const int waves = kBalanceWaves<T, C>;
    const size_t lds = ((size_t)(waves + 1) * a.num_experts + 1) * 4;
    hipLaunchKernelGGL((bmmc_balance_rows_kernel<T, C>), dim3(a.blocks), dim3(64 * waves), lds, s, a,
                       shift);
    if (a.blocks > 1)
        hipLaunchKernelGGL(bmmc_balance_join_kernel, dim3((a.num_experts + kColumns - 1) / kColumns),
                           dim3(1024), 0, s, a);
    return hipGetLastError() == hipSuccess ? BMMC_OK : BMMC_ERR_HIP;
}

template <typename T, int C> int backward(const BalanceArgs &x, int shift, hipStream_t s) {
    BalanceArgs a = x;
    const int64_t each = 4 * (64 >> shift);  // rows of a workgroup at once
    // up to four rounds of rows, where that leaves enough workgroups
    const int64_t rounds = (a.tokens + each - 1) / each;
    a.chunk = std::max<int64_t>(1, std::min<int64_t>(4, rounds / 2048));
    return in_launches((rounds + a.chunk - 1) / a.chunk, 256, [&](uint32_t nb, int64_t b0) {
        hipLaunchKernelGGL((bmmc_balance_backward_kernel<T, C>), dim3(nb), dim3(256), 0, s, a, shift, b0);
    });
}

template <typename T, class F> int by_vectors(int experts, F call) {
    const Cut c = cut_of<T>(experts);
    switch (c.vectors) {
    case 1: return call(std::integral_constant<int, 1>(), c.shift);
    case 2: return call(std::integral_constant<int, 2>(), c.shift);
    default: break;
    }
    // BMMC_MAX_EXPERTS in 32 bits are 8 vectors in each of 64 lanes, in 16 bits 4
    if constexpr (sizeof(T) == 4)
        if (c.vectors == 8) return call(std::integral_constant<int, 8>(), c.shift);
    return call(std::integral_constant<int, 4>(), c.shift);
}

template <class F> int by_type(int type, F call) {
    switch (type) {
    case BMMC_F32: return call(float());
    case BMMC_F16: return call(dev::f16_t());
    default: return call(dev::bf16_t());
    }
}

}  // namespace

int launch_expert_balance(const BalanceArgs &a, hipStream_t s) {
    return by_type(a.type, [&](auto type) {
        typedef decltype(type) T;
        return by_vectors<T>(a.num_experts, [&](auto c, int shift) {
            return forward<T, decltype(c)::value>(a, shift, s);
        });
    });
}

int launch_expert_balance_backward(const BalanceArgs &a, hipStream_t s) {
    return by_type(a.type, [&](auto type) {
        typedef decltype(type) T;
        return by_vectors<T>(a.num_experts, [&](auto c, int shift) {
            return backward<T, decltype(c)::value>(a, shift, s);
        });
    });
}

}  // namespace bmmc
