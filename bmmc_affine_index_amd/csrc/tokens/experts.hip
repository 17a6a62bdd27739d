// experts.hip -- token rows to their experts and back (gfx950).
//
// All three passes are bound by memory.  They go token by token, so that each
// token's own row is read or written once however many choices it has, and
// the rows by expert, which are choices times as many, are touched once each:
//   gather    reads T D, writes R D elements
//   combine   reads up to T K D, writes T D
//   backward  reads T D + T K D, writes R D
// A lane holds one 16-byte vector of the token's row and moves the same
// columns of all its choices' rows, whose loads are in flight together.
#include "device.h"
#include "tokens.h"

namespace bmmc {

namespace {

constexpr int kMoveThreads = 256;
constexpr int kMoveWaves = kMoveThreads / 64;
// Rows of the order that one wave looks through for padding.
constexpr int kPadRows = 16;

// This lane's token and first element; at < 0 without any.  A row that is not
// whole vectors ends in one that overlaps the vector before it: both write the
// same values there, and no lane needs a form of its own.  Rows of less than
// one vector take kernels of N = 1.
struct Place {
    int64_t token, at;
};

struct Cut {
    FastDiv by;        // WAVE: waves a token; else vectors a token
    uint32_t parts;    // workgroups of the tokens
    uint32_t vectors;  // vectors a token
};

// WAVE: each wave is one token's, so that its row numbers and weights are
// scalars; else lanes take the vectors of successive tokens in turn, which
// leaves no lane without work when a row is not a multiple of 64 vectors.
template <bool WAVE, int N>
__device__ __forceinline__ Place locate(const Cut &c, int64_t tokens, int64_t dim,
                                        uint32_t block) {
    uint32_t token, vec;
    if constexpr (WAVE) {
        const uint32_t task = block * kMoveWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        token = quotient(c.by, task);
        vec = (task - token * c.by.d) * 64 + (threadIdx.x & 63);
    } else {
        const uint32_t task = block * kMoveThreads + threadIdx.x;
        token = quotient(c.by, task);
        vec = task - token * c.by.d;
    }
    const int64_t at = min((int64_t)vec * N, dim - N);
    return Place{(int64_t)token, token < tokens && vec < c.vectors ? at : -1};
}

// Rows and weights of G choices from i on; -1 for one without a row.
template <typename T, int G>
__device__ __forceinline__ void choices_at(const MoveArgs &a, int64_t i, int32_t (&row)[G],
                                           float (&w)[G]) {
#pragma unroll
    for (int g = 0; g < G; ++g) row[g] = a.rows[i + g];
    if (!a.weights) {
#pragma unroll
        for (int g = 0; g < G; ++g) w[g] = 1.0f;
    } else if (a.weights_are_f32) {
#pragma unroll
        for (int g = 0; g < G; ++g) w[g] = static_cast<const float *>(a.weights)[i + g];
    } else {
#pragma unroll
        for (int g = 0; g < G; ++g) w[g] = (float)static_cast<const T *>(a.weights)[i + g];
    }
#pragma unroll
    for (int g = 0; g < G; ++g) row[g] = row[g] < a.capacity ? row[g] : -1;
}

// Zero the padding among kPadRows rows of the order, by one wave.
template <typename T, int N>
__device__ __forceinline__ void zero_padding(const MoveArgs &a, int64_t wave) {
    const int lane = threadIdx.x & 63;
    const int64_t r0 = wave * kPadRows;
    const int64_t r = r0 + lane;
    const bool pad = lane < kPadRows && r < a.capacity && a.slots[r] < 0;
    uint64_t todo = __ballot(pad);
    const dev::Vec<T, N> none = dev::narrow<T, N>(dev::Floats<N>(0.0f));
    while (todo) {
        const int k = __builtin_ctzll(todo);
        todo &= todo - 1;
        T *out = static_cast<T *>(a.out) + (r0 + k) * a.out_stride;
        for (int64_t at = (int64_t)lane * N; at < a.dim; at += 64 * N)
            dev::store<T, N>(out + min(at, a.dim - N), none);
    }
}

template <typename T, int N, bool WAVE>
__global__ void __launch_bounds__(kMoveThreads)
    bmmc_expert_gather_kernel(const MoveArgs a, const Cut c, uint32_t block0) {
    const uint32_t block = block0 + blockIdx.x;
    if (block >= c.parts) {
        zero_padding<T, N>(a, (int64_t)(block - c.parts) * kMoveWaves + (threadIdx.x >> 6));
        return;
    }
    const Place p = locate<WAVE, N>(c, a.tokens, a.dim, block);
    if (p.at < 0) return;
    const dev::Vec<T, N> v =
        dev::load<T, N>(static_cast<const T *>(a.x) + p.token * a.x_stride + p.at);
    const int32_t *rows = a.rows + p.token * a.choices;
    T *out = static_cast<T *>(a.out) + p.at;
    for (int k = 0; k < a.choices; ++k) {
        const int32_t r = rows[k];
        if (r >= 0 && r < a.capacity) dev::store<T, N>(out + r * a.out_stride, v);
    }
}

// Adds G choices from k on, their rows' loads in flight together.
template <typename T, int N, int G>
__device__ __forceinline__ void add_rows(const MoveArgs &a, const Place &p, int k,
                                         dev::Floats<N> &sum) {
    dev::Vec<T, N> v[G];
    float w[G];
    int32_t row[G];
    choices_at<T, G>(a, p.token * a.choices + k, row, w);
    // a dropped choice reads row 0, which is there, and adds nothing
#pragma unroll
    for (int g = 0; g < G; ++g)
        v[g] = dev::load<T, N>(static_cast<const T *>(a.x) + max(row[g], 0) * a.x_stride + p.at);
#pragma unroll
    for (int g = 0; g < G; ++g) {
        const dev::Floats<N> f = dev::widen<T, N>(v[g]);
#pragma unroll
        for (int j = 0; j < N; ++j) sum[j] = row[g] >= 0 ? fmaf(w[g], f[j], sum[j]) : sum[j];
    }
}

template <typename T, int N, bool WAVE>
__global__ void __launch_bounds__(kMoveThreads)
    bmmc_expert_combine_kernel(const MoveArgs a, const Cut c, uint32_t block0) {
    const Place p = locate<WAVE, N>(c, a.tokens, a.dim, block0 + blockIdx.x);
    if (p.at < 0) return;
    dev::Floats<N> sum = 0.0f;
    int k = 0;
    for (; k + 8 <= a.choices; k += 8) add_rows<T, N, 8>(a, p, k, sum);
    if (a.choices & 4) add_rows<T, N, 4>(a, p, k, sum), k += 4;
    if (a.choices & 2) add_rows<T, N, 2>(a, p, k, sum), k += 2;
    if (a.choices & 1) add_rows<T, N, 1>(a, p, k, sum);
    dev::store<T, N>(static_cast<T *>(a.out) + p.token * a.out_stride + p.at,
                     dev::narrow<T, N>(sum));
}

// Gradients of G choices from k on of one token, by WAVES waves: each lane
// sums its columns, then the lanes, then the waves, in a fixed order.
template <typename T, int N, int WAVES, int G>
__device__ __forceinline__ void choices_backward(const MoveArgs &a, int64_t token, int k,
                                                 int part, float *lds) {
    const int lane = threadIdx.x & 63;
    float dot[G], w[G];
    int32_t row[G];
    const int64_t i = token * a.choices + k;
    choices_at<T, G>(a, i, row, w);
#pragma unroll
    for (int g = 0; g < G; ++g) dot[g] = 0.0f;
    const T *grad = static_cast<const T *>(a.x) + token * a.x_stride;
    for (int64_t from = (int64_t)(part * 64 + lane) * N; from < a.dim; from += WAVES * 64 * N) {
        const int64_t at = min(from, a.dim - N);
        const dev::Floats<N> d = dev::widen<T, N>(dev::load<T, N, false>(grad + at));
        dev::Vec<T, N> v[G];
#pragma unroll
        for (int g = 0; g < G; ++g)
            v[g] = dev::load<T, N>(static_cast<const T *>(a.in) +
                                   max(row[g], 0) * a.in_stride + at);
#pragma unroll
        for (int g = 0; g < G; ++g) {
            const dev::Floats<N> f = dev::widen<T, N>(v[g]);
            // elements that the vector before holds too are summed there alone
#pragma unroll
            for (int j = 0; j < N; ++j) dot[g] = j >= from - at ? fmaf(d[j], f[j], dot[g]) : dot[g];
            if (row[g] >= 0)
                dev::store<T, N>(static_cast<T *>(a.out) + row[g] * a.out_stride + at,
                                 dev::narrow<T, N>(d * w[g]));
        }
    }
#pragma unroll
    for (int g = 0; g < G; ++g) dot[g] = dev::wave_sum(dot[g]);
    if constexpr (WAVES > 1) {
        __syncthreads();  // the last group's sums have been read
        if (lane == 0)
#pragma unroll
            for (int g = 0; g < G; ++g) lds[part * 8 + g] = dot[g];
        __syncthreads();
#pragma unroll
        for (int g = 0; g < G; ++g) {
            dot[g] = 0.0f;
            for (int p = 0; p < WAVES; ++p) dot[g] += lds[p * 8 + g];
        }
    }
    if (part == 0 && lane == 0) {
#pragma unroll
        for (int g = 0; g < G; ++g) {
            const float r = row[g] < 0 ? 0.0f : dot[g];
            if (a.weights_are_f32)
                static_cast<float *>(a.grad_weights)[i + g] = r;
            else
                static_cast<T *>(a.grad_weights)[i + g] = (T)r;
        }
    }
}

template <typename T, int N, int WAVES>
__global__ void __launch_bounds__(kMoveThreads)
    bmmc_expert_combine_backward_kernel(const MoveArgs a, uint32_t parts, uint32_t block0) {
    __shared__ float lds[kMoveWaves * 8];
    const uint32_t block = block0 + blockIdx.x;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (block >= parts) {
        zero_padding<T, N>(a, (int64_t)(block - parts) * kMoveWaves + wave);
        return;
    }
    const int64_t token = (int64_t)block * (kMoveWaves / WAVES) + (WAVES == 1 ? wave : 0);
    const int part = WAVES == 1 ? 0 : wave;
    if (token >= a.tokens) return;  // a whole wave, or with 4 waves a token the workgroup
    int k = 0;
    for (; k + 8 <= a.choices; k += 8) choices_backward<T, N, WAVES, 8>(a, token, k, part, lds);
    if (a.choices & 4) choices_backward<T, N, WAVES, 4>(a, token, k, part, lds), k += 4;
    if (a.choices & 2) choices_backward<T, N, WAVES, 2>(a, token, k, part, lds), k += 2;
    if (a.choices & 1) choices_backward<T, N, WAVES, 1>(a, token, k, part, lds);
}

// Whether each wave is one token's: where that leaves at most a fifth of the
// lanes idle, or where the vectors of all tokens pass the 31 bits of a
// quotient.  *fits is false where the waves pass them too.
template <int N> bool by_waves(const MoveArgs &a, Cut *c, bool *fits) {
    constexpr int64_t kMost = int64_t(1) << 31;
    const int64_t vectors = (a.dim + N - 1) / N, waves = (vectors + 63) / 64;
    c->vectors = (uint32_t)vectors;
    *fits = a.tokens * waves < kMost - kMoveThreads;
    if (vectors * 5 >= waves * 64 * 4 || a.tokens * vectors >= kMost - kMoveThreads) {
        c->by = fast_div((uint32_t)waves);
        c->parts = (uint32_t)((a.tokens * waves + kMoveWaves - 1) / kMoveWaves);
        return true;
    }
    c->by = fast_div((uint32_t)vectors);
    c->parts = (uint32_t)((a.tokens * vectors + kMoveThreads - 1) / kMoveThreads);
    return false;
}

int64_t pad_blocks(int64_t capacity) {
    return (capacity + kMoveWaves * kPadRows - 1) / (kMoveWaves * kPadRows);
}

template <typename T, int N> int gather_n(const MoveArgs &a, hipStream_t s) {
    Cut c;
    bool fits;
    const bool wave = by_waves<N>(a, &c, &fits);
    if (!fits) return BMMC_ERR_UNSUPPORTED;
    return in_launches(c.parts + pad_blocks(a.capacity), kMoveThreads, [&](uint32_t nb, int64_t b0) {
        if (wave)
            hipLaunchKernelGGL((bmmc_expert_gather_kernel<T, N, true>), dim3(nb),
                               dim3(kMoveThreads), 0, s, a, c, (uint32_t)b0);
        else
            hipLaunchKernelGGL((bmmc_expert_gather_kernel<T, N, false>), dim3(nb),
                               dim3(kMoveThreads), 0, s, a, c, (uint32_t)b0);
    });
}

template <typename T, int N> int combine_n(const MoveArgs &a, hipStream_t s) {
    Cut c;
    bool fits;
    const bool wave = by_waves<N>(a, &c, &fits);
    if (!fits) return BMMC_ERR_UNSUPPORTED;
    return in_launches(c.parts, kMoveThreads, [&](uint32_t nb, int64_t b0) {
        if (wave)
            hipLaunchKernelGGL((bmmc_expert_combine_kernel<T, N, true>), dim3(nb),
                               dim3(kMoveThreads), 0, s, a, c, (uint32_t)b0);
        else
            hipLaunchKernelGGL((bmmc_expert_combine_kernel<T, N, false>), dim3(nb),
                               dim3(kMoveThreads), 0, s, a, c, (uint32_t)b0);
    });
}

// One wave a token fills the card from about four waves a SIMD on (1024
// SIMDs); below that four waves share a token.
constexpr int64_t kBackwardWaveTokens = 4096;

template <typename T, int N> int combine_backward_n(const MoveArgs &a, hipStream_t s) {
    const bool wide = a.tokens < kBackwardWaveTokens;
    const int64_t parts = wide ? a.tokens : (a.tokens + kMoveWaves - 1) / kMoveWaves;
    return in_launches(parts + pad_blocks(a.capacity), kMoveThreads, [&](uint32_t nb, int64_t b0) {
        if (wide)
            hipLaunchKernelGGL((bmmc_expert_combine_backward_kernel<T, N, kMoveWaves>), dim3(nb),
                               dim3(kMoveThreads), 0, s, a, (uint32_t)parts, (uint32_t)b0);
        else
            hipLaunchKernelGGL((bmmc_expert_combine_backward_kernel<T, N, 1>), dim3(nb),
                               dim3(kMoveThreads), 0, s, a, (uint32_t)parts, (uint32_t)b0);
    });
}

// Whole vectors, or single elements for rows of less than one.
#define BMMC_BY_WIDTH(call, T, a, s)                                                  \
    ((a).dim >= dev::Lanes<T>::N ? call<T, dev::Lanes<T>::N>((a), (s)) : call<T, 1>((a), (s)))

}  // namespace

int launch_expert_gather(const MoveArgs &a, int type, hipStream_t s) {
    // rows are copied as they are: 16-bit types share one kernel
    return type == BMMC_F32 ? BMMC_BY_WIDTH(gather_n, float, a, s)
                            : BMMC_BY_WIDTH(gather_n, dev::f16_t, a, s);
}

int launch_expert_combine(const MoveArgs &a, int type, hipStream_t s) {
    switch (type) {
    case BMMC_F32: return BMMC_BY_WIDTH(combine_n, float, a, s);
    case BMMC_F16: return BMMC_BY_WIDTH(combine_n, dev::f16_t, a, s);
    default: return BMMC_BY_WIDTH(combine_n, dev::bf16_t, a, s);
    }
}

int launch_expert_combine_backward(const MoveArgs &a, int type, hipStream_t s) {
    switch (type) {
    case BMMC_F32: return BMMC_BY_WIDTH(combine_backward_n, float, a, s);
    case BMMC_F16: return BMMC_BY_WIDTH(combine_backward_n, dev::f16_t, a, s);
    default: return BMMC_BY_WIDTH(combine_backward_n, dev::bf16_t, a, s);
    }
}

}  // namespace bmmc
