// experts.hip -- token rows to their experts and back (gfx950).
//
// All three passes are bound by memory:
//   gather    reads T D, writes R D elements
//   combine   reads up to T K D, writes T D
//   backward  reads T D + T K D, writes R D
// They go token by token, so that each token's own row comes from memory or goes
// there once however many choices it has.  In gather and combine a lane holds one
// 16-byte vector of the token's row and moves the same columns of its choices'
// rows, whose loads are in flight together; the backward pass, which sums along
// the rows, has a wave for each choice.
#include "device.h"
#include "tokens.h"

namespace bmmc {

namespace {

// Threads of a workgroup, measured on 16384 tokens of 8 choices, 8 KiB a row:
// gather 224 us with 256 and 230 with 128, combine 212 and 200; at other sizes
// (2 to 14 KiB a row) the two differ by up to 3% the same way.
constexpr int kGatherThreads = 256;
constexpr int kCombineThreads = 128;
constexpr int kBackwardThreads = 256;
// Rows of the order that one wave looks through for padding: where there is
// much, few waves would take long over it; where there is none, many cost time
// (65536 rows without any: 2% of the backward pass with 4 rows a wave, nothing
// to be seen with 8).
constexpr int kPadRows = 8;

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
// SHARES waves next to each other have the same place.
template <int THREADS, bool WAVE, int N, int SHARES = 1>
__device__ __forceinline__ Place locate(const Cut &c, int64_t tokens, int64_t dim,
                                        uint32_t block) {
    uint32_t token, vec;
    if constexpr (WAVE) {
        const uint32_t task = block * (THREADS / 64 / SHARES) +
                              __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) / SHARES;
        token = quotient(c.by, task);
        vec = (task - token * c.by.d) * 64 + (threadIdx.x & 63);
    } else {
        const uint32_t task = block * THREADS + threadIdx.x;
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
        dev::by_hint(a.whole_lines, [&](auto nt) {
            for (int64_t at = (int64_t)lane * N; at < a.dim; at += 64 * N)
                dev::store<T, N, nt.value>(out + min(at, a.dim - N), none);
        });
    }
}

// SHARES: waves that share a token's choices, each with the token's row.
template <typename T, int N, bool WAVE, int SHARES>
__global__ void __launch_bounds__(kGatherThreads)
    bmmc_expert_gather_kernel(const MoveArgs a, const Cut c, uint32_t pads, uint32_t block0) {
    const uint32_t block = block0 + blockIdx.x;
    if (block < pads) {
        zero_padding<T, N>(a, (int64_t)block * (kGatherThreads / 64) + (threadIdx.x >> 6));
        return;
    }
    const Place p = locate<kGatherThreads, WAVE, N, SHARES>(c, a.tokens, a.dim, block - pads);
    if (p.at < 0) return;
    // a layer's input, which the layer before has just written: through the
    // caches (16384 tokens of 8 choices, 4 KiB a row: 102 us, 114 streamed)
    const dev::Vec<T, N> v =
        dev::load<T, N, false>(static_cast<const T *>(a.x) + p.token * a.x_stride + p.at);
    const int32_t *rows = a.rows + p.token * a.choices;
    const int share = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) % SHARES;
    T *out = static_cast<T *>(a.out) + p.at;
    dev::by_hint(a.whole_lines, [&](auto nt) {
        for (int k = share; k < a.choices; k += SHARES) {
            const int32_t r = rows[k];
            if (r >= 0 && r < a.capacity) dev::store<T, N, nt.value>(out + r * a.out_stride, v);
        }
    });
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
    dev::by_hint(a.stream, [&](auto nt) {
#pragma unroll
        for (int g = 0; g < G; ++g)
            v[g] = dev::load<T, N, nt.value>(static_cast<const T *>(a.x) +
                                             max(row[g], 0) * a.x_stride + p.at);
    });
#pragma unroll
    for (int g = 0; g < G; ++g) {
        const dev::Floats<N> f = dev::widen<T, N>(v[g]);
#pragma unroll
        for (int j = 0; j < N; ++j) sum[j] = row[g] >= 0 ? fmaf(w[g], f[j], sum[j]) : sum[j];
    }
}

template <typename T, int N, bool WAVE>
__global__ void __launch_bounds__(kCombineThreads)
    bmmc_expert_combine_kernel(const MoveArgs a, const Cut c, uint32_t block0) {
    const Place p = locate<kCombineThreads, WAVE, N>(c, a.tokens, a.dim, block0 + blockIdx.x);
    if (p.at < 0) return;
    dev::Floats<N> sum = 0.0f;
    int k = 0;
    for (; k + 8 <= a.choices; k += 8) add_rows<T, N, 8>(a, p, k, sum);
    // the loads of the last choices, too, are in flight together
    switch (a.choices - k) {
    case 7: add_rows<T, N, 7>(a, p, k, sum); break;
    case 6: add_rows<T, N, 6>(a, p, k, sum); break;
    case 5: add_rows<T, N, 5>(a, p, k, sum); break;
    case 4: add_rows<T, N, 4>(a, p, k, sum); break;
    case 3: add_rows<T, N, 3>(a, p, k, sum); break;
    case 2: add_rows<T, N, 2>(a, p, k, sum); break;
    case 1: add_rows<T, N, 1>(a, p, k, sum); break;
    default: break;
    }
    dev::by_hint(a.whole_lines, [&](auto nt) {
        dev::store<T, N, nt.value>(static_cast<T *>(a.out) + p.token * a.out_stride + p.at,
                                   dev::narrow<T, N>(sum));
    });
}

// Gradients of one choice by 2^lanes_log2 lanes (WAVE: by a wave, so that its
// numbers are scalars): grad_in of its row = weight * its token's gradient, and
// that gradient's product with the row.  The choices of a token are next to each
// other, so that its gradient comes from memory once and then from the caches.
// V vectors of a lane of both rows are in flight together.  8192 tokens of 8
// choices, 4 KiB a row: 102 us; 104 with four waves that each take a part of all 8
// rows and join their sums, 112 in the order of the rows, which reads and writes
// in sequence but has each gradient from memory 8 times.
//
// Each lane sums its columns, then the lanes are joined, in a fixed order.
template <typename T, int N, int V, bool WAVE>
__global__ void __launch_bounds__(kBackwardThreads)
    bmmc_expert_combine_backward_kernel(const MoveArgs a, const FastDiv by_choices,
                                        int lanes_log2, uint32_t pads, uint32_t block0) {
    uint32_t block = block0 + blockIdx.x;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (block < pads) {
        zero_padding<T, N>(a, (int64_t)block * (kBackwardThreads / 64) + wave);
        return;
    }
    block -= pads;
    uint32_t i;
    int lane, lanes;
    if constexpr (WAVE) {
        i = block * (kBackwardThreads / 64) + wave;
        lane = threadIdx.x & 63;
        lanes = 64;
    } else {
        lanes = 1 << lanes_log2;
        i = block * (kBackwardThreads >> lanes_log2) + (threadIdx.x >> lanes_log2);
        lane = threadIdx.x & (lanes - 1);
    }
    if (i >= a.tokens * a.choices) return;
    const int32_t row = a.rows[i];
    float dot = 0.0f;
    if (row >= 0 && row < a.capacity) {
        const float w = a.weights_are_f32 ? static_cast<const float *>(a.weights)[i]
                                          : (float)static_cast<const T *>(a.weights)[i];
        const T *grad =
            static_cast<const T *>(a.x) + (int64_t)quotient(by_choices, i) * a.x_stride;
        const T *in = static_cast<const T *>(a.in) + row * a.in_stride;
        T *out = static_cast<T *>(a.out) + row * a.out_stride;
        const int dim = (int)a.dim, last = dim - N, step = lanes * N;
        for (int from = lane * N; from < dim; from += V * step) {
            dev::Vec<T, N> f[V], d[V];
            // a vector past the row's end is the last one again
            dev::by_hint(a.stream, [&](auto nt) {
#pragma unroll
                for (int v = 0; v < V; ++v)
                    f[v] = dev::load<T, N, nt.value>(in + min(from + v * step, last));
            });
#pragma unroll
            for (int v = 0; v < V; ++v)
                d[v] = dev::load<T, N, false>(grad + min(from + v * step, last));
            // every load is under way before the first is waited for
            __builtin_amdgcn_sched_barrier(0);
            dev::by_hint(a.whole_lines, [&](auto nt) {
#pragma unroll
                for (int v = 0; v < V; ++v)
                    if (from + v * step < dim)
                        dev::store<T, N, nt.value>(
                            out + min(from + v * step, last),
                            dev::narrow<T, N>(dev::widen<T, N>(d[v]) * w));
            });
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int want = from + v * step;
                if (want >= dim) break;
                const dev::Floats<N> x = dev::widen<T, N>(f[v]), g = dev::widen<T, N>(d[v]);
                if (want > last) {  // what the vector before holds too is summed there
#pragma unroll
                    for (int j = 0; j < N; ++j) dot = j >= want - last ? fmaf(g[j], x[j], dot) : dot;
                } else {
#pragma unroll
                    for (int j = 0; j < N; ++j) dot = fmaf(g[j], x[j], dot);
                }
            }
        }
    }
    if constexpr (WAVE)
        dot = dev::wave_sum(dot);
    else
        for (int d = lanes / 2; d; d >>= 1) dot += __shfl_xor(dot, d, 64);
    if (lane != 0) return;
    if (a.weights_are_f32)
        static_cast<float *>(a.grad_weights)[i] = dot;
    else
        static_cast<T *>(a.grad_weights)[i] = (T)dot;
}

// Whether each wave is one token's: where that leaves at most two fifths of the
// lanes idle, or where the vectors of all tokens pass the 31 bits of a quotient.
// 8192 tokens of 8 choices, by waves and by lanes in turn: combine of rows of 8
// vectors 7.2 and 5.4 us, 25 vectors 8.5 and 7.9, 72 vectors 15.0 and 14.9, 88
// vectors 17.8 and 17.9; gather 7.7 and 5.1, 8.5 and 8.0, 17.7 and 16.6, 18.6 and
// 20.0.  *fits is false where the waves pass them too.
template <int N, int THREADS>
bool by_waves(const MoveArgs &a, int shares, Cut *c, bool *fits) {
    constexpr int64_t kMost = int64_t(1) << 31;
    const int kWaves = THREADS / 64 / shares;
    const int64_t vectors = (a.dim + N - 1) / N, waves = (vectors + 63) / 64;
    c->vectors = (uint32_t)vectors;
    *fits = a.tokens * waves < kMost - THREADS;
    if (vectors * 5 >= waves * 64 * 3 || a.tokens * vectors >= kMost - THREADS) {
        c->by = fast_div((uint32_t)waves);
        c->parts = (uint32_t)((a.tokens * waves + kWaves - 1) / kWaves);
        return true;
    }
    c->by = fast_div((uint32_t)vectors);
    c->parts = (uint32_t)((a.tokens * vectors + THREADS - 1) / THREADS);
    return false;
}

int64_t pad_blocks(int64_t capacity) {
    static_assert(kGatherThreads == kBackwardThreads, "both look for padding");
    constexpr int kRows = kGatherThreads / 64 * kPadRows;
    return (capacity + kRows - 1) / kRows;
}

// What the caches can still hold of rows that were written just before.
constexpr int64_t kMoveCached = int64_t(96) << 20;

// Waves that share a token's choices in the gather.  With few choices for each,
// a wave's stores end sooner; with one choice for each, tokens that come from
// memory and not from the caches are waited for.  Measured with one, two and four
// waves, rows of whole cache lines: tokens of up to 67 MB (8192 x 6 rows of 8 KiB)
// 75, 73, 67 us, (16384 x 5 of 4 KiB) 63, 61, 56; of 134 MB (16384 x 8 of 8 KiB,
// with the order) 236, 230, 225, (8192 x 6 of 16 KiB) 171, 162, 179, (8192 x 4)
// 121, 112, 135.  Where rows share lines, one wave writes them all, and the
// workgroup's waves write next to each other (16384 x 8 rows of 4094 bytes: 131 us,
// 183 with four).
int gather_shares(const MoveArgs &a, int64_t size) {
    if (!a.whole_lines || a.choices < 4) return 1;
    return a.choices < 8 && a.tokens * a.dim > kMoveCached / size ? 2 : 4;
}

template <typename T, int N> int gather_n(const MoveArgs &a, hipStream_t s) {
    Cut c;
    bool fits;
    const int shares = gather_shares(a, sizeof(T));
    const bool wave = by_waves<N, kGatherThreads>(a, shares, &c, &fits);
    if (!fits) return BMMC_ERR_UNSUPPORTED;
    const int64_t pads = pad_blocks(a.capacity);
    return in_launches(pads + c.parts, kGatherThreads, [&](uint32_t nb, int64_t b0) {
        const auto launch = [&](auto kernel) {
            hipLaunchKernelGGL(kernel, dim3(nb), dim3(kGatherThreads), 0, s, a, c,
                               (uint32_t)pads, (uint32_t)b0);
        };
        if (!wave)
            launch(bmmc_expert_gather_kernel<T, N, false, 1>);
        else if (shares == 1)
            launch(bmmc_expert_gather_kernel<T, N, true, 1>);
        else if (shares == 2)
            launch(bmmc_expert_gather_kernel<T, N, true, 2>);
        else
            launch(bmmc_expert_gather_kernel<T, N, true, 4>);
    });
}

template <typename T, int N> int combine_n(const MoveArgs &a, hipStream_t s) {
    Cut c;
    bool fits;
    const bool wave = by_waves<N, kCombineThreads>(a, 1, &c, &fits);
    if (!fits) return BMMC_ERR_UNSUPPORTED;
    return in_launches(c.parts, kCombineThreads, [&](uint32_t nb, int64_t b0) {
        if (wave)
            hipLaunchKernelGGL((bmmc_expert_combine_kernel<T, N, true>), dim3(nb),
                               dim3(kCombineThreads), 0, s, a, c, (uint32_t)b0);
        else
            hipLaunchKernelGGL((bmmc_expert_combine_kernel<T, N, false>), dim3(nb),
                               dim3(kCombineThreads), 0, s, a, c, (uint32_t)b0);
    });
}

// Lanes of a choice: the power of two that leaves none without a vector, at
// most a wave; a lane's vectors in flight: as many as the row has, at most 4.
template <typename T, int N> int combine_backward_n(const MoveArgs &a, hipStream_t s) {
    const int64_t vectors = (a.dim + N - 1) / N;
    int lanes_log2 = 0;
    while (lanes_log2 < 6 && (int64_t(2) << lanes_log2) <= vectors) ++lanes_log2;
    const int64_t a_lane = (vectors + (1 << lanes_log2) - 1) >> lanes_log2;
    const int64_t choices = kBackwardThreads >> lanes_log2;  // a workgroup
    const int64_t parts = (a.tokens * a.choices + choices - 1) / choices;
    const int64_t pads = pad_blocks(a.capacity);
    const FastDiv by = fast_div((uint32_t)a.choices);
    return in_launches(pads + parts, kBackwardThreads, [&](uint32_t nb, int64_t b0) {
        const auto launch = [&](auto kernel) {
            hipLaunchKernelGGL(kernel, dim3(nb), dim3(kBackwardThreads), 0, s, a, by, lanes_log2,
                               (uint32_t)pads, (uint32_t)b0);
        };
        if (lanes_log2 < 6)
            launch(bmmc_expert_combine_backward_kernel<T, N, 2, false>);
        else if (a_lane <= 1)
            launch(bmmc_expert_combine_backward_kernel<T, N, 1, true>);
        else if (a_lane <= 2)
            launch(bmmc_expert_combine_backward_kernel<T, N, 2, true>);
        else
            launch(bmmc_expert_combine_backward_kernel<T, N, 4, true>);
    });
}

// Rows of whole cache lines are streamed out, others written through the caches,
// which put the lines that two rows share together: 16384 tokens of 8 choices
// gather rows of 4094 bytes in 131 us, 146 streamed; rows of 4096 bytes in 118 us
// and 102 streamed.
//
// Rows by expert that the caches can still hold since they were written are
// read through them, more are streamed in.  Combine and its backward pass, 8
// choices of 4 KiB a token: 67 MB of rows 14.0 and 24.2 us cached, 16.0 and 28.0
// streamed; 98 MB 20.4 and 41.4, 20.5 and 39.1; 134 MB 29.4 and 55.1, 26.7 and 51.6.
MoveArgs with_hints(MoveArgs a, int type) {
    constexpr int64_t kLine = 128;
    const int64_t size = type == BMMC_F32 ? 4 : 2;
    a.whole_lines = (int64_t)((uintptr_t)a.out % kLine) == 0 &&
                    a.out_stride * size % kLine == 0 && a.dim * size % kLine == 0;
    a.stream = a.capacity * a.dim > kMoveCached / size;
    return a;
}

// Whole vectors, or single elements for rows of less than one.
#define BMMC_BY_WIDTH(call, T, a, s)                                                  \
    ((a).dim >= dev::Lanes<T>::N ? call<T, dev::Lanes<T>::N>((a), (s)) : call<T, 1>((a), (s)))

}  // namespace

int launch_expert_gather(const MoveArgs &args, int type, hipStream_t s) {
    const MoveArgs a = with_hints(args, type);
    // rows are copied as they are: 16-bit types share one kernel
    return type == BMMC_F32 ? BMMC_BY_WIDTH(gather_n, float, a, s)
                            : BMMC_BY_WIDTH(gather_n, dev::f16_t, a, s);
}

int launch_expert_combine(const MoveArgs &args, int type, hipStream_t s) {
    const MoveArgs a = with_hints(args, type);
    switch (type) {
    case BMMC_F32: return BMMC_BY_WIDTH(combine_n, float, a, s);
    case BMMC_F16: return BMMC_BY_WIDTH(combine_n, dev::f16_t, a, s);
    default: return BMMC_BY_WIDTH(combine_n, dev::bf16_t, a, s);
    }
}

int launch_expert_combine_backward(const MoveArgs &args, int type, hipStream_t s) {
    const MoveArgs a = with_hints(args, type);
    switch (type) {
    case BMMC_F32: return BMMC_BY_WIDTH(combine_backward_n, float, a, s);
    case BMMC_F16: return BMMC_BY_WIDTH(combine_backward_n, dev::f16_t, a, s);
    default: return BMMC_BY_WIDTH(combine_backward_n, dev::bf16_t, a, s);
    }
}

}  // namespace bmmc
