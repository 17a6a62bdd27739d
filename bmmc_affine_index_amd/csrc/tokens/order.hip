// order.hip -- choices sorted by expert, stable (gfx950).
//
// A counting sort: with h(b, e) the choices of expert e in part b of the
// array, the first row of part b's choices of e is
//     offset(e) + sum over b' < b of h(b', e),
//     offset(e) = sum over e' < e of the padded sum over b of h(b, e').
// The parts here are the waves' pieces of each workgroup's chunk, so a wave
// places its choices 64 at a time: a lane's rank among the lanes with its
// expert comes from one ballot per bit of the expert's number, and a counter
// per wave and expert in LDS holds how many came before.  Nothing depends on
// the order in which waves run.
//
// Every row counts as padding, slots = -1, until a choice is placed there: the
// rows are filled before, by the launch that counts or by the one workgroup.
//
// Bound by latency: it reads 4 or 8 bytes and writes 8 for each choice, in two
// launches for many choices.  256 choices of 64 experts take 3.1 us, 8192 of 64
// experts 7.8 us, 131072 of 64 experts 9.9 us.
#include "tokens.h"

namespace bmmc {

namespace {

constexpr int kOrderWaves = 16;  // of a workgroup, but for few choices
// Rows that one workgroup fills; more take a launch of their own (200 choices,
// 16520 rows: 4.7 us and 5.0 with that launch, 32904 rows 6.3 and 5.0, which the
// host's time for it outweighs, 65672 rows 9.6 and 5.0).
constexpr int64_t kOrderFill = 1 << 15;

__device__ __forceinline__ int32_t expert_at(const OrderArgs &a, int64_t i) {
    if (a.is64) {
        const int64_t e = static_cast<const int64_t *>(a.experts)[i];
        return e >= 0 && e < a.num_experts ? (int32_t)e : -1;
    }
    const int32_t e = static_cast<const int32_t *>(a.experts)[i];
    return e >= 0 && e < a.num_experts ? e : -1;
}

// This workgroup's share of the rows.
__device__ __forceinline__ void fill_slots(const OrderArgs &a) {
    for (int64_t r = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; r < a.capacity;
         r += (int64_t)gridDim.x * blockDim.x)
        a.slots[r] = -1;
}

__global__ void __launch_bounds__(256) bmmc_expert_fill_kernel(const OrderArgs a) {
    fill_slots(a);
}

// Choices of each expert in each chunk.
__global__ void __launch_bounds__(kOrderWaves * 64)
    bmmc_expert_count_kernel(const OrderArgs a, int fill) {
    extern __shared__ int32_t cnt[];
    if (fill) fill_slots(a);
    const int tid = threadIdx.x;
    for (int e = tid; e < a.num_experts; e += blockDim.x) cnt[e] = 0;
    __syncthreads();
    const int64_t from = blockIdx.x * a.chunk;
    const int64_t to = min(from + a.chunk, a.n);
    for (int64_t i = from + tid; i < to; i += blockDim.x) {
        const int32_t e = expert_at(a, i);
        if (e >= 0) atomicAdd(&cnt[e], 1);
    }
    __syncthreads();
    int32_t *h = a.hist + (int64_t)blockIdx.x * a.num_experts;
    for (int e = tid; e < a.num_experts; e += blockDim.x) h[e] = cnt[e];
}

// Exclusive scan over the workgroup of one value a thread; *total is the sum.
template <int WAVES>
__device__ __forceinline__ int32_t block_scan(int32_t v, int32_t *wsum, int32_t *total) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int32_t inc = v;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int32_t o = __shfl_up(inc, d, 64);
        if (lane >= d) inc += o;
    }
    __syncthreads();  // wsum may still be read from the last scan
    if (lane == 63) wsum[wave] = inc;
    __syncthreads();
    int32_t before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
        const int32_t s = wsum[w];
        before += w < wave ? s : 0;
        all += s;
    }
    *total = all;
    return before + inc - v;
}

// This lane's place among its wave's choices of expert e (-1: none) so far;
// my[e] counts them.
__device__ __forceinline__ int32_t place_in_wave(int32_t *my, int32_t e, int E, int bits) {
    const int lane = threadIdx.x & 63;
    const uint32_t key = e >= 0 ? (uint32_t)e : (uint32_t)E;
    uint64_t same = ~uint64_t(0);
    for (int b = 0; b < bits; ++b) {
        const uint64_t set = __ballot((key >> b) & 1u);
        same &= ((key >> b) & 1u) ? set : ~set;
    }
    int32_t at = -1;
    if (e >= 0)
        at = __hip_atomic_load(&my[e], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP) +
             __popcll(same & ((uint64_t(1) << lane) - 1));
    // every lane has read before the last lane of each expert writes
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    if (e >= 0 && (same >> lane) == 1)
        __hip_atomic_store(&my[e], at + 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    return at;
}

// Sums over the chunks of a.hist for this workgroup's expert e0 + column: of
// those before this chunk and of all.  The threads take the chunks of a column
// in turn, as many threads a column as there are, so that the loads of 64
// chunks and 128 experts are 8 a thread and not 64 in a row (the kernel took
// 20.6 us of 131072 choices with one thread a column).
struct Before {
    int32_t before, all;
};
template <int THREADS>
__device__ __forceinline__ Before sum_chunks(const OrderArgs &a, int e0, int32_t (*part)[THREADS]) {
    const int tid = threadIdx.x, E = a.num_experts;
    const int columns = min(E - e0, THREADS);
    const int threads = THREADS / columns;  // a column
    const int share = tid / columns, e = tid - share * columns;
    int32_t before = 0, all = 0;
    if (share < threads) {
        const int32_t *h = a.hist + e0 + e;
#pragma unroll 4
        for (int b = share; b < (int)gridDim.x; b += threads) {
            const int32_t c = h[(int64_t)b * E];
            before += b < (int)blockIdx.x ? c : 0;
            all += c;
        }
    }
    __syncthreads();  // part may still be read from the last columns
    part[0][tid] = before;
    part[1][tid] = all;
    __syncthreads();
    Before sum{0, 0};
    if (tid < columns)
        for (int s = 0; s < threads; ++s) {
            sum.before += part[0][s * columns + tid];
            sum.all += part[1][s * columns + tid];
        }
    return sum;
}

// Rows of every choice of this workgroup's chunk.  MANY: the other chunks'
// counts come from a.hist.  ROUNDS: choices a lane, kept in registers; 0: as
// many as there are, read a second time.
template <int WAVES, int ROUNDS, bool MANY>
__global__ void __launch_bounds__(WAVES * 64)
    bmmc_expert_place_kernel(const OrderArgs a, int fill) {
    constexpr int kThreads = WAVES * 64;
    extern __shared__ int32_t cnt[];  // [WAVES][num_experts]
    __shared__ int32_t wsum[WAVES];
    __shared__ int32_t part[2][MANY ? kThreads : 1];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int E = a.num_experts;
    const int bits = 32 - __clz(E);  // of the numbers 0 .. E

    // each wave's piece of the chunk, in order
    const int64_t from = blockIdx.x * a.chunk;
    const int64_t to = min(from + a.chunk, a.n);
    const int rounds = (int)((a.chunk + kThreads - 1) / kThreads);
    const int64_t mine = from + (int64_t)wave * rounds * 64 + lane;
    int32_t *my = cnt + wave * E;
    int32_t held[ROUNDS ? ROUNDS : 1], at[ROUNDS ? ROUNDS : 1];
    if constexpr (ROUNDS > 0) {
#pragma unroll
        for (int r = 0; r < ROUNDS; ++r) {
            const int64_t i = mine + r * 64;
            held[r] = r < rounds && i < to ? expert_at(a, i) : -1;
        }
    }
    if (fill) fill_slots(a);
    for (int i = tid; i < WAVES * E; i += kThreads) cnt[i] = 0;
    __syncthreads();
    if constexpr (ROUNDS > 0) {
#pragma unroll
        for (int r = 0; r < ROUNDS; ++r)
            if (r < rounds) at[r] = place_in_wave(my, held[r], E, bits);
    } else {
        for (int r = 0; r < rounds; ++r) {
            const int64_t i = mine + (int64_t)r * 64;
            const int32_t e = i < to ? expert_at(a, i) : -1;
            if (e >= 0) atomicAdd(&my[e], 1);
        }
    }
    __syncthreads();

    // first row of each wave's choices of each expert
    int32_t start = 0;
    for (int e0 = 0; e0 < E; e0 += kThreads) {
        const int e = e0 + tid;
        int32_t here[WAVES], sum = 0;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) here[w] = e < E ? cnt[w * E + e] : 0;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) {
            const int32_t c = here[w];
            here[w] = sum;
            sum += c;
        }
        Before b{0, sum};
        if constexpr (MANY) b = sum_chunks<kThreads>(a, e0, part);
        const int32_t padded =
            e < E ? (int32_t)((b.all + a.align - 1) / a.align * a.align) : 0;
        int32_t total;
        const int32_t off = start + block_scan<WAVES>(padded, wsum, &total);
        start += total;
        if (e < E) {
#pragma unroll
            for (int w = 0; w < WAVES; ++w) cnt[w * E + e] = here[w] + off + b.before;
            if (blockIdx.x == 0) {
                a.offsets[e] = off;
                a.counts[e] = b.all;
            }
        }
    }
    if (blockIdx.x == 0 && tid == 0) a.offsets[E] = start;
    __syncthreads();  // also orders the fill before the choices' stores

    if constexpr (ROUNDS > 0) {
#pragma unroll
        for (int r = 0; r < ROUNDS; ++r) {
            const int64_t i = mine + r * 64;
            if (r >= rounds || i >= to) continue;
            const int32_t row = held[r] >= 0 ? my[held[r]] + at[r] : -1;
            a.rows[i] = row;
            if (row >= 0) a.slots[row] = (int32_t)i;
        }
    } else {
        for (int r = 0; r < rounds; ++r) {
            const int64_t i = mine + (int64_t)r * 64;
            if (i - lane >= to) break;
            const int32_t row = place_in_wave(my, i < to ? expert_at(a, i) : -1, E, bits);
            if (i < to) a.rows[i] = row;
            if (row >= 0) a.slots[row] = (int32_t)i;
        }
    }
}

template <int WAVES, int ROUNDS, bool MANY>
void place(const OrderArgs &a, int blocks, int fill, hipStream_t s) {
    hipLaunchKernelGGL((bmmc_expert_place_kernel<WAVES, ROUNDS, MANY>), dim3(blocks),
                       dim3(WAVES * 64), sizeof(int32_t) * (size_t)a.num_experts * WAVES, s, a,
                       fill);
}

}  // namespace

int launch_expert_order(const OrderArgs &a, int blocks, hipStream_t s) {
    constexpr int kThreads = kOrderWaves * 64;
    constexpr int kRounds = (int)(kOrderOneBlockMax / kThreads);
    const bool apart = a.capacity > kOrderFill * blocks;
    if (apart)
        hipLaunchKernelGGL(bmmc_expert_fill_kernel, dim3((uint32_t)((a.capacity + 4095) / 4096)),
                           dim3(256), 0, s, a);
    if (blocks == 1) {
        // few waves have less to wait for and to sum: 512 choices of 64 experts
        // take 8 waves 3.5 us and 16 waves 4.2
        if (a.n <= 4 * 64)
            place<4, 1, false>(a, 1, !apart, s);
        else if (a.n <= 2 * 8 * 64)
            place<8, 2, false>(a, 1, !apart, s);
        else
            place<kOrderWaves, kRounds, false>(a, 1, !apart, s);
    } else {
        hipLaunchKernelGGL(bmmc_expert_count_kernel, dim3(blocks), dim3(kThreads),
                           sizeof(int32_t) * (size_t)a.num_experts, s, a, !apart);
        if (a.chunk <= kThreads)
            place<kOrderWaves, 1, true>(a, blocks, 0, s);
        else if (a.chunk <= kOrderOneBlockMax)
            place<kOrderWaves, kRounds, true>(a, blocks, 0, s);
        else
            place<kOrderWaves, 0, true>(a, blocks, 0, s);
    }
    return hipGetLastError() == hipSuccess ? BMMC_OK : BMMC_ERR_HIP;
}

}  // namespace bmmc
