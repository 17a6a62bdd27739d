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
// Bound by latency: it reads 4 or 8 bytes and writes 8 for each choice.
#include "tokens.h"

namespace bmmc {

namespace {

constexpr int kOrderThreads = 1024;
// Counters per wave and expert: 16 waves up to 1024 experts, 8 beyond, so
// that the counters fill at most 64 KiB of LDS.
constexpr int kOrderWideExperts = 1024;

__device__ __forceinline__ int32_t expert_at(const OrderArgs &a, int64_t i) {
    if (a.is64) {
        const int64_t e = static_cast<const int64_t *>(a.experts)[i];
        return e >= 0 && e < a.num_experts ? (int32_t)e : -1;
    }
    const int32_t e = static_cast<const int32_t *>(a.experts)[i];
    return e >= 0 && e < a.num_experts ? e : -1;
}

// Choices of each expert in each chunk.
__global__ void __launch_bounds__(kOrderThreads)
    bmmc_expert_count_kernel(const OrderArgs a) {
    extern __shared__ int32_t cnt[];
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
__device__ __forceinline__ int32_t block_scan(int32_t v, int32_t *wsum, int32_t *total) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
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
    for (int w = 0; w < waves; ++w) {
        const int32_t s = wsum[w];
        before += w < wave ? s : 0;
        all += s;
    }
    *total = all;
    return before + inc - v;
}

// Rows of every choice of this workgroup's chunk.  MANY: the other chunks'
// counts come from a.hist.
template <bool MANY>
__global__ void __launch_bounds__(kOrderThreads) bmmc_expert_place_kernel(const OrderArgs a) {
    extern __shared__ int32_t cnt[];  // [waves][num_experts]
    __shared__ int32_t wsum[16];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, waves = blockDim.x >> 6;
    const int E = a.num_experts;
    for (int i = tid; i < waves * E; i += blockDim.x) cnt[i] = 0;
    __syncthreads();

    // each wave's piece of the chunk, in order
    const int64_t from = blockIdx.x * a.chunk;
    const int64_t to = min(from + a.chunk, a.n);
    const int64_t rounds = (a.chunk + 64 * waves - 1) / (64 * waves);
    const int64_t mine = from + wave * rounds * 64;
    int32_t *my = cnt + wave * E;
    for (int64_t r = 0; r < rounds; ++r) {
        const int64_t i = mine + r * 64 + lane;
        const int32_t e = i < to ? expert_at(a, i) : -1;
        if (e >= 0) atomicAdd(&my[e], 1);
    }
    __syncthreads();

    // first row of each wave's choices of each expert
    int64_t start = 0;
    for (int e0 = 0; e0 < E; e0 += blockDim.x) {
        const int e = e0 + tid;
        int32_t here = 0, before = 0, all = 0;
        if (e < E) {
            for (int w = 0; w < waves; ++w) {
                const int32_t c = cnt[w * E + e];
                cnt[w * E + e] = here;
                here += c;
            }
            all = here;
            if constexpr (MANY) {
                all = 0;
                for (int b = 0; b < (int)gridDim.x; ++b) {
                    const int32_t c = a.hist[(int64_t)b * E + e];
                    before += b < (int)blockIdx.x ? c : 0;
                    all += c;
                }
            }
        }
        const int32_t padded = (int32_t)((all + a.align - 1) / a.align * a.align);
        int32_t sum;
        const int32_t off = (int32_t)start + block_scan(padded, wsum, &sum);
        start += sum;
        if (e < E) {
            for (int w = 0; w < waves; ++w) cnt[w * E + e] += off + before;
            if (blockIdx.x == 0) {
                a.offsets[e] = off;
                a.counts[e] = all;
                for (int32_t r = off + all; r < off + padded; ++r) a.slots[r] = -1;
            }
        }
    }
    if (blockIdx.x == 0 && tid == 0) a.offsets[E] = (int32_t)start;
    // rows past the last expert's
    for (int64_t r = start + (int64_t)blockIdx.x * blockDim.x + tid; r < a.capacity;
         r += (int64_t)gridDim.x * blockDim.x)
        a.slots[r] = -1;
    __syncthreads();

    const int bits = 32 - __clz(E);  // of the numbers 0 .. E
    for (int64_t r = 0; r < rounds; ++r) {
        const int64_t i = mine + r * 64 + lane;
        if (mine + r * 64 >= to) break;
        const int32_t e = i < to ? expert_at(a, i) : -1;
        const uint32_t key = e >= 0 ? (uint32_t)e : (uint32_t)E;
        uint64_t same = ~uint64_t(0);
        for (int b = 0; b < bits; ++b) {
            const uint64_t set = __ballot((key >> b) & 1u);
            same &= ((key >> b) & 1u) ? set : ~set;
        }
        const int rank = __popcll(same & ((uint64_t(1) << lane) - 1));
        int32_t row = -1;
        if (e >= 0) {
            row = __hip_atomic_load(&my[e], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP) + rank;
        }
        // every lane has read before the last lane of each expert writes
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        if (e >= 0) {
            if ((same >> lane) == 1)
                __hip_atomic_store(&my[e], row + 1, __ATOMIC_RELAXED,
                                   __HIP_MEMORY_SCOPE_WORKGROUP);
            a.slots[row] = (int32_t)i;
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        if (i < to) a.rows[i] = row;
    }
}

}  // namespace

int launch_expert_order(const OrderArgs &a, int blocks, hipStream_t s) {
    const int threads = a.num_experts > kOrderWideExperts ? kOrderThreads / 2 : kOrderThreads;
    const size_t lds = sizeof(int32_t) * (size_t)a.num_experts * (threads / 64);
    if (blocks == 1) {
        hipLaunchKernelGGL(bmmc_expert_place_kernel<false>, dim3(1), dim3(threads), lds, s, a);
    } else {
        hipLaunchKernelGGL(bmmc_expert_count_kernel, dim3(blocks), dim3(kOrderThreads),
                           sizeof(int32_t) * (size_t)a.num_experts, s, a);
        hipLaunchKernelGGL(bmmc_expert_place_kernel<true>, dim3(blocks), dim3(threads), lds, s, a);
    }
    return hipGetLastError() == hipSuccess ? BMMC_OK : BMMC_ERR_HIP;
}

}  // namespace bmmc
