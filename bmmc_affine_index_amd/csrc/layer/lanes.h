// lanes.h -- a number of each lane joined with the other lanes' (gfx950).
//
// Lanes of a row of 16 exchange by data-parallel moves of the vector unit, rows
// and halves of a wave by its swaps: none of it goes through LDS, as a shuffle
// does.  All lanes of the wave take part; partners join the same two numbers, so
// that all of them get the same result.
#pragma once

#include <hip/hip_runtime.h>

namespace bmmc {
namespace dev {

struct Largest {
    __device__ __forceinline__ float operator()(float a, float b) const { return fmaxf(a, b); }
};
struct Sum {
    __device__ __forceinline__ float operator()(float a, float b) const { return a + b; }
};

template <int MOVE, class Op> __device__ __forceinline__ float in_16(float v, Op op) {
    const uint32_t w = __builtin_bit_cast(uint32_t, v);
    return op(v, __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0u, w, MOVE, 0xf, 0xf, true)));
}
// with the lane 16 (32) away
template <class Op> __device__ __forceinline__ float over_16(float v, Op op) {
    const uint32_t w = __builtin_bit_cast(uint32_t, v);
    const auto both = __builtin_amdgcn_permlane16_swap(w, w, false, false);
    return op(__builtin_bit_cast(float, (uint32_t)both[0]), __builtin_bit_cast(float, (uint32_t)both[1]));
}
template <class Op> __device__ __forceinline__ float over_32(float v, Op op) {
    const uint32_t w = __builtin_bit_cast(uint32_t, v);
    const auto both = __builtin_amdgcn_permlane32_swap(w, w, false, false);
    return op(__builtin_bit_cast(float, (uint32_t)both[0]), __builtin_bit_cast(float, (uint32_t)both[1]));
}

// Over the 1 << shift lanes that lie together; shift is the same in all lanes.
template <class Op> __device__ __forceinline__ float over_lanes(float v, int shift, Op op) {
    if (shift > 0) v = in_16<0xb1>(v, op);   // lanes 1 0 3 2 of four
    if (shift > 1) v = in_16<0x4e>(v, op);   // lanes 2 3 0 1
    if (shift > 2) v = in_16<0x141>(v, op);  // 8 lanes the other way round
    if (shift > 3) v = in_16<0x140>(v, op);  // 16 lanes the other way round
    if (shift > 4) v = over_16(v, op);
    if (shift > 5) v = over_32(v, op);
    return v;
}

}  // namespace dev
}  // namespace bmmc
