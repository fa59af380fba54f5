// reduce.hpp -- reductions over the lanes and waves of a workgroup, shared by the operators on
// rows, gfx950.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

namespace qtcq {

__device__ __forceinline__ uint32_t abs_bits(float v) { return __builtin_bit_cast(uint32_t, v) & 0x7FFFFFFFu; }

// Largest of m over the wave's 64 lanes.
__device__ __forceinline__ uint32_t wave_max(uint32_t m)
{
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
        const uint32_t v = (uint32_t)__shfl_xor((int)m, o, 64);
        m = v > m ? v : m;
    }
    return m;
}

// The larger of |x| over both halves of 16-bit pairs, as 16-bit patterns (an infinity or NaN
// is above every finite value).
__device__ __forceinline__ uint32_t pair_max(uint32_t m, uint32_t pair)
{
    typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, m),
                                                                  __builtin_bit_cast(u16x2, pair & 0x7FFF7FFFu)));
}

// Largest of m over each aligned group of 8 lanes (all of them active).
__device__ __forceinline__ uint32_t max_of_8(uint32_t m)
{
    auto with = [&](auto ctrl) {
        const uint32_t v = (uint32_t)__builtin_amdgcn_mov_dpp((int)m, decltype(ctrl)::value, 0xF, 0xF, true);
        m = v > m ? v : m;
    };
    with(std::integral_constant<int, 0xB1>{});      // lane ^ 1
    with(std::integral_constant<int, 0x4E>{});      // lane ^ 2
    with(std::integral_constant<int, 0x141>{});     // 7 - lane: the other four
    return m;
}

// Sum of v over the wave's 64 lanes, the same in all of them.
__device__ __forceinline__ float wave_sum(float v)
{
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
    return v;
}

}  // namespace qtcq
