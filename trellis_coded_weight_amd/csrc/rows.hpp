// rows.hpp -- elements of rows as the operators on rows read and write them, gfx950: 16 bytes of
// T at a time, from any element on.
#pragma once

#include "dense.hpp"

namespace qtcq {

template <typename T, int E>
struct Elems { T e[E]; };

// E elements at `at` of a row of n, `fill` past its end
template <typename T, int E>
__device__ __forceinline__ Elems<T, E> load_elems(const T* row, int at, int n, T fill)
{
    struct __attribute__((packed, aligned(sizeof(T)))) Loose { Elems<T, E> v; };
    if (at + E <= n) return reinterpret_cast<const Loose*>(row + at)->v;
    Elems<T, E> o;
#pragma unroll
    for (int e = 0; e < E; ++e) o.e[e] = at + e < n ? row[at + e] : fill;
    return o;
}

// The elements of 16 bytes in binary32.
template <typename T>
__device__ __forceinline__ void unpack(u32x4 v, float (&o)[16 / sizeof(T)])
{
    typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (std::is_same_v<T, __bf16>) {
            o[2 * i] = __builtin_bit_cast(float, v[i] << 16);
            o[2 * i + 1] = __builtin_bit_cast(float, v[i] & 0xFFFF0000u);
        } else if constexpr (std::is_same_v<T, _Float16>) {
            const f16x2 h = __builtin_bit_cast(f16x2, (uint32_t)v[i]);
            o[2 * i] = (float)h.x;
            o[2 * i + 1] = (float)h.y;
        } else {
            o[i] = __builtin_bit_cast(float, (uint32_t)v[i]);
        }
    }
}

// Their rounding, once each, to nearest even.
template <typename T>
__device__ __forceinline__ u32x4 pack(const float (&v)[16 / sizeof(T)])
{
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    u32x4 o;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (std::is_same_v<T, __bf16>) {
            o[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{v[2 * i], v[2 * i + 1]}, bf16x2));
        } else if constexpr (std::is_same_v<T, _Float16>) {
            // the binary32 values as computed, as from_f32 has it
            float a = v[2 * i], b = v[2 * i + 1];
            asm("" : "+v"(a), "+v"(b));
            o[i] = (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)a) | (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)b) << 16;
        } else {
            o[i] = __builtin_bit_cast(uint32_t, v[i]);
        }
    }
    return o;
}

// 16 bytes to p, which need only be aligned to their element
template <typename T>
__device__ __forceinline__ void store_loose(T* p, u32x4 v)
{
    struct __attribute__((packed, aligned(sizeof(T)))) Loose { u32x4 v; };
    reinterpret_cast<Loose*>(p)->v = v;
}

// the elements of a chunk at `at` of a row of n that are inside it
template <typename T>
__device__ __forceinline__ void store_chunk(T* row, int at, int n, u32x4 v)
{
    constexpr int E = 16 / (int)sizeof(T);
    if (at + E <= n) {
        store_loose(row + at, v);
        return;
    }
    const Elems<T, E> o = __builtin_bit_cast(Elems<T, E>, v);
#pragma unroll
    for (int e = 0; e < E; ++e)
        if (at + e < n) row[at + e] = o.e[e];
}

// 16 bytes at `at` of a row of n, `fill` past its end
template <typename T>
__device__ __forceinline__ u32x4 load_filled(const T* row, int at, int n, T fill)
{
    return __builtin_bit_cast(u32x4, load_elems<T, 16 / (int)sizeof(T)>(row, at, n, fill));
}

}  // namespace qtcq
