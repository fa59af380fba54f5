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

// Where a thread's chunk c of a row of n elements is read: whole chunks where they are, and a
// last one that is not whole as the row's last 16 bytes, which `behind` then shifts into place.
// So every load of a row is one instruction with no branch around it (n >= E).
struct Place { int at, bits; };
template <typename T>
__device__ __forceinline__ Place place_of(int c, int n)
{
    constexpr int E = 16 / (int)sizeof(T);
    const int at = c * E, over = at + E - n;
    return over <= 0 ? Place{at, 0} : Place{n - E, over < E ? over * 8 * (int)sizeof(T) : 128};
}

// v without its first `bits` bits (0 to 128), zeros behind
__device__ __forceinline__ u32x4 behind(u32x4 v, int bits)
{
    typedef uint64_t u64x2 __attribute__((ext_vector_type(2)));
    u64x2 o = __builtin_bit_cast(u64x2, v);
    const int b = bits & 63;
    const uint64_t lo = o.x >> b | (o.y << 1) << (63 - b), hi = o.y >> b;
    o.x = bits < 64 ? lo : (bits < 128 ? hi : 0u);
    o.y = bits < 64 ? hi : 0u;
    return __builtin_bit_cast(u32x4, o);
}

// a row of fewer than E elements, zeros behind it
template <typename T>
__device__ __forceinline__ u32x4 load_short(const T* row, int n)
{
    constexpr int BITS = 8 * (int)sizeof(T);
    typedef uint64_t u64x2 __attribute__((ext_vector_type(2)));
    u64x2 v = {0u, 0u};
#pragma unroll 1
    for (int e = n - 1; e >= 0; --e) {
        uint64_t o;
        if constexpr (sizeof(T) == 2)
            o = __builtin_bit_cast(uint16_t, row[e]);
        else
            o = __builtin_bit_cast(uint32_t, row[e]);
        v.y = v.y << BITS | v.x >> (64 - BITS);
        v.x = v.x << BITS | o;
    }
    return __builtin_bit_cast(u32x4, v);
}

// chunk c of a row of n elements, zeros behind it
template <typename T>
__device__ __forceinline__ u32x4 load_zero(const T* row, int c, int n)
{
    if (n < 16 / (int)sizeof(T)) return load_short(row, n);
    const Place p = place_of<T>(c, n);
    return behind(load_loose(row + p.at), p.bits);
}

// 16 bytes at `at` of a row of n, `fill` past its end
template <typename T>
__device__ __forceinline__ u32x4 load_filled(const T* row, int at, int n, T fill)
{
    return __builtin_bit_cast(u32x4, load_elems<T, 16 / (int)sizeof(T)>(row, at, n, fill));
}

}  // namespace qtcq
