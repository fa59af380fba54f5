// dense.hpp -- element types, roundings and gate activations shared by the dense
// operators (row quantization, decode to rows, 8-bit product, gated projections), gfx950.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

namespace qtcq {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// the activation of the gate (qtcq_activation)
enum : int { kActSilu = 0, kActGelu = 1, kActGeluTanh = 2, kActRelu = 3, kActSigmoid = 4 };

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__bf16 v) { return (float)v; }
__device__ __forceinline__ float to_f32(_Float16 v) { return (float)v; }

// One rounding of the binary32 value, to nearest even (out of fp16's range: infinity).
// The value is kept as computed: without that, a product about to become fp16 turns into a
// v_fma_mixlo_f16, which rounds the exact product once and not the binary32 one.
template <typename T>
__device__ __forceinline__ T from_f32(float v)
{
    if constexpr (sizeof(T) == 2) asm volatile("" : "+v"(v));
    return (T)v;
}

// v as the sum of two values of T, both of v's sign: hi is the largest one below |v| in
// magnitude (in fp16 2^-24 below at least), lo the rest, rounded.  Their sum is within 2^-15 (bf16) or 2^-21 (fp16, and
// 2^-25 absolute) of v, and a v of up to 131008 stays finite in fp16.  hi stays below |v| also
// where v itself is a value of T, so that lo is not 0 where hi is not: an infinite factor
// then gives v's infinity twice and not inf + 0 * inf.  (Not so for |v| under 2^-110 in bf16,
// 2^-23 in fp16.)  0, infinities and NaN are both parts.
template <typename T>
__device__ __forceinline__ void two_parts(float v, T& hi, T& lo)
{
    const uint32_t b = __builtin_bit_cast(uint32_t, v), mag = b & 0x7FFFFFFFu;
    const float below = __builtin_bit_cast(float, mag - 1u);
    float h;
    if constexpr (std::is_same_v<T, __bf16>) {
        h = __builtin_bit_cast(float, (mag - 1u) & 0xFFFF0000u);
    } else {
        // 2^-24 below |v| at least, half of which would round to a lo of 0; then toward zero:
        // the mantissa's upper 10 bits, or whole multiples of 2^-24 under 2^-14
        float u = __builtin_fminf(below, __builtin_bit_cast(float, mag) - 0x1p-24f);
        u = __builtin_fminf(__builtin_fmaxf(u, 0.0f), 65504.0f);
        h = u >= 0x1p-14f ? __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, u) & 0xFFFFE000u)
                          : __builtin_truncf(u * 0x1p24f) * 0x1p-24f;
    }
    const bool whole = mag == 0u || mag >= 0x7F800000u;
    h = whole ? v : __builtin_copysignf(h, v);
    hi = (T)h;
    lo = whole ? hi : from_f32<T>(v - h);
}

// 16 bytes at p, which need only be aligned to their element
template <typename T>
__device__ __forceinline__ u32x4 load_loose(const T* p)
{
    struct __attribute__((packed, aligned(sizeof(T)))) Loose { u32x4 v; };
    return reinterpret_cast<const Loose*>(p)->v;
}

// 16 bytes at p + at of a row with n elements, zero past its end
template <typename T>
__device__ __forceinline__ u32x4 load_chunk(const T* p, int at, int n)
{
    constexpr int E = 16 / (int)sizeof(T);
    if (at + E <= n) return load_loose(p + at);
    struct Parts { T e[E]; } o;
#pragma unroll
    for (int e = 0; e < E; ++e) o.e[e] = at + e < n ? p[at + e] : (T)0;
    return __builtin_bit_cast(u32x4, o);
}

// sigmoid(g) = 1 / (1 + exp(-g)) and its complement sigmoid(-g), from the hardware's exp2 and
// reciprocal (one unit in the last place each; the rounding of g log2 e adds a few |g| 2^-24
// relative): far below the roundings of the 16-bit operands and results, and a seventh of the
// instructions of the full-precision ones.  With e = exp(-|g|) the larger of the two is
// 1 / (1 + e) and the smaller e / (1 + e), so neither is a difference that loses its digits,
// and nothing overflows.  e is the square of exp(-|g| / 2), as the hardware's exp2 flushes
// results below 2^-126 to 0, which g sigmoid(g) may still exceed; it is 0 itself below 2^-149.
__device__ __forceinline__ void sigmoids_f32(float g, float& s, float& c)
{
    const float h = __builtin_amdgcn_exp2f(-0.72134752044448170f * __builtin_fabsf(g)), e = h * h;
    const float r = __builtin_amdgcn_rcpf(1.0f + e), t = e * r;
    s = g < 0.0f ? t : r;
    c = g < 0.0f ? r : t;
}

__device__ __forceinline__ float sigmoid_f32(float g)
{
    float s, c;
    sigmoids_f32(g, s, c);
    return s;
}

constexpr float kGeluTanhC = 1.5957691216057308f;        // 2 sqrt(2 / pi)
constexpr float kGeluTanhC3 = 0.0713548162726009f;       // 0.044715 * 2 sqrt(2 / pi)

// act(g).  gelu_tanh: g (1 + tanh z) / 2 = g sigmoid(2 z), z = sqrt(2 / pi) (g + 0.044715 g^3).
template <int ACT>
__device__ __forceinline__ float activate(float g)
{
    if constexpr (ACT == kActSilu) return g * sigmoid_f32(g);
    if constexpr (ACT == kActGelu) return 0.5f * g * erfcf(-0.7071067811865476f * g);
    if constexpr (ACT == kActGeluTanh) return g * sigmoid_f32(g * (kGeluTanhC + kGeluTanhC3 * g * g));
    if constexpr (ACT == kActRelu) return g < 0.0f ? 0.0f : g;            // NaN stays NaN
    return sigmoid_f32(g);
}

// act(g) and act'(g).  A saturated sigmoid times a large g: its complement underflows to 0
// before their product can matter.  An infinite g, which may be a finite one that the type it
// was saved in does not hold, has the limits of both: the slope is taken at the largest
// finite g of its sign, and so is act at -infinity.
template <int ACT>
__device__ __forceinline__ void activate_grad(float gate, float& a, float& d)
{
    const float g = __builtin_fabsf(gate) == __builtin_inff() ? __builtin_copysignf(0x1.fffffep127f, gate) : gate;
    float s, c;
    if constexpr (ACT == kActSilu) {
        sigmoids_f32(g, s, c);
        a = g * s;
        d = s * (1.0f + g * c);
    } else if constexpr (ACT == kActGelu) {
        c = 0.5f * erfcf(-0.7071067811865476f * g);
        a = g * c;
        d = c + g * (0.3989422804014327f * expf(-0.5f * g * g));
    } else if constexpr (ACT == kActGeluTanh) {
        sigmoids_f32(g * (kGeluTanhC + kGeluTanhC3 * g * g), s, c);
        a = g * s;
        // g^2 s (1 - s): the polynomial's slope multiplies s (1 - s) before g, so that a
        // large |g| meets an exact 0
        const float t = s * c;
        d = t == 0.0f ? s : s + g * t * (kGeluTanhC + 3.0f * kGeluTanhC3 * g * g);
    } else if constexpr (ACT == kActRelu) {
        a = g < 0.0f ? 0.0f : g;
        d = g > 0.0f ? 1.0f : (g == g ? 0.0f : g);
    } else {
        sigmoids_f32(g, s, c);
        a = s;
        d = s * c;
    }
    if constexpr (ACT != kActSigmoid) a = gate == __builtin_inff() ? gate : a;
}

}  // namespace qtcq
