// block_quantize.hpp -- rows to 8-bit floating point (e4m3) with a scale for each block of 128
// columns of a row (activations) or of 128 x 128 elements (weights), gfx950.
//
// A block's scale is s = fl32(max|x| / 448), 448 the largest e4m3 value, and q is the exact
// quotient x / s rounded to the nearest e4m3 value, halves to even: q is a function of x and s
// alone.  A block of zeros (or one so small that its scale underflows to 0) has s = 0 and
// q = 0; a block that holds an infinity or NaN has s = NaN and q = 0.
//
// t = fl(x r), r the hardware's reciprocal of s (one unit off), is within 3 units in its last place
// of x / s, so rounding t is right unless x / s lies that close to a point half way between two
// e4m3 values.  Those points have bits 0x80000 below the three kept ones, in t itself or, under
// 2^-6 where e4m3 is evenly spaced by 2^-9, in t + 2^-6.  A value found within 8 units of such a
// point h is put on it or beside it by the sign of x - h s, which one fused step has exactly (h
// has 5 digits, s 24, and s >= 2^-100 keeps the difference from underflowing).  About 1 value in
// 60,000 of random binary32 ones is, but in bf16 6 in 100 where the block's largest is 7 times a
// short number.  Where s is smaller, the quotient is taken in binary64 (it differs from h by
// 2^-29 relative at least or not at all, so that decides as the exact one).
//
// The pass is bound by memory: x read once, held in registers between the largest magnitude
// and the rounding (28672x8192 bf16, calls in a row: 136 us in square blocks, 5.2 TB/s, 144 us by rows,
// 8192x8192 45 us; 1x8192 3.1 us in the kernel).  With about 20 instructions an element the units are busy
// a third of that time, which is why the exact quotients above are kept off the common path.
#pragma once

#include "dense.hpp"
#include "reduce.hpp"

namespace qtcq {

struct BlockScale {
    float s, r;
    bool tiny;      // s so small that 1 / s or x / s may leave binary32 (and not 0)
    bool zero;      // every q is 0 (s is 0 or NaN)
};

// amax: the block's largest |x| as its binary32 bits
__device__ __forceinline__ BlockScale block_scale(uint32_t amax)
{
    BlockScale o;
    const bool finite = amax < 0x7F800000u;
    const float m = __builtin_bit_cast(float, amax);
    // m / 448 rounded right: with y the constant's rounded reciprocal and q = fl(m y), q + y (m - 448 q)
    // in two fused steps, as long as nothing underflows
    constexpr float y = 1.0f / 448.0f;
    const float q = m * y;
    o.s = __builtin_fmaf(__builtin_fmaf(-448.0f, q, m), y, q);
    if (__builtin_expect(m < 0x1p-90f, 0)) o.s = m / 448.0f;
    o.s = finite ? o.s : __builtin_nanf("");
    o.zero = !finite || o.s == 0.0f;
    o.tiny = !o.zero && o.s < 0x1p-100f;
    o.r = __builtin_amdgcn_rcpf(o.s);
    return o;
}

// x / s rounded to e4m3 in binary64, as a float that holds it
__device__ __forceinline__ float e4m3_of_quotient(float x, float s)
{
    double v = __builtin_fabs((double)x / (double)s);
    v = v < 448.0 ? v : 448.0;
    int e = (int)(__builtin_bit_cast(uint64_t, v) >> 52) - 1023;
    e = e < -6 ? -6 : e;
    const double step = __builtin_bit_cast(double, (uint64_t)(e - 3 + 1023) << 52);
    const double inv = __builtin_bit_cast(double, (uint64_t)(3 - e + 1023) << 52);
    return __builtin_copysignf((float)(rint(v * inv) * step), x);
}

// |t|, moved to where points half way between e4m3 values have the bits 0x80000 below the kept ones
__device__ __forceinline__ uint32_t placed(float t)
{
    const float a = __builtin_fabsf(t);
    return __builtin_bit_cast(uint32_t, a < 0x1p-6f ? a + 0x1p-6f : a);
}

// t, or if it is within 8 units of such a point h: h or a neighbour on the side of x / s, by the
// sign of x - h s
__device__ __forceinline__ float off_half_way(float t, float x, float s)
{
    const uint32_t b = placed(t), d = (b + 0x80008u) & 0xFFFFFu;
    const float w = __builtin_bit_cast(float, b + 8u - d);
    const float h = __builtin_fabsf(t) < 0x1p-6f ? w - 0x1p-6f : w;
    const float over = __builtin_fmaf(-h, s, __builtin_fabsf(x));
    const uint32_t side = __builtin_bit_cast(uint32_t, h) + (over > 0.0f ? 1u : 0u) - (over < 0.0f ? 1u : 0u);
    return d <= 16u ? __builtin_copysignf(__builtin_bit_cast(float, side), x) : t;
}

// N values (a multiple of 4) to e4m3, four to a word.
template <int N>
__device__ __forceinline__ void to_e4m3(const float (&x)[N], const BlockScale& o, uint32_t (&w)[N / 4])
{
    float t[N];
    uint32_t near = ~0u;
#pragma unroll
    for (int e = 0; e < N; ++e) {
        t[e] = x[e] * o.r;
        // how far past 8 units below the half way point, times 2^12
        const uint32_t d = (placed(t[e]) << 12) + 0x80008000u;
        near = d < near ? d : near;
    }
    if (__builtin_expect(o.tiny || o.zero, 0)) {
#pragma unroll
        for (int e = 0; e < N; ++e) t[e] = o.zero ? 0.0f : e4m3_of_quotient(x[e], o.s);
    } else if (near <= 16u << 12) {
#pragma unroll
        for (int e = 0; e < N; ++e) t[e] = off_half_way(t[e], x[e], o.s);
    }
#pragma unroll
    for (int g = 0; g < N / 4; ++g) {
        int v = __builtin_amdgcn_cvt_pk_fp8_f32(t[4 * g], t[4 * g + 1], 0, false);
        w[g] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(t[4 * g + 2], t[4 * g + 3], v, true);
    }
}

// Sixteen elements of a row, the piece of one thread, as they are in memory.
template <typename T>
struct Sixteen {
    static constexpr int E = 16 / (int)sizeof(T), C = 16 / E;     // elements a chunk, chunks
    u32x4 v[C];

    // from element `at` of a row of n, zero past its end
    __device__ __forceinline__ void load(const T* row, int at, int n)
    {
#pragma unroll
        for (int c = 0; c < C; ++c) v[c] = at + c * E < n ? load_chunk<T>(row, at + c * E, n) : u32x4{0u, 0u, 0u, 0u};
    }
    // the largest magnitude as binary32 bits (an infinity or NaN is above every finite value)
    __device__ __forceinline__ uint32_t largest() const
    {
        uint32_t m = 0;
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if constexpr (sizeof(T) == 2) {
                    m = pair_max(m, v[c][e]);
                } else {
                    const uint32_t a = v[c][e] & 0x7FFFFFFFu;
                    m = a > m ? a : m;
                }
            }
        if constexpr (sizeof(T) == 2) {
            const uint32_t h = (m & 0xFFFFu) > (m >> 16) ? m & 0xFFFFu : m >> 16;
            m = abs_bits(to_f32(__builtin_bit_cast(T, (uint16_t)h)));
        }
        return m;
    }
    __device__ __forceinline__ u32x4 rounded(const BlockScale& o) const
    {
        struct Chunk { T e[E]; };
        float x[16];
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int e = 0; e < E; ++e) x[c * E + e] = to_f32(__builtin_bit_cast(Chunk, v[c]).e[e]);
        uint32_t w[4];
        to_e4m3(x, o, w);
        return u32x4{w[0], w[1], w[2], w[3]};
    }
};

// bytes of a row from `at`, those inside its n
__device__ __forceinline__ void store_sixteen(uint8_t* row, int at, int n, u32x4 v)
{
    struct __attribute__((packed)) Loose { u32x4 v; };
    if (at + 16 <= n) {
        reinterpret_cast<Loose*>(row + at)->v = v;
        return;
    }
#pragma unroll
    for (int e = 0; e < 16; ++e)
        if (at + e < n) row[at + e] = (uint8_t)(v[e >> 2] >> (8 * (e & 3)));
}

// Blocks of one row: eight threads of 16 elements each a block, 8 rows by 4 blocks a
// workgroup, so that the scales of adjacent rows, which the product reads together, are
// written together.
//   workgroup b of strips * ceil(rows / 8), strips = ceil(cols / 512), in turn; block = 256
struct BlockQuantShape {
    static constexpr int kThreads = 256;
    static constexpr int kRows = 8;
    static constexpr int kCols = 512;
};

template <typename T>
__global__ void __launch_bounds__(BlockQuantShape::kThreads)
quantize_row_blocks(const T* __restrict__ x, int64_t rows, int cols, int64_t ldx, uint8_t* __restrict__ q, int64_t ldq,
                    float* __restrict__ scale, int64_t scale_row, int64_t scale_col, unsigned groups)
{
    const unsigned strips = (unsigned)(cols + BlockQuantShape::kCols - 1) / BlockQuantShape::kCols;
    for (unsigned b = blockIdx.x; b < groups; b += gridDim.x) {
        const unsigned band = b / strips;
        const int64_t row = (int64_t)band * BlockQuantShape::kRows + (threadIdx.x >> 5);
        const int col = (int)(b - band * strips) * BlockQuantShape::kCols + (threadIdx.x & 31) * 16;
        const int n = row < rows ? cols : 0;
        Sixteen<T> v;
        v.load(x + (row < rows ? row : 0) * ldx, col, n);
        const BlockScale sc = block_scale(max_of_8(v.largest()));
        if (col >= n) continue;
        if ((threadIdx.x & 7) == 0) scale[row * scale_row + (col >> 7) * scale_col] = sc.s;
        store_sixteen(q + row * ldq, col, n, v.rounded(sc));
    }
}

// Blocks of 128 x 128: a workgroup a block, 32 rows at a time, held in registers.
//   workgroup b of ceil(cols / 128) * ceil(rows / 128), in turn; block = 256
template <typename T>
__global__ void __launch_bounds__(BlockQuantShape::kThreads)
quantize_square_blocks(const T* __restrict__ x, int64_t rows, int cols, int64_t ldx, uint8_t* __restrict__ q, int64_t ldq,
                       float* __restrict__ scale, int64_t scale_row, int64_t scale_col, unsigned groups)
{
    __shared__ uint32_t red[2][BlockQuantShape::kThreads / 64];
    const unsigned wide = (unsigned)(cols + 127) / 128;
    int turn = 0;
    for (unsigned b = blockIdx.x; b < groups; b += gridDim.x, turn ^= 1) {
        const unsigned band = b / wide;
        const int64_t row0 = (int64_t)band * 128 + (threadIdx.x >> 3);
        const int col = (int)(b - band * wide) * 128 + (threadIdx.x & 7) * 16;
        Sixteen<T> v[4];
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t row = row0 + 32 * i;
            v[i].load(x + (row < rows ? row : 0) * ldx, col, row < rows ? cols : 0);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t a = v[i].largest();
            m = a > m ? a : m;
        }
        m = wave_max(m);
        // two sets of partial results in turn: a wave may be a block ahead of another's reads
        if ((threadIdx.x & 63) == 0) red[turn][threadIdx.x >> 6] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < BlockQuantShape::kThreads / 64; ++w) m = red[turn][w] > m ? red[turn][w] : m;
        const BlockScale sc = block_scale(m);
        if (threadIdx.x == 0) scale[band * scale_row + (col >> 7) * scale_col] = sc.s;
        if (col >= cols) continue;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t row = row0 + 32 * i;
            if (row < rows) store_sixteen(q + row * ldq, col, cols, v[i].rounded(sc));
        }
    }
}

}  // namespace qtcq
