// quantize.hpp -- rows to 8-bit integers with one scale a row, from dense rows
// (quantize_rows) and straight from trellis streams (decode_matrix), gfx950.
//
// A row's scale is s = fl32(max|x| / 127) and q = x / s rounded to the nearest integer,
// halves to even, of the exact quotient: the int8 of a value is a function of the value
// and of s alone, whichever path or launch shape computes it.  A row of zeros has s = 0
// and q = 0; a row holding an infinity or NaN has s = NaN and q = 0, so that a product
// with its scale says so.
//
// The exact quotient without a division: with r = fl32(1 / s), u = fma(x, r, 1.5 * 2^23)
// holds the integer nearest to x r in its low bits.  x r is within 2^-17 of x / s
// (|x / s| <= 127), so that integer is right unless x / s lies that close to a half step.
// The residual d = fma(-q, s, x) shows it: |d| < s / 2 proves q (the rounding of d is
// monotone and s / 2 is exact), anything else is settled in binary64, where x - q s is
// exact.  Halves come up only where a value is an odd multiple of s / 2 to 24 bits, so
// the branch is all but never taken.
#pragma once

#include "codes.hpp"
#include "dense.hpp"

namespace qtcq {

// below this s the residual test could meet subnormals: the row is rounded in binary64
constexpr float kQuantTiny = 0x1p-100f;

struct RowScale {
    float s, r, half;
    bool tiny;      // s below kQuantTiny (and not 0)
    bool zero;      // every q is 0 (s is 0 or NaN)
};

// amax: the row's largest |x| as its binary32 bits (an infinity or NaN is above every
// finite value as an integer)
__device__ __forceinline__ RowScale row_scale(uint32_t amax)
{
    RowScale o;
    const bool finite = amax < 0x7F800000u;
    o.s = finite ? __builtin_bit_cast(float, amax) / 127.0f : __builtin_nanf("");
    o.zero = !finite || o.s == 0.0f;
    o.tiny = !o.zero && o.s < kQuantTiny;
    o.r = 1.0f / o.s;
    o.half = 0.5f * o.s;
    return o;
}

// x / s in binary64 where s is small enough for subnormals (x / s may pass 127 there)
__device__ __forceinline__ int quant_tiny(float x, float s)
{
    double t = rint((double)x / (double)s);
    t = t > 127.0 ? 127.0 : (t < -127.0 ? -127.0 : t);
    return (int)t;
}

constexpr float kQuantMagic = 12582912.0f;                 // 1.5 * 2^23

// the int8 of x in the low byte of the result (a row that is neither tiny nor zero)
__device__ __forceinline__ uint32_t quant_bits(float x, const RowScale& o)
{
    const float u = __builtin_fmaf(x, o.r, kQuantMagic);
    const float q = u - kQuantMagic;
    const float d = __builtin_fmaf(-q, o.s, x);
    uint32_t b = __builtin_bit_cast(uint32_t, u);
    if (__builtin_expect(!(__builtin_fabsf(d) < o.half), 0)) {
        const double e = __builtin_fma(-(double)q, (double)o.s, (double)x), h = 0.5 * (double)o.s;
        const bool odd = (b & 1u) != 0u;
        if (e > h || (e == h && odd)) b += 1u;
        if (e < -h || (e == -h && odd)) b -= 1u;
    }
    return b;
}

// The same of E values at once: one test of the largest residual for all of them.
template <int E>
__device__ __forceinline__ void quant_bits(const float (&x)[E], const RowScale& o, uint32_t (&b)[E])
{
    float worst = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const float u = __builtin_fmaf(x[e], o.r, kQuantMagic);
        const float d = __builtin_fmaf(-(u - kQuantMagic), o.s, x[e]);
        worst = __builtin_fmaxf(worst, __builtin_fabsf(d));
        b[e] = __builtin_bit_cast(uint32_t, u);
    }
    if (__builtin_expect(!(worst < o.half), 0)) {
#pragma unroll
        for (int e = 0; e < E; ++e) b[e] = quant_bits(x[e], o);
    }
}

__device__ __forceinline__ uint32_t quant_any(float x, const RowScale& o)
{
    if (o.zero) return 0u;
    return o.tiny ? (uint32_t)quant_tiny(x, o.s) : quant_bits(x, o);
}

__device__ __forceinline__ uint32_t pack4(uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    const uint32_t lo = __builtin_amdgcn_perm(b, a, 0x0C0C0400u), hi = __builtin_amdgcn_perm(d, c, 0x04000C0Cu);
    return lo | hi;
}

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

struct QuantShape {
    static constexpr int kThreads = 256;
};

// One row per RT threads (64: a wave a row; 256: a workgroup a row).  E elements of T in
// 16 bytes; a thread holds NCH such chunks of its row in registers between the two
// passes, and rows longer than RT * NCH chunks are read a second time.  Rows may start on
// any element (neither loads nor stores need more alignment); a row's last chunk, if it is
// not whole, goes element by element.
//   grid.x = ceil(rows / (256 / RT)), block = 256
template <typename T, int RT, int NCH>
__global__ void __launch_bounds__(QuantShape::kThreads)
quantize_rows(const T* __restrict__ x, int64_t rows, int cols, int64_t ldx, int8_t* __restrict__ q, int64_t ldq,
              float* __restrict__ scale)
{
    constexpr int E = 16 / (int)sizeof(T);
    __shared__ uint32_t red[QuantShape::kThreads / 64];
    const int tid = threadIdx.x, t = tid % RT;
    const int64_t row = (int64_t)blockIdx.x * (QuantShape::kThreads / RT) + tid / RT;
    const bool live = row < rows;
    const T* xr = x + (live ? row : 0) * ldx;
    const int n = live ? cols : 0;
    const int nch = (n + E - 1) / E;

    struct Chunk { T v[E]; };
    auto load = [&](int c) { return __builtin_bit_cast(Chunk, load_chunk<T>(xr, c * E, n)); };
    Chunk held[NCH];
    uint32_t m = 0;
    auto take = [&](const Chunk& o) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t w = __builtin_bit_cast(u32x4, o)[e];
            if constexpr (sizeof(T) == 2) {
                m = pair_max(m, w);
            } else {
                const uint32_t a = w & 0x7FFFFFFFu;
                m = a > m ? a : m;
            }
        }
    };
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
        const int c = t + i * RT;
        if (c < nch) {
            held[i] = load(c);
            take(held[i]);
        }
    }
    for (int c = t + NCH * RT; c < nch; c += RT) take(load(c));
    if constexpr (sizeof(T) == 2) {                    // the larger half, as binary32 bits
        const uint32_t h = (m & 0xFFFFu) > (m >> 16) ? m & 0xFFFFu : m >> 16;
        m = abs_bits(to_f32(__builtin_bit_cast(T, (uint16_t)h)));
    }
    m = wave_max(m);
    if constexpr (RT > 64) {
        if ((tid & 63) == 0) red[tid >> 6] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < RT / 64; ++w) m = red[w] > m ? red[w] : m;
    }
    if (!live) return;
    const RowScale sc = row_scale(m);
    if (t == 0) scale[row] = sc.s;
    int8_t* qr = q + row * ldq;
    auto store = [&](int c, const Chunk& o) {
        uint32_t b[E];
        float v[E];
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = to_f32(o.v[e]);
        if (__builtin_expect(sc.zero || sc.tiny, 0)) {
#pragma unroll
            for (int e = 0; e < E; ++e) b[e] = quant_any(v[e], sc);
        } else {
            quant_bits(v, sc, b);
        }
        int8_t* p = qr + (int64_t)c * E;
        if ((c + 1) * E <= n) {
            struct __attribute__((packed)) Loose { uint32_t w[E / 4]; } l;
#pragma unroll
            for (int g = 0; g < E / 4; ++g) l.w[g] = pack4(b[4 * g], b[4 * g + 1], b[4 * g + 2], b[4 * g + 3]);
            *reinterpret_cast<Loose*>(p) = l;
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (c * E + e < n) p[e] = (int8_t)b[e];
        }
    };
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
        const int c = t + i * RT;
        if (c < nch) store(c, held[i]);
    }
    for (int c = t + NCH * RT; c < nch; c += RT) store(c, load(c));
}

// ---- streams to rows ----------------------------------------------------------------------
// W [M][N] from its tile streams (tile (I, J) is sequence I (N/16) + J, weight 16 r + c of
// a tile is row 16 I + r, column 16 J + c).  One workgroup of 4 waves per quarter of a band
// of 16 rows: wave w decodes the four rows of tiles 64 w + lane, + 256, ...: a lane reads the
// five stream words of its rows and writes whole tile rows, so that a wave's stores of one
// row are contiguous.  Row r of a tile is stream bits [32 r, 32 r + 30 + L), inside words r
// and r + 1 (word 16 of a tail-biting stream is word 0).  The quarters of a band share its
// streams' lines, so they run on one XCD: workgroups go round the 8 XCDs, and workgroup b of
// each 32 takes quarter b / 8 of band b % 8.
//
// int8 first finds the largest magnitude of each row, on the codes before their rescale
// (exact in fp16; code_rescale is odd and monotone).  HOLD tiles a lane keep those codes in
// registers for the second pass; tiles beyond HOLD * 256 are decoded again.
//
// The int8 of a code is that of its rescaled value c: with D the code's divisor, raw / (D s)
// is within 2^-15 of c / s (three roundings of at most 127), so its nearest integer is the
// int8 wherever it lies further than 2^-14 from a half step; the rest goes through c.
//
// At 2 bits in and 8 out the memory moves 235 million weights (28672x8192) in 57 us; the call
// takes 103.  Its VALU work is 11 instructions a weight (6.7 in the first pass, 4.4 in the
// second), 16 as counted with the second looks near half steps: 47 us at the VALU's peak.
// Load, decode and store of a workgroup follow each other, so these times only partly
// overlap.
struct DecodeRowsShape {
    static constexpr int kThreads = 256;
    static constexpr int kTiles = 256;       // tiles of a band in flight
};

template <int CODE>
constexpr float code_divisor()
{
    return CODE == kCode1Mad ? 147.8f : (CODE == kCode3Inst ? 1.244f : 1.0f);
}

// OUT: 0 int8 + scale, 1 bf16, 2 fp16, 3 binary32.  grid.x = 4 bands.
template <int L, int CODE, bool TB, int OUT, int HOLD>
__global__ void __launch_bounds__(DecodeRowsShape::kThreads)
decode_rows(const uint32_t* __restrict__ bits, int bands, int NTJ, void* __restrict__ w, int64_t ldw,
            float* __restrict__ scale, CodeArg ca)
{
    constexpr int Wd = TB ? 16 : (L + 2 * 255 + 31) / 32, NT = DecodeRowsShape::kTiles;
    __shared__ uint32_t red[4][4];
    const int lane = threadIdx.x & 63, j0 = threadIdx.x;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // whole groups of 8 bands by quarters, the bands after them in order
    const int b = blockIdx.x, grouped = bands >> 3 << 3;
    const int I = b < 4 * grouped ? (b >> 5) * 8 + (b & 7) : b >> 2;
    const int r0 = 4 * (b < 4 * grouped ? (b >> 3) & 3 : b & 3);
    const uint32_t* band = bits + (int64_t)I * NTJ * Wd;
    const uint32_t kbias = vgpr_u32(0xE5FEE5FEu);   // fp16 -1534 in both halves

    struct Words { uint32_t w[5]; };
    auto load = [&](int j) {
        Words o;
        const uint32_t* p = band + (int64_t)j * Wd;
#pragma unroll
        for (int i = 0; i < 5; ++i) o.w[i] = p[TB ? ((r0 + i) & 15) : (r0 + i)];
        return o;
    };
    // the 16 codes of row r0 + a before their rescale, as fp16 pairs
    struct Row { uint32_t h[8]; };
    auto raw_row = [&](const Words& o, int a) {
        const uint32_t f0 = o.w[a], f1 = __builtin_amdgcn_alignbit(o.w[a], o.w[a + 1], 16);
        Row v;
#pragma unroll
        for (int g = 0; g < 8; ++g) {
            const uint32_t f = g < 4 ? f0 : f1;
            v.h[g] = code_raw_pair_f16<CODE>((f >> (32 - L - 4 * (g & 3))) & ((1u << L) - 1u),
                                             (f >> (30 - L - 4 * (g & 3))) & ((1u << L) - 1u), kbias, ca);
        }
        return v;
    };
    const int64_t row0 = 16 * (int64_t)I + r0;
    if constexpr (OUT == 0) {
        Row held[HOLD][4];
        uint32_t m[4] = {0u, 0u, 0u, 0u};
        auto take = [&](const Row& v, int a) {
#pragma unroll
            for (int g = 0; g < 8; ++g) m[a] = pair_max(m[a], v.h[g]);
        };
#pragma unroll
        for (int t = 0; t < HOLD; ++t) {
            if (j0 + t * NT < NTJ) {
                const Words o = load(j0 + t * NT);
#pragma unroll
                for (int a = 0; a < 4; ++a) {
                    held[t][a] = raw_row(o, a);
                    take(held[t][a], a);
                }
            }
        }
        for (int j = j0 + HOLD * NT; j < NTJ; j += NT) {
            const Words o = load(j);
#pragma unroll
            for (int a = 0; a < 4; ++a) take(raw_row(o, a), a);
        }
#pragma unroll
        for (int a = 0; a < 4; ++a) {
            const uint32_t h = (m[a] & 0xFFFFu) > (m[a] >> 16) ? m[a] & 0xFFFFu : m[a] >> 16;
            const uint32_t mm = wave_max(h);
            if (lane == 0) red[wave][a] = mm;
        }
        __syncthreads();
        RowScale sc[4];
        float rho[4];
#pragma unroll
        for (int a = 0; a < 4; ++a) {
            uint32_t mm = 0;
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const uint32_t v = red[g][a];
                mm = v > mm ? v : mm;
            }
            // the smallest nonzero code value of any code is far above kQuantTiny
            const float top = (float)__builtin_bit_cast(_Float16, (uint16_t)mm);
            sc[a] = row_scale(__builtin_bit_cast(uint32_t, code_rescale<CODE>(top)));
            rho[a] = sc[a].zero ? 0.0f : sc[a].r / code_divisor<CODE>();
            if (threadIdx.x == 0) scale[row0 + a] = sc[a].s;
        }
        int8_t* out = static_cast<int8_t*>(w) + row0 * ldw;
        auto put = [&](int j, int a, const Row& row) {
            uint32_t b[16];
            float worst = 0.0f;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const float x = (float)__builtin_bit_cast(code_half2, row.h[e >> 1])[e & 1];
                const float u = __builtin_fmaf(x, rho[a], kQuantMagic);
                const float d = __builtin_fmaf(x, rho[a], -(u - kQuantMagic));
                worst = __builtin_fmaxf(worst, __builtin_fabsf(d));
                b[e] = __builtin_bit_cast(uint32_t, u);
            }
            if (__builtin_expect(worst > 0.5f - 0x1p-14f, 0)) {
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    b[e] = quant_bits(code_rescale<CODE>((float)__builtin_bit_cast(code_half2, row.h[e >> 1])[e & 1]), sc[a]);
            }
            const u32x4 p = {pack4(b[0], b[1], b[2], b[3]), pack4(b[4], b[5], b[6], b[7]),
                             pack4(b[8], b[9], b[10], b[11]), pack4(b[12], b[13], b[14], b[15])};
            *reinterpret_cast<u32x4*>(out + a * ldw + 16 * (int64_t)j) = p;
        };
#pragma unroll
        for (int t = 0; t < HOLD; ++t) {
            if (j0 + t * NT < NTJ) {
#pragma unroll
                for (int a = 0; a < 4; ++a) put(j0 + t * NT, a, held[t][a]);
            }
        }
        for (int j = j0 + HOLD * NT; j < NTJ; j += NT) {
            const Words o = load(j);
#pragma unroll
            for (int a = 0; a < 4; ++a) put(j, a, raw_row(o, a));
        }
    } else {
        for (int j = j0; j < NTJ; j += NT) {
            const Words o = load(j);
#pragma unroll
            for (int a = 0; a < 4; ++a) {
                const Row row = raw_row(o, a);
                float v[16];
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    v[e] = code_rescale<CODE>((float)__builtin_bit_cast(code_half2, row.h[e >> 1])[e & 1]);
                const int64_t at = (row0 + a) * ldw + 16 * (int64_t)j;
                if constexpr (OUT == 3) {
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        const f32x4 p = {v[4 * g], v[4 * g + 1], v[4 * g + 2], v[4 * g + 3]};
                        reinterpret_cast<f32x4*>(static_cast<float*>(w) + at)[g] = p;
                    }
                } else {
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        if constexpr (OUT == 1) {
                            bf16x8 p;
#pragma unroll
                            for (int e = 0; e < 8; ++e) p[e] = from_f32<__bf16>(v[8 * g + e]);
                            reinterpret_cast<bf16x8*>(static_cast<__bf16*>(w) + at)[g] = p;
                        } else {
                            f16x8 p;
#pragma unroll
                            for (int e = 0; e < 8; ++e) p[e] = from_f32<_Float16>(v[8 * g + e]);
                            reinterpret_cast<f16x8*>(static_cast<_Float16*>(w) + at)[g] = p;
                        }
                    }
                }
            }
        }
    }
}

}  // namespace qtcq
