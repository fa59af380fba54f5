// tile_product.hpp -- matrix products on the matrix cores for operands of any alignment,
// gfx950: the 8-bit product with token and channel scales, the gated projections and the
// two products of their gradient.
//
// Every one of them is out[i][j] = sum_k P(i, k) Q(j, k) over one or two pairs of operands,
// with an epilogue of its own:
//   kInt8    P = a [M][K], Q = w [N][K]; out = acc * a_scale[i] * w_scale[j]
//   kGated   P = x [M][K], Q = Wg and Wu [F][K], both in one workgroup (the tile's columns
//            are half gate, half up); out = act(gate) * up
//   kGradX   P = dg then du [M][F], Q(j, k) = Wg[k][j] then Wu[k][j]; one sum over both
//   kGradW   P(i, k) = dg[k][i] (z = 0) or du[k][i] (z = 1), Q(j, k) = x[k][j]
//
// v_mfma_*_16x16x(64 bytes) on Q rows times P rows: lane l holds 16 bytes of Q row l % 16
// and of P row l % 16 from byte 16 (l / 16) of a 64-byte step, and the result
// D[4 (l / 16) + v][l % 16], v = 0..3: four consecutive columns j of the row i = l % 16,
// stored together.  Sums are held in binary32 (int32 for kInt8, where they are exact:
// K <= 131071).
//
// Rows of either operand may start on any element.  A tile is loaded by threads in chunks
// of 16 bytes, whole where they lie inside the matrix (global loads need no alignment
// here) and element by element at its edges; what lies outside is zero.
#pragma once

#include "dense.hpp"

namespace qtcq {

enum : int { kInt8 = 0, kGated = 1, kGradX = 2, kGradW = 3 };

struct ProductArgs {
    const void* p[2];        // operand P (kGradX, kGradW: dg and du)
    const void* q[2];        // operand Q (kGated, kGradX: Wg and Wu)
    int64_t ldp, ldq;        // their row strides, in elements
    void* out[2];            // out (kGradW: both weight gradients)
    int64_t ldo;
    int m, n, k;             // rows and columns of out, length of one sum
    int kp;                  // kGradX: k of P with its zero-filled columns
    const float* p_scale;    // kInt8
    const float* q_scale;
    void* save[2];           // kGated: the projections, or NULL
    int64_t lds;
};

struct TileShape {
    static constexpr int kThreads = 256;
    static constexpr int kRows = 128;         // rows of P and of Q in a tile
    static constexpr int kStep = 64;          // bytes of k in a step
    static constexpr int kPitch = 80;         // bytes between rows in LDS (16 apart in banks)
    // columns of out covered by a tile of Q
    static constexpr int cols(int mode) { return mode == kGated ? kRows / 2 : kRows; }
};

template <typename T> struct Mfma;
template <> struct Mfma<__bf16> {
    typedef f32x4 Acc;
    static __device__ __forceinline__ Acc mul(u32x4 a, u32x4 b, Acc c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b),
                                                       c, 0, 0, 0);
    }
};
template <> struct Mfma<_Float16> {
    typedef f32x4 Acc;
    static __device__ __forceinline__ Acc mul(u32x4 a, u32x4 b, Acc c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b),
                                                      c, 0, 0, 0);
    }
};
template <> struct Mfma<int8_t> {
    typedef i32x4 Acc;
    static __device__ __forceinline__ Acc mul(u32x4 a, u32x4 b, Acc c)
    {
        return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a), __builtin_bit_cast(i32x4, b),
                                                     c, 0, 0, 0);
    }
};

// 16 bytes at p + at of a row with n elements, zero past its end
template <typename T>
__device__ __forceinline__ u32x4 load_chunk(const T* p, int at, int n)
{
    constexpr int E = 16 / (int)sizeof(T);
    struct __attribute__((packed, aligned(sizeof(T)))) Loose { u32x4 v; };
    if (at + E <= n) return reinterpret_cast<const Loose*>(p + at)->v;
    struct Parts { T e[E]; } o;
#pragma unroll
    for (int e = 0; e < E; ++e) o.e[e] = at + e < n ? p[at + e] : (T)0;
    return __builtin_bit_cast(u32x4, o);
}

// four consecutive outputs of a row, of which n are inside the matrix (stores need no
// alignment beyond the element's here)
template <typename O>
__device__ __forceinline__ void store4(O* p, const float (&v)[4], int n)
{
    struct __attribute__((packed, aligned(sizeof(O)))) Four { O e[4]; };
    if (n >= 4) {
        *reinterpret_cast<Four*>(p) = Four{{from_f32<O>(v[0]), from_f32<O>(v[1]), from_f32<O>(v[2]), from_f32<O>(v[3])}};
        return;
    }
#pragma unroll
    for (int e = 0; e < 3; ++e)
        if (e < n) p[e] = from_f32<O>(v[e]);
}

// grid.x = tiles of out (columns fastest), grid.z = 2 for kGradW; block = 256.
template <typename T, typename O, int MODE, int ACT = 0>
__global__ void __launch_bounds__(TileShape::kThreads)
tile_product(ProductArgs a)
{
    typedef Mfma<T> MM;
    constexpr int E = 16 / (int)sizeof(T);           // elements of a 16-byte chunk
    constexpr int KS = TileShape::kStep / (int)sizeof(T);
    constexpr int R = TileShape::kRows, PITCH = TileShape::kPitch;
    constexpr bool PT = MODE == kGradW;              // P is stored with k as its row index
    constexpr bool QT = MODE == kGradX || MODE == kGradW;
    constexpr int COLS = TileShape::cols(MODE);
    __shared__ __align__(16) char ldsp[R * PITCH];
    __shared__ __align__(16) char ldsq[R * PITCH];

    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int wm = wave >> 1, wn = wave & 1;
    const int tiles_n = (a.n + COLS - 1) / COLS;
    const int i0 = (int)(blockIdx.x / tiles_n) * R, j0 = (int)(blockIdx.x % tiles_n) * COLS;
    const int z = MODE == kGradW ? blockIdx.z : 0;
    const int steps1 = (a.k + KS - 1) / KS;
    const int steps = MODE == kGradX ? 2 * steps1 : steps1;

    // a tile of 128 rows x KS from a row-major [rows][k] matrix: two chunks a thread
    auto load_rows = [&](const T* base, int64_t ld, int row, int nrows, int k0, u32x4* v) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = row + h * 64;
            v[h] = u32x4{0u, 0u, 0u, 0u};
            if (r < nrows) v[h] = load_chunk<T>(base + (int64_t)r * ld, k0 + (tid & 3) * E, a.k);
        }
    };
    // the same tile from a [k][rows] matrix: chunks of E rows of one k
    auto load_cols = [&](const T* base, int64_t ld, int row0, int nrows, int k0, u32x4* v) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int kk = k0 + (tid >> 4) + 16 * h;
            v[h] = u32x4{0u, 0u, 0u, 0u};
            if (kk < a.k) v[h] = load_chunk<T>(base + (int64_t)kk * ld, row0 + (tid & 15) * E, nrows);
        }
    };
    u32x4 pv[2], qv[2];
    auto load = [&](int s) {
        const int seg = MODE == kGradX && s >= steps1 ? 1 : 0;
        const int k0 = (s - seg * steps1) * KS;
        const T* p = static_cast<const T*>(a.p[MODE == kGradW ? z : seg]);
        if constexpr (PT)
            load_cols(p, a.ldp, i0, a.m, k0, pv);
        else
            load_rows(p, a.ldp, i0 + (tid >> 2), a.m, k0, pv);
        if constexpr (MODE == kGated) {
            // rows 0..63 of the Q tile are gate columns, 64..127 up columns
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int j = j0 + (tid >> 2);
                qv[h] = u32x4{0u, 0u, 0u, 0u};
                if (j < a.n)
                    qv[h] = load_chunk<T>(static_cast<const T*>(a.q[h]) + (int64_t)j * a.ldq, k0 + (tid & 3) * E, a.k);
            }
        } else if constexpr (QT) {
            load_cols(static_cast<const T*>(a.q[seg]), a.ldq, j0, a.n, k0, qv);
        } else {
            load_rows(static_cast<const T*>(a.q[0]), a.ldq, j0 + (tid >> 2), a.n, k0, qv);
        }
    };
    auto put = [&](char* lds, const u32x4* v, bool transposed) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (!transposed) {
                *reinterpret_cast<u32x4*>(lds + ((tid >> 2) + 64 * h) * PITCH + (tid & 3) * 16) = v[h];
            } else {
                struct Parts { T e[E]; } o = __builtin_bit_cast(Parts, v[h]);
#pragma unroll
                for (int e = 0; e < E; ++e)
                    *reinterpret_cast<T*>(lds + ((tid & 15) * E + e) * PITCH + ((tid >> 4) + 16 * h) * sizeof(T)) = o.e[e];
            }
        }
    };

    // wave (wm, wn): rows 64 wm .. + 63 of P; four groups of 16 rows of Q (kGated: two of
    // gate columns, the two of up columns beside them)
    auto qrow = [&](int j) {
        return MODE == kGated ? (j >> 1) * 64 + wn * 32 + (j & 1) * 16 : wn * 64 + j * 16;
    };
    typename MM::Acc acc[4][4] = {};
    if (steps > 0) load(0);
    for (int s = 0; s < steps; ++s) {
        __syncthreads();
        put(ldsp, pv, PT);
        put(ldsq, qv, QT);
        __syncthreads();
        if (s + 1 < steps) load(s + 1);
        u32x4 pf[4], qf[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            pf[i] = *reinterpret_cast<const u32x4*>(ldsp + (wm * 64 + i * 16 + (lane & 15)) * PITCH + (lane >> 4) * 16);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            qf[j] = *reinterpret_cast<const u32x4*>(ldsq + (qrow(j) + (lane & 15)) * PITCH + (lane >> 4) * 16);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = MM::mul(qf[j], pf[i], acc[i][j]);
    }

    constexpr int NJ = MODE == kGated ? 2 : 4;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = i0 + wm * 64 + i * 16 + (lane & 15);
        if (row >= a.m) continue;
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const int col = j0 + (MODE == kGated ? wn * 32 : wn * 64) + j * 16 + 4 * (lane >> 4);
            const int left = a.n - col;
            if (left <= 0) continue;
            float v[4];
            if constexpr (MODE == kGated) {
                float g[4], u[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    g[e] = acc[i][j][e];
                    u[e] = acc[i][j + 2][e];
                    v[e] = activate<ACT>(g[e]) * u[e];
                }
                if (a.save[0]) {
                    store4(static_cast<O*>(a.save[0]) + (int64_t)row * a.lds + col, g, left);
                    store4(static_cast<O*>(a.save[1]) + (int64_t)row * a.lds + col, u, left);
                }
            } else if constexpr (MODE == kInt8) {
                const float ps = a.p_scale[row];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    v[e] = (float)acc[i][j][e] * ps * (e < left ? a.q_scale[col + e] : 0.0f);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = acc[i][j][e];
            }
            store4(static_cast<O*>(a.out[z]) + (int64_t)row * a.ldo + col, v, left);
        }
    }
}

// dg = dh u act'(g) and du = dh act(g), each formed in binary32 and rounded once to the
// operands' type, the operand type of the matrix instructions that take them next.  The
// rounding's relative 2^-9 (bf16) or 2^-12 (fp16) a term adds in squares over a sum, about
// what the rounding of the gradient itself costs.  d [2][M][ldd]: columns from F to ldd
// are written as zero.
//   grid.x covers M * ldd / 8 chunks of 8 columns, block = 256; ldd a multiple of 8.
template <typename T, int ACT>
__global__ void __launch_bounds__(256)
gated_slopes(const T* __restrict__ gate, const T* __restrict__ up, int64_t ldg, const T* __restrict__ gh, int64_t ldh,
             int64_t M, int F, int ldd, T* __restrict__ dgate, T* __restrict__ dup)
{
    typedef T T8 __attribute__((ext_vector_type(8)));
    const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int per = ldd >> 3;
    const int64_t row = c / per;
    if (row >= M) return;
    const int col = (int)(c - row * per) * 8;
    const T8 g = __builtin_bit_cast(T8, load_chunk<T>(gate + row * ldg, col, F));
    const T8 u = __builtin_bit_cast(T8, load_chunk<T>(up + row * ldg, col, F));
    const T8 h = __builtin_bit_cast(T8, load_chunk<T>(gh + row * ldh, col, F));
    T8 dg, du;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        float av, dv;
        activate_grad<ACT>((float)g[e], av, dv);
        const float hv = (float)h[e];
        dg[e] = col + e < F ? from_f32<T>(hv * (float)u[e] * dv) : (T)0.0f;
        du[e] = col + e < F ? from_f32<T>(hv * av) : (T)0.0f;
    }
    *reinterpret_cast<T8*>(dgate + row * ldd + col) = dg;
    *reinterpret_cast<T8*>(dup + row * ldd + col) = du;
}

}  // namespace qtcq
