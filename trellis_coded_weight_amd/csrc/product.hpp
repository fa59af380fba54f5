// product.hpp -- what the matrix products share, gfx950: the 8-bit product with token and
// channel scales, the gated projections and the two products of their gradient.
//
// Every one of them is out[i][j] = sum_k P(i, k) Q(j, k) over one or two pairs of operands,
// with an epilogue of its own:
//   kInt8    P = a [M][K], Q = w [N][K]; out = acc * a_scale[i] * w_scale[j]
//   kGated   P = x [M][K], Q = Wg and Wu [F][K], both in one workgroup; out = act(gate) * up
//   kGradX   P = dg then du [M][F], Q(j, k) = Wg[k][j] then Wu[k][j]; one sum over both
//   kGradW   P(i, k) = dg[k][i] (z = 0) or du[k][i] (z = 1), Q(j, k) = x[k][j]
// dg and du are the sums of two parts each (gated_slopes), whose products with Q are added
// one after the other, or one part, where the caller has them rounded.
//
// v_mfma_*_16x16x(64 bytes) on Q rows times P rows: lane l holds 16 bytes of Q row l % 16
// and of P row l % 16 from byte 16 (l / 16) of a 64-byte step, and the result
// D[4 (l / 16) + v][l % 16], v = 0..3: four consecutive columns j of the row i = l % 16,
// stored together.  Sums are held in binary32 (int32 for kInt8, where they are exact:
// K <= 131071).
//
// Two kernels share the work: few rows of P, rows on any element (skinny_product.hpp), and
// any number of rows on whole 16-byte chunks (block_product.hpp).  Operands that are not
// whole chunks go to the second through a copy with a padded pitch (pad_rows).
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
    int pk, qk;              // k of operands stored [row][k], with their zero padding
    int pm, qn;              // rows of operands stored [k][row], with their padding
    const float* p_scale;    // kInt8
    const float* q_scale;
    void* save[2];           // kGated: the projections, or NULL
    int64_t lds;
    void* part;              // the shares' sums [shares][m][part_pitch], or NULL
    int part_pitch;
    int shares, share_steps; // shares of k, and the steps of each
    int pieces;              // kGradX, kGradW: parts that P is the sum of, 1 or 2,
    int64_t piece_step;      // and the elements from one to the next
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

// Four consecutive results of row `row` from column `col` (those inside the matrix), from
// their sums s (kGated: the gate's, and u the up's).
template <typename O, int MODE, int ACT, typename Acc>
__device__ __forceinline__ void finish_at(const ProductArgs& a, int z, int row, int col, const Acc& s, const Acc& u)
{
    const int left = a.n - col;
    float v[4];
    if constexpr (MODE == kGated) {
        const float gv[4] = {s[0], s[1], s[2], s[3]}, uv[4] = {u[0], u[1], u[2], u[3]};
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = activate<ACT>(gv[e]) * uv[e];
        if (a.save[0]) {
            store4(static_cast<O*>(a.save[0]) + (int64_t)row * a.lds + col, gv, left);
            store4(static_cast<O*>(a.save[1]) + (int64_t)row * a.lds + col, uv, left);
        }
    } else if constexpr (MODE == kInt8) {
        const float ps = a.p_scale[row];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = (float)s[e] * ps * (e < left ? a.q_scale[col + e] : 0.0f);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = s[e];
    }
    store4(static_cast<O*>(a.out[z]) + (int64_t)row * a.ldo + col, v, left);
}

// Threads over the rows of a matrix, `per` pieces a row, in blocks of 256: whole rows in a
// block, or a row over several blocks (an index division a block, not a 64-bit one a
// thread).
struct RowGrid {
    int per;
    __host__ __device__ int wide() const { return (per + 255) / 256; }        // blocks a row
    __host__ __device__ int rows() const { return per < 256 ? 256 / per : 1; }  // rows a block
    int64_t blocks(int64_t n) const { return per > 0 ? (n + rows() - 1) / rows() * wide() : 0; }
    // this thread's row and piece in block b; false for a thread without one
    __device__ __forceinline__ bool at(unsigned b, int64_t& row, int& piece) const
    {
        if (per < 256) {
            const int r = threadIdx.x / per;
            row = (int64_t)b * rows() + r;
            piece = threadIdx.x - r * per;
            return r < rows();
        }
        const unsigned w = wide(), r = b / w;
        row = r;
        piece = (int)(b - r * w) * 256 + threadIdx.x;
        return piece < per;
    }
};

// The shares of k added in order, then the epilogue.  part [shares][m][part_pitch], four
// columns a thread (kGated: the gate's sums, then the up's, part_pitch / 2 apart).
//   grid.x = RowGrid{columns / 4}.blocks(m), block = 256.
template <typename T, typename O, int MODE, int ACT>
__global__ void __launch_bounds__(256)
join_shares(ProductArgs a)
{
    typedef typename Mfma<T>::Acc Acc;
    const int width = MODE == kGated ? a.part_pitch / 2 : a.part_pitch;
    int64_t row;
    int col;
    if (!RowGrid{width >> 2}.at(blockIdx.x, row, col) || row >= a.m) return;
    col *= 4;
    const int64_t next = (int64_t)a.m * a.part_pitch >> 2, at = (row * a.part_pitch + col) >> 2;
    const Acc* p = static_cast<const Acc*>(a.part) + at;
    Acc s = {}, u = {};
    for (int i = 0; i < a.shares; ++i) {
        s += p[i * next];
        if constexpr (MODE == kGated) u += p[i * next + (width >> 2)];
    }
    finish_at<O, MODE, ACT>(a, 0, (int)row, col, s, u);
}

// Up to three matrices of rows of `cols` elements, on any element, to rows of whole 16-byte
// chunks, zero past cols, in one launch.
//   matrix i: blocks first[i] .. first[i + 1] - 1 (RowGrid over its chunks), which any
//   grid.x takes in turn; block = 256; pitch a multiple of E.
struct PadArgs {
    const void* src[3];
    void* dst[3];
    int64_t ld[3], rows[3], first[4];
    int cols, pitch;
};

template <typename T>
__global__ void __launch_bounds__(256)
pad_rows(PadArgs a)
{
    constexpr int E = 16 / (int)sizeof(T);
    const RowGrid g{a.pitch / E};
    for (int64_t b = blockIdx.x; b < a.first[3]; b += gridDim.x) {
        const int i = b >= a.first[2] ? 2 : (b >= a.first[1] ? 1 : 0);
        int64_t row;
        int at;
        if (!g.at((unsigned)(b - a.first[i]), row, at) || row >= a.rows[i]) continue;
        *reinterpret_cast<u32x4*>(static_cast<T*>(a.dst[i]) + row * a.pitch + at * E) =
            load_chunk<T>(static_cast<const T*>(a.src[i]) + row * a.ld[i], at * E, a.cols);
    }
}

// dg = dh u act'(g) and du = dh act(g), each formed in binary32.  The matrix instructions
// that take them next have 16-bit operands, so each is written as two parts (two_parts), or,
// with one piece, rounded once to the operands' type: its relative 2^-8 (bf16) or 2^-11 (fp16)
// at most a term adds in squares over a sum, about what the rounding of the gradient itself
// costs.  An infinite gate or up may be a finite one that T does not hold, saved as such, so
// an upstream gradient or slope of 0 makes 0 of it and not NaN: a masked token's projections do
// not reach the gradients of the weights.  d [pieces][2][M][ldd], dgate and dup in the first piece; columns from F to ldd are
// written as zero.
//   grid.x = RowGrid{ldd / 8}.blocks(M), block = 256; ldd a multiple of 8.
template <typename T, int ACT>
__global__ void __launch_bounds__(256)
gated_slopes(const T* __restrict__ gate, const T* __restrict__ up, int64_t ldg, const T* __restrict__ gh, int64_t ldh,
             int64_t M, int F, int ldd, T* __restrict__ dgate, T* __restrict__ dup, int pieces, int64_t piece_step)
{
    typedef T T8 __attribute__((ext_vector_type(8)));
    int64_t row;
    int col;
    if (!RowGrid{ldd >> 3}.at(blockIdx.x, row, col) || row >= M) return;
    col *= 8;
    const T8 g = __builtin_bit_cast(T8, load_chunk<T>(gate + row * ldg, col, F));
    const T8 u = __builtin_bit_cast(T8, load_chunk<T>(up + row * ldg, col, F));
    const T8 h = __builtin_bit_cast(T8, load_chunk<T>(gh + row * ldh, col, F));
    T8 dg, du, dg2, du2;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        float av, dv;
        activate_grad<ACT>((float)g[e], av, dv);
        const float hv = (float)h[e];
        const float up_v = (float)u[e];
        // beside an infinite projection, which stands for a large finite one, a 0 stays 0
        const bool gz = col + e >= F || (__builtin_fabsf(up_v) == __builtin_inff() && hv * dv == 0.0f);
        const bool uz = col + e >= F || (__builtin_fabsf(av) == __builtin_inff() && hv == 0.0f);
        const float gv = gz ? 0.0f : hv * up_v * dv, uv = uz ? 0.0f : hv * av;
        T hi, lo;
        two_parts(gv, hi, lo);
        dg[e] = pieces == 2 ? hi : from_f32<T>(gv);
        dg2[e] = lo;
        two_parts(uv, hi, lo);
        du[e] = pieces == 2 ? hi : from_f32<T>(uv);
        du2[e] = lo;
    }
    const int64_t at = row * ldd + col;
    *reinterpret_cast<T8*>(dgate + at) = dg;
    *reinterpret_cast<T8*>(dup + at) = du;
    if (pieces == 2) {
        *reinterpret_cast<T8*>(dgate + piece_step + at) = dg2;
        *reinterpret_cast<T8*>(dup + piece_step + at) = du2;
    }
}

}  // namespace qtcq
