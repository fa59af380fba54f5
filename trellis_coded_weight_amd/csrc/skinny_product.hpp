// skinny_product.hpp -- the 8-bit product and the gated projections for few rows of P
// (tokens), where reading Q (the weights) once is the work, gfx950.
//
// A workgroup of 8 waves takes all rows of P, MI groups of 16, and NJ groups of 16 rows of Q
// (kGated: NJ of Wg and NJ of Wu); its waves share k: wave w takes the 128-byte blocks w,
// w + 8, ... of every row, so that a workgroup reads each row in kilobytes.  Operands go from
// memory to registers in the matrix instructions' layout -- lane l holds 16 bytes of row
// l % 16 -- with no LDS and no barrier on the way; DEPTH blocks are in flight a wave.  The
// waves' sums are then added in wave order through LDS and finished by the epilogue.
// (v_mfma_*_16x16x(64 bytes), Q rows times P rows, as in product.hpp.)
//
// ALIGNED: rows start on 16 bytes and are whole chunks; buffer loads whose range check
// returns zeros past the matrices.  Otherwise rows past the last are read as the last one
// (their results are not stored), and the last block of k is loaded with its end guarded.
#pragma once

#include "codes.hpp"
#include "product.hpp"

namespace qtcq {

struct SkinnyShape {
    static constexpr int kThreads = 512;
    static constexpr int kWaves = kThreads / 64;
    static constexpr int kBlock = 128;        // bytes of k a wave takes at a time
    static constexpr int kMaxFrags = 8;       // fragments of sums a wave (64 KB of LDS)
};

// a.m <= 16 MI.  grid.x = ceil(a.n / (16 NJ)), block = 512.
template <typename T, typename O, int MODE, int ACT, int MI, int NJ, int DEPTH, bool ALIGNED>
__global__ void __launch_bounds__(SkinnyShape::kThreads)
skinny_product(ProductArgs a)
{
    typedef Mfma<T> MM;
    typedef typename MM::Acc Acc;
    constexpr int NW = SkinnyShape::kWaves, SZ = (int)sizeof(T), E = 16 / SZ;
    constexpr int NQ = MODE == kGated ? 2 * NJ : NJ;      // groups of Q: gate first, then up
    constexpr int KB = SkinnyShape::kBlock / SZ;          // k of a block
    constexpr int F = MI * NQ;                            // fragments of sums
    static_assert(F <= SkinnyShape::kMaxFrags, "a wave finishes one fragment");
    __shared__ Acc red[NW][F][64];

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int j0 = blockIdx.x * 16 * NJ;
    const int64_t ldp = a.ldp * SZ, ldq = a.ldq * SZ;
    const int kb = a.k * SZ;                              // bytes of a row
    const int r = lane & 15, c = lane >> 4;

    // all rows of P and rows j0.. of Q through descriptors that end with the matrix
    auto rsrc = [&](const void* p, int64_t ld, int row0, int nrows, int rows) {
        const int n = nrows - row0 < rows ? nrows - row0 : rows;
        return __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(static_cast<const char*>(p) + row0 * ld), (short)0,
                                                 n > 0 ? (n - 1) * (int)ld + kb : 0, kRawBufferWord3);
    };
    __amdgpu_buffer_rsrc_t rp, rq[2];
    if constexpr (ALIGNED) {
        rp = rsrc(a.p[0], ldp, 0, a.m, 16 * MI);
        rq[0] = rsrc(a.q[0], ldq, j0, a.n, 16 * NJ);
        rq[1] = rsrc(a.q[MODE == kGated], ldq, j0, a.n, 16 * NJ);
    }
    struct Set { u32x4 p[2][MI], q[2][NQ]; };
    auto load = [&](int blk, Set& o) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int at = blk * SkinnyShape::kBlock + 64 * h + 16 * c;    // byte in the row
            if constexpr (ALIGNED) {
                // a chunk past the row's end goes out of range
                const int ap = at < kb ? r * (int)ldp + at : 0x7FFFFFFF, aq = at < kb ? r * (int)ldq + at : 0x7FFFFFFF;
#pragma unroll
                for (int j = 0; j < NQ; ++j)
                    o.q[h][j] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                        rq[j >= NJ], at < kb ? aq + (j % NJ) * 16 * (int)ldq : aq, 0, 0));
#pragma unroll
                for (int i = 0; i < MI; ++i)
                    o.p[h][i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                        rp, at < kb ? ap + i * 16 * (int)ldp : ap, 0, 0));
            } else {
                auto chunk = [&](const void* base, int64_t ld, int row, int nrows) {
                    const T* p = static_cast<const T*>(base) + (int64_t)(row < nrows ? row : nrows - 1) * ld;
                    return (blk + 1) * KB <= a.k ? load_loose(p + at / SZ)
                           : blk * KB < a.k      ? load_chunk<T>(p, at / SZ, a.k)
                                                 : u32x4{0u, 0u, 0u, 0u};
                };
#pragma unroll
                for (int j = 0; j < NQ; ++j) o.q[h][j] = chunk(a.q[j >= NJ], a.ldq, j0 + (j % NJ) * 16 + r, a.n);
#pragma unroll
                for (int i = 0; i < MI; ++i) o.p[h][i] = chunk(a.p[0], a.ldp, i * 16 + r, a.m);
            }
        }
    };
    Acc acc[MI][NQ] = {};
    auto multiply = [&](const Set& o) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < MI; ++i)
#pragma unroll
                for (int j = 0; j < NQ; ++j) acc[i][j] = MM::mul(o.q[h][j], o.p[h][i], acc[i][j]);
    };
    // DEPTH register sets in turn; blocks past the last are zeros
    const int nblk = (a.k + KB - 1) / KB;
    if (wave < nblk) {
        Set set[DEPTH];
#pragma unroll
        for (int d = 0; d < DEPTH - 1; ++d) load(wave + d * NW, set[d]);
        for (int b = wave; b < nblk; b += DEPTH * NW) {
#pragma unroll
            for (int d = 0; d < DEPTH; ++d) {
                load(b + (d + DEPTH - 1) * NW, set[(d + DEPTH - 1) % DEPTH]);
                multiply(set[d]);
            }
        }
    }

    // sums of the waves in order: wave w finishes fragment w (kGated: gate fragment w and the
    // up fragment beside it; fragments are numbered gate groups, then up groups, of each
    // row group)
#pragma unroll
    for (int f = 0; f < F; ++f) red[wave][f][lane] = acc[f / NQ][f % NQ];
    __syncthreads();
    constexpr int DONE = MODE == kGated ? F / 2 : F;
    if (wave < DONE) {
        const int f = MODE == kGated ? wave / NJ * NQ + wave % NJ : wave;
        const int i = f / NQ, j = f % NQ;
        Acc s = red[0][f][lane], u = {};
        if constexpr (MODE == kGated) u = red[0][f + NJ][lane];
#pragma unroll
        for (int w = 1; w < NW; ++w) {
            s += red[w][f][lane];
            if constexpr (MODE == kGated) u += red[w][f + NJ][lane];
        }
        const int row = i * 16 + r, col = j0 + j * 16 + 4 * c;
        if (row < a.m && col < a.n) finish_at<O, MODE, ACT>(a, 0, row, col, s, u);
    }
}

}  // namespace qtcq
