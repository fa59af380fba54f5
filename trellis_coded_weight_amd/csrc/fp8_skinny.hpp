// fp8_skinny.hpp -- the product of e4m3 matrices for few rows of activations, where reading
// the weights once is the work, gfx950.
//
// A workgroup of 8 waves takes all rows of a, MI groups of 16, and 16 rows of w; its waves share
// k: wave v takes the blocks v, v + 8, ... of 128 bytes of every row.  Operands go from memory
// to registers in the matrix instruction's layout with no LDS and no barrier on the way, DEPTH
// blocks in flight a wave, a block's scales with it; blocks past the last are neither loaded
// nor multiplied (1x26392x1024 10 us, 16 with zeros in their place).  The waves' sums are added
// in wave order through LDS.
//
// Bound by memory with one row (28672x8192 41 us, 5.7 TB/s), by the groups of 16 rows and their
// conversions to fp16 with more (8 rows 48.5 us); small ones by the launch (1x4096x4096 6.4 us
// in the kernel).
//
// ALIGNED: rows start on 16 bytes and are whole chunks; buffer loads whose range check returns
// zeros past the matrices.  Otherwise rows past the last are read as the last one (their
// results are not stored), and what is behind the last whole block of k is loaded apart.
#pragma once

#include "fp8_product.hpp"
#include "rows.hpp"

namespace qtcq {

struct Fp8SkinnyShape {
    static constexpr int kThreads = 512;
    static constexpr int kWaves = kThreads / 64;
};

// a.m <= 16 MI.  grid.x = ceil(n / 16), block = 512
template <typename O, int MI, int DEPTH, bool ALIGNED>
__global__ void __launch_bounds__(Fp8SkinnyShape::kThreads)
fp8_skinny_product(Fp8Args a)
{
    constexpr int NW = Fp8SkinnyShape::kWaves;
    static_assert(MI <= NW, "a wave finishes one fragment");
    __shared__ f32x4 red[NW][MI][64];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int j0 = blockIdx.x * 16;
    const int r = lane & 15, c = lane >> 4;
    // whole blocks, and where rows need not be whole chunks, what is left behind them
    const int nblk = ALIGNED ? (a.k + 127) / 128 : a.k / 128, left = ALIGNED ? 0 : a.k % 128;

    __amdgpu_buffer_rsrc_t ra, rw;
    if constexpr (ALIGNED) {
        // both end with their matrix
        auto rsrc = [&](const uint8_t* p, int64_t ld, int row0, int nrows, int rows) {
            const int n = nrows - row0 < rows ? nrows - row0 : rows;
            return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(p + row0 * ld), (short)0,
                                                     n > 0 ? (n - 1) * (int)ld + a.k : 0, kRawBufferWord3);
        };
        ra = rsrc(a.a, a.lda, 0, a.m, 16 * MI);
        rw = rsrc(a.w, a.ldw, j0, a.n, 16);
    }
    struct Set { u32x4 p[2][MI], q[2]; float s[MI]; float t; };
    auto a_row = [&](int i) { return a.a + (int64_t)(16 * i + r < a.m ? 16 * i + r : a.m - 1) * a.lda; };
    const uint8_t* w_row = a.w + (int64_t)(j0 + r < a.n ? j0 + r : a.n - 1) * a.ldw;
    auto load_scales = [&](int blk, Set& o) {
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            const int row = 16 * i + r < a.m ? 16 * i + r : a.m - 1;
            o.s[i] = a.a_scale[row * a.as_row + blk * a.as_col];
        }
        o.t = a.w_scale[(j0 >> 7) * a.ws_row + blk * a.ws_col];
    };
    auto load = [&](int blk, Set& o) {
        if (blk >= nblk) return;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int at = blk * 128 + 64 * h + 16 * c;
            if constexpr (ALIGNED) {
                o.q[h] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                    rw, at < a.k ? r * (int)a.ldw + at : 0x7FFFFFFF, 0, 0));
#pragma unroll
                for (int i = 0; i < MI; ++i)
                    o.p[h][i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                        ra, at < a.k ? (r + 16 * i) * (int)a.lda + at : 0x7FFFFFFF, 0, 0));
            } else {
                o.q[h] = load_loose(w_row + at);
#pragma unroll
                for (int i = 0; i < MI; ++i) o.p[h][i] = load_loose(a_row(i) + at);
            }
        }
        load_scales(blk, o);
    };
    f32x4 acc[MI] = {};
    auto multiply = [&](const Set& o) {
        typedef BlockOperand<false> Op;
        const Op q(o.q[0], o.q[1]);
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            const float f = o.s[i] * o.t;
            const f32x4 t = Op::mul(q, Op(o.p[0][i], o.p[1][i]));
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i][e] = __builtin_fmaf(t[e], f, acc[i][e]);
        }
    };
    // What is left: chunks past a row's last byte are read as its last 16 bytes and moved into
    // place when they are multiplied, by the wave whose turn it is.
    Set rest;
    const bool mine = left > 0 && wave == nblk % NW;
    if (mine) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int n = nblk * 8 + 4 * h + c;
            auto chunk = [&](const uint8_t* p) {
                if (a.k < 16) return n == 0 ? load_chunk<uint8_t>(p, 0, a.k) : u32x4{0u, 0u, 0u, 0u};
                return load_loose(p + place_of<uint8_t>(n, a.k).at);
            };
            rest.q[h] = chunk(w_row);
#pragma unroll
            for (int i = 0; i < MI; ++i) rest.p[h][i] = chunk(a_row(i));
        }
        load_scales(nblk, rest);
    }
    if (wave < nblk) {
        Set set[DEPTH];
#pragma unroll
        for (int d = 0; d < DEPTH - 1; ++d) load(wave + d * NW, set[d]);
        for (int b = wave; b < nblk; b += DEPTH * NW) {
#pragma unroll
            for (int d = 0; d < DEPTH; ++d) {
                load(b + (d + DEPTH - 1) * NW, set[(d + DEPTH - 1) % DEPTH]);
                if (b + d * NW < nblk) multiply(set[d]);
            }
        }
    }
    if (mine) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int bits = a.k < 16 ? 0 : place_of<uint8_t>(nblk * 8 + 4 * h + c, a.k).bits;
            rest.q[h] = behind(rest.q[h], bits);
#pragma unroll
            for (int i = 0; i < MI; ++i) rest.p[h][i] = behind(rest.p[h][i], bits);
        }
        multiply(rest);
    }
#pragma unroll
    for (int i = 0; i < MI; ++i) red[wave][i][lane] = acc[i];
    __syncthreads();
    if (wave < MI) {
        f32x4 s = red[0][wave][lane];
#pragma unroll
        for (int w = 1; w < NW; ++w) s += red[w][wave][lane];
        const int row = wave * 16 + r, col = j0 + 4 * c;
        if (row < a.m && col < a.n) {
            const float v[4] = {s[0], s[1], s[2], s[3]};
            store4(static_cast<O*>(a.y) + (int64_t)row * a.ldy + col, v, a.n - col);
        }
    }
}

}  // namespace qtcq
