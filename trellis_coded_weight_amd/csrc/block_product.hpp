// block_product.hpp -- the products of tile_product.hpp for operands whose rows start on
// 16 bytes and hold whole 16-byte chunks, in workgroup tiles of 256 x 256, gfx950.
//
// Eight waves, 2 x 4, each 128 rows of P by 64 rows of Q (128 accumulator registers a
// lane).  A step is 128 bytes of k: two half tiles of 32 KB, P's and Q's, which go from
// memory straight to LDS (buffer loads with the lds bit).  Half tiles 0, 1, 2, ... = P0, Q0,
// P1, Q1, ... take the five 32 KB places of the compute unit's LDS in turn.
//
// A wave works in half steps of 64 bytes of k, with the next half step's fragments on
// their way from LDS to registers (two sets of 48) during the matrix instructions of the
// present one.  Step s:
//   read the fragments of its second half; matrix instructions of its first half;
//   wait until this wave's reads are done and its loads of step s + 1 have landed, barrier
//   (now step s + 1 is in LDS and step s's two places are free);
//   start the loads of half tiles 2 s + 5 and 2 s + 6 into those places;
//   read the fragments of step s + 1's first half; matrix instructions of the second half.
// So three half tiles are in flight during a step.  Steps of 64 bytes with five of them in
// LDS were slower (958 against 875 us on the 4096x14336x4096 gated product, even with all
// loads behind one wait there): each row's 128-byte line is then fetched twice.  Half tiles
// past the last step are loaded as zeros (every lane out of range), which keeps the count
// of loads in flight the same.
//
// LDS holds an operand in one of two layouts, both written by the loads in whole kilobytes
// of consecutive lanes, so the order inside a tile is chosen by which chunk of memory each
// lane fetches:
//   rows of k  (operand stored [row][k])  row r at 128 r, its 16-byte chunk c at place
//              c ^ ((r >> 1) & 7): the 16 lanes that read one chunk of 16 rows at once
//              (ds_read_b128) touch 16 different places of the 256-byte bank row;
//   columns    (operand stored [k][row])  k at 512 k, its 32-byte block b (16 rows) at place
//              b ^ h(k), h = (k & 3) | (k >> 3 & 1) << 2; ds_read_b64_tr_b16 hands lane j of
//              each 16 the four k of row j, from four such blocks; h spreads the eight
//              k that two groups of 16 lanes read over the banks.
//
// Reads past an operand's rows or its last k return zero by the buffer descriptor's range
// check (offsets of chunks past the end of k inside a row are moved out of range).  The
// descriptor is rebased each step, so offsets stay within a tile: below 2^31 for row
// strides up to kMaxStride bytes.
#pragma once

#include <type_traits>

#include "codes.hpp"
#include "tile_product.hpp"

namespace qtcq {

struct BlockShape {
    static constexpr int kThreads = 512;
    static constexpr int kRows = 256;         // rows of P and of Q in a tile
    static constexpr int kStep = 128;         // bytes of k in a step ([k][row] operands: 64 k)
    static constexpr int kTile = kRows * kStep;
    static constexpr int kPlaces = 5;         // half tiles in LDS: 5 x 32 KB
    static constexpr int kLoads = 4;          // loads of a half tile by one wave
    static constexpr int64_t kMaxStride = (int64_t)1 << 22;
    static constexpr int cols(int mode) { return mode == kGated ? kRows / 2 : kRows; }
};

typedef __attribute__((address_space(3))) char lds_char;
typedef short s16x4 __attribute__((ext_vector_type(4)));

// The tile of workgroup `b` of `n`: consecutive workgroups go round the 8 XCDs, so XCD x
// takes a contiguous run of tiles; runs go down groups of 8 tile rows, column by column,
// so that an XCD's concurrent tiles share operands in its L2.
__device__ __forceinline__ void block_tile(int b, int tiles_m, int tiles_n, int& ti, int& tj)
{
    const int n = tiles_m * tiles_n, x = b & 7, q = n >> 3, r = n & 7;
    const int t = x * q + (x < r ? x : r) + (b >> 3);
    constexpr int G = 8;
    const int per = G * tiles_n, g = t / per, first = g * G;
    const int rows = tiles_m - first < G ? tiles_m - first : G;
    const int in = t - g * per;
    ti = first + in % rows;
    tj = in / rows;
}

// grid.x = tiles, grid.z = 2 for kGradW; block = 512.
template <typename T, typename O, int MODE, int ACT = 0>
__global__ void __launch_bounds__(BlockShape::kThreads)
block_product(ProductArgs a)
{
    typedef Mfma<T> MM;
    constexpr int R = BlockShape::kRows, TILE = BlockShape::kTile, NP = BlockShape::kPlaces;
    constexpr int SZ = (int)sizeof(T);
    constexpr int KS = BlockShape::kStep / SZ;           // k of a step
    constexpr bool PT = MODE == kGradW, QT = MODE == kGradX || MODE == kGradW;
    constexpr int COLS = BlockShape::cols(MODE);
    __shared__ __align__(1024) char lds[NP * TILE];

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave >> 2, wn = wave & 3;
    int ti, tj;
    block_tile(blockIdx.x, (a.m + R - 1) / R, (a.n + COLS - 1) / COLS, ti, tj);
    const int i0 = ti * R, j0 = tj * COLS;
    const int z = MODE == kGradW ? blockIdx.z : 0;
    const int steps1 = (a.k + KS - 1) / KS;
    const int steps = MODE == kGradX ? 2 * steps1 : steps1;
    const int64_t ldp = a.ldp * SZ, ldq = a.ldq * SZ;     // in bytes

    // where a lane's chunks come from: row-of-k tiles, row 64 h + 8 wave + lane / 8;
    // column tiles, k 16 h + 2 wave + lane / 32
    const int rk_row = 8 * wave + (lane >> 3);
    const int rk_chunk = (lane & 7) ^ (((wave & 1) << 2) | (lane >> 4));
    const int ct_k = 2 * wave + (lane >> 5);
    const int ct_h = (ct_k & 3) | ((wave >> 2) << 2);
    const int ct_chunk = ((((lane & 31) >> 1) ^ ct_h) << 1) | (lane & 1);

    // A raw buffer descriptor of `bytes` from p (both the same in every lane).  Sizes fit
    // 32 bits: a tile's rows or a step's k, times at most kMaxStride.
    auto rsrc = [](const char* p, int bytes) {
        const uint64_t at = reinterpret_cast<uint64_t>(p);
        return u32x4{(uint32_t)at, (uint32_t)(at >> 32) & 0xFFFFu, (uint32_t)bytes, (uint32_t)kRawBufferWord3};
    };
    // 16 bytes a lane from r + off to LDS at dst + 16 lane.  Written out because the compiler
    // would wait for all such loads ahead of every ds_read_b64_tr_b16; `landed` below waits
    // for the ones that matter.  It has no output register: the data goes to LDS.
    auto to_lds = [&](u32x4 r, const char* dst, int off) {
        const uint32_t at = (uint32_t)reinterpret_cast<uintptr_t>((lds_char*)dst);
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                     ::"s"(at), "v"(off), "s"(r) : "memory", "m0");
    };
    // HR groups of 64 rows (of k) from row0 of `base` [nrows][k] into dst
    auto stage_rows = [&](const void* base, int64_t ld, int row0, int nrows, int k, int k0, char* dst, auto hr) {
        const int left = (k - k0) * SZ;                 // bytes of k from k0
        const u32x4 r = rsrc(static_cast<const char*>(base) + row0 * ld + (int64_t)k0 * SZ,
                                              (nrows - row0 < R ? nrows - row0 - 1 : R - 1) * (int)ld + left);
        int off = rk_row * (int)ld + rk_chunk * 16;
        const bool out = rk_chunk * 16 >= left;           // every lane past the last step
#pragma unroll
        for (int h = 0; h < decltype(hr)::value; ++h)
            to_lds(r, dst + (64 * h + 8 * wave) * 128, out ? 0x7FFFFFFF : off + h * 64 * (int)ld);
    };
    auto stage_cols = [&](const void* base, int64_t ld, int row0, int nrows, int k0, char* dst) {
        const int left = a.k - k0 < KS ? a.k - k0 : KS;
        const u32x4 r = rsrc(static_cast<const char*>(base) + k0 * ld + (int64_t)row0 * SZ,
                                              left > 0 ? (left - 1) * (int)ld + (nrows - row0) * SZ : 0);
        const int off = ct_k * (int)ld + ct_chunk * 16;
#pragma unroll
        for (int h = 0; h < 4; ++h) to_lds(r, dst + (16 * h + 2 * wave) * 512, off + h * 16 * (int)ld);
    };
    // half tile 2 s (P) or 2 s + 1 (Q) into a place
    auto stage_p = [&](int s, int place) {
        char* dst = lds + place * TILE;
        const int seg = MODE == kGradX && s >= steps1 ? 1 : 0;
        const int k0 = (s - seg * steps1) * KS;
        const void* p = a.p[MODE == kGradW ? z : seg];
        if constexpr (PT)
            stage_cols(p, ldp, i0, a.m, k0, dst);
        else
            stage_rows(p, ldp, i0, a.m, MODE == kGradX ? a.kp : a.k, k0, dst, std::integral_constant<int, 4>{});
    };
    auto stage_q = [&](int s, int place) {
        char* dst = lds + place * TILE;
        const int seg = MODE == kGradX && s >= steps1 ? 1 : 0;
        const int k0 = (s - seg * steps1) * KS;
        if constexpr (MODE == kGated) {
            stage_rows(a.q[0], ldq, j0, a.n, a.k, k0, dst, std::integral_constant<int, 2>{});
            stage_rows(a.q[1], ldq, j0, a.n, a.k, k0, dst + TILE / 2, std::integral_constant<int, 2>{});
        } else if constexpr (QT) {
            stage_cols(a.q[seg], ldq, j0, a.n, k0, dst);
        } else {
            stage_rows(a.q[0], ldq, j0, a.n, a.k, k0, dst, std::integral_constant<int, 4>{});
        }
    };

    // first row of Q's group j of 16 (kGated: two gate groups, the two up groups beside them)
    auto qrow = [&](int j) { return MODE == kGated ? (j >> 1) * 128 + wn * 32 + (j & 1) * 16 : wn * 64 + j * 16; };
    // LDS address of a lane's 16 bytes: rows of k, the two halves of a step
    const int rk0 = (lane & 15) * 128 + (((lane >> 4) ^ ((lane >> 1) & 7)) * 16);
    const int rk1 = rk0 ^ 64;
    // columns: k 8 (lane / 16) + (lane / 4 & 3) of a half step, block b of 16 rows
    const int ct_hr = ((lane >> 2) & 3) | (((lane >> 4) & 1) << 2);
    const int ct0 = (8 * (lane >> 4) + ((lane >> 2) & 3)) * 512 + (lane & 3) * 8;
    auto frag_rows = [&](const char* t, int row, int half) {
        return *reinterpret_cast<const u32x4*>(t + row * 128 + (half ? rk1 : rk0));
    };
    auto frag_cols = [&](const char* t, int row, int half) {
        const char* p = t + ct0 + (((row >> 4) ^ ct_hr) << 5) + half * 32 * 512;
        const u32x2 lo = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (__attribute__((address_space(3))) s16x4*)(lds_char*)const_cast<char*>(p)));
        const u32x2 hi = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (__attribute__((address_space(3))) s16x4*)(lds_char*)const_cast<char*>(p + 4 * 512)));
        return u32x4{lo.x, lo.y, hi.x, hi.y};
    };
    struct Frags { u32x4 p[8], q[4]; };
    // the reads are issued here, ahead of the matrix instructions that follow (the compiler
    // would move each next to its use)
    auto read = [&](int pp, int pq, int half, Frags& f) {
        const char* tp = lds + pp * TILE;
        const char* tq = lds + pq * TILE;
#pragma unroll
        for (int j = 0; j < 4; ++j) f.q[j] = QT ? frag_cols(tq, qrow(j), half) : frag_rows(tq, qrow(j), half);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            f.p[i] = PT ? frag_cols(tp, wm * 128 + i * 16, half) : frag_rows(tp, wm * 128 + i * 16, half);
        asm volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
    };
    typename MM::Acc acc[8][4] = {};
    auto multiply = [&](const Frags& f) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = MM::mul(f.q[j], f.p[i], acc[i][j]);
    };
    // this wave's reads are done and all but its newest n half tiles' loads have landed,
    // then the same of all waves
    auto landed = [&](auto n) {
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(decltype(n)::value * BlockShape::kLoads) : "memory");
        __builtin_amdgcn_sched_barrier(0);
    };
    auto place = [&](int p) { return p < NP ? p : p - NP; };
    if (steps > 0) {
        Frags f0, f1;
        stage_p(0, 0);
        stage_q(0, 1);
        stage_p(1, 2);
        stage_q(1, 3);
        stage_p(2, 4);
        landed(std::integral_constant<int, 3>{});
        int pp = 0;                           // the place of P of step s; Q's is the next
        read(0, 1, 0, f0);
        for (int s = 0; s < steps; ++s) {
            const int pq = place(pp + 1), np = place(pp + 2), nq = place(pp + 3);
            read(pp, pq, 1, f1);
            multiply(f0);
            landed(std::integral_constant<int, 1>{});
            stage_q(s + 2, pp);
            stage_p(s + 3, pq);
            read(np, nq, 0, f0);
            multiply(f1);
            pp = np;
        }
        // nothing may still be on its way to LDS when the workgroup ends
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    }

    constexpr int NJ = MODE == kGated ? 2 : 4;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int row = i0 + wm * 128 + i * 16 + (lane & 15);
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

}  // namespace qtcq
