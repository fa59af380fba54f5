// block_product.hpp -- the products of product.hpp for operands whose rows start on 16
// bytes and hold whole 16-byte chunks, in workgroup tiles of 32 FP x 256 (FP = 8, 4, 2),
// gfx950.
//
// Eight waves, 2 x 4, each 16 FP rows of P by 64 rows of Q (FP = 8: 128 accumulator
// registers a lane).  A step is 128 bytes of k.  Its half tiles, P's of 4 FP KB and Q's of
// 32 KB, go from memory straight to LDS (buffer loads with the lds bit), where P and Q have
// a ring of places each, together all of the compute unit's 160 KB: 3 and 2 at FP = 8, 3
// and 3 at FP = 4, 4 and 4 at FP = 2.
//
// A wave works in half steps of 64 bytes of k, with the next half step's fragments on
// their way from LDS to registers (two sets of 4 FP + 16) during the matrix instructions of
// the present one.  Step s:
//   read the fragments of its second half; matrix instructions of its first half;
//   wait until this wave's reads are done and its loads of step s + 1 have landed, barrier
//   (now step s + 1 is in LDS and step s's two places are free);
//   start the loads of the next half tiles into those places;
//   read the fragments of step s + 1's first half; matrix instructions of the second half.
// So at FP = 8 three half tiles are in flight during a step.  Steps of 64 bytes with five of
// them in LDS were slower (958 against 875 us on the 4096x14336x4096 gated product, even
// with all loads behind one wait there): each row's 128-byte line is then fetched twice.
// Half tiles past the last step are loaded as zeros (every lane out of range), which keeps
// the count of loads in flight the same.
//
// Where the tiles of out are fewer than the compute units, k is cut into shares of
// share_steps steps; each writes its sums in 32 bits, and join_shares adds them
// in order.
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
#include "product.hpp"

namespace qtcq {

struct BlockShape {
    static constexpr int kThreads = 512;
    static constexpr int kRows = 256;         // rows of Q in a tile
    static constexpr int kStep = 128;         // bytes of k in a step ([k][row] operands: 64 k)
    static constexpr int kTile = kRows * kStep;
    static constexpr int64_t kMaxStride = (int64_t)1 << 22;
    static constexpr int rows(int fp) { return 32 * fp; }
    static constexpr int cols(int mode) { return mode == kGated ? kRows / 2 : kRows; }
    // places of the two rings in LDS
    static constexpr int p_places(int fp) { return fp == 2 ? 4 : 3; }
    static constexpr int q_places(int fp) { return fp == 8 ? 2 : (fp == 4 ? 3 : 4); }
};

typedef __attribute__((address_space(3))) char lds_char;
typedef short s16x4 __attribute__((ext_vector_type(4)));

// The share of k and the tile of workgroup `b` of shares * tiles.  Consecutive workgroups go
// round the 8 XCDs, so XCD x takes a contiguous run of them: whole shares where there are
// several, whose tiles read the same rows of P (8-bit 77x8192x28672 46.3 us, with each
// share's tiles dealt round the XCDs 48.5), and within a share runs that go down groups of
// 8 tile rows, column by column, so that an XCD's concurrent tiles share operands in its L2
// (groups of 2, 4 and 8 are alike on the large products).
__device__ __forceinline__ void block_tile(int b, int shares, int tiles_m, int tiles_n, int& share, int& ti, int& tj)
{
    const int tiles = tiles_m * tiles_n, n = shares * tiles, x = b & 7, q = n >> 3, r = n & 7;
    int t = x * q + (x < r ? x : r) + (b >> 3);
    share = t / tiles;
    t -= share * tiles;
    constexpr int G = 8;
    const int per = G * tiles_n, g = t / per, first = g * G;
    const int rows = tiles_m - first < G ? tiles_m - first : G;
    const int in = t - g * per;
    ti = first + in % rows;
    tj = in / rows;
}

// LDS of a workgroup.
constexpr int block_lds_bytes(int fp)
{
    return BlockShape::p_places(fp) * BlockShape::rows(fp) * BlockShape::kStep + BlockShape::q_places(fp) * BlockShape::kTile;
}

// Workgroup b of shares * tiles (kGradW: of 2 * tiles, the gate's gradient first); lds has
// block_lds_bytes(FP).  FP = 8 for kGradW, whose P is stored [k][row].
template <typename T, typename O, int MODE, int ACT, int FP>
__device__ __forceinline__ void block_tile_product(const ProductArgs& a, int b, char* lds)
{
    typedef Mfma<T> MM;
    constexpr int TQ = BlockShape::kTile, TP = BlockShape::rows(FP) * BlockShape::kStep;
    constexpr int NPP = BlockShape::p_places(FP), NPQ = BlockShape::q_places(FP);
    constexpr int LP = FP / 2, LQ = 4;                   // loads of a half tile by one wave
    constexpr int SZ = (int)sizeof(T);
    constexpr int KS = BlockShape::kStep / SZ;           // k of a step
    constexpr bool PT = MODE == kGradW, QT = MODE == kGradX || MODE == kGradW;
    constexpr int COLS = BlockShape::cols(MODE);
    static_assert(!PT || FP == 8, "[k][row] tiles are 256 rows wide");

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave >> 2, wn = wave & 3;
    int share, ti, tj;
    block_tile(b, MODE == kGradW ? 2 : a.shares, (a.m + BlockShape::rows(FP) - 1) / BlockShape::rows(FP),
               (a.n + COLS - 1) / COLS, share, ti, tj);
    const int i0 = ti * BlockShape::rows(FP), j0 = tj * COLS;
    const int z = MODE == kGradW ? share : 0;
    const int steps1 = (a.k + KS - 1) / KS;
    const int steps = MODE == kGradX ? 2 * steps1 : steps1;
    // this workgroup's share of the steps; where P is in two pieces each of them is taken
    // twice, with the one and then the other (Q's half tile then comes from the L2)
    const int twice = MODE == kGradX || MODE == kGradW ? a.pieces - 1 : 0;
    const int first = MODE == kGradW ? 0 : share * a.share_steps;
    const int s0 = first << twice, s1 = (first + a.share_steps < steps ? first + a.share_steps : steps) << twice;
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
        // (m0 is a register the compiler does not give to values, which it warns about)
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                     ::"s"(at), "v"(off), "s"(r) : "m0", "memory");
#pragma clang diagnostic pop
    };
    // HR groups of 64 rows (of k) from row0 of `base` [nrows][k] into dst; nothing but zeros
    // if this step is not there
    auto stage_rows = [&](bool there, const void* base, int64_t ld, int row0, int nrows, int k, int k0, char* dst, auto hr) {
        constexpr int HR = decltype(hr)::value;
        const int left = there ? (k - k0) * SZ : 0;       // bytes of k from k0
        const u32x4 r = rsrc(static_cast<const char*>(base) + row0 * ld + (int64_t)k0 * SZ,
                             (nrows - row0 < 64 * HR ? nrows - row0 - 1 : 64 * HR - 1) * (int)ld + left);
        int off = rk_row * (int)ld + rk_chunk * 16;
        const bool out = rk_chunk * 16 >= left;
#pragma unroll
        for (int h = 0; h < HR; ++h)
            to_lds(r, dst + (64 * h + 8 * wave) * 128, out ? 0x7FFFFFFF : off + h * 64 * (int)ld);
    };
    auto stage_cols = [&](bool there, const void* base, int64_t ld, int row0, int nrows, int k0, char* dst) {
        const int left = !there ? 0 : (a.k - k0 < KS ? a.k - k0 : KS);
        const u32x4 r = rsrc(static_cast<const char*>(base) + k0 * ld + (int64_t)row0 * SZ,
                             left > 0 ? (left - 1) * (int)ld + (nrows - row0) * SZ : 0);
        const int off = ct_k * (int)ld + ct_chunk * 16;
#pragma unroll
        for (int h = 0; h < 4; ++h) to_lds(r, dst + (16 * h + 2 * wave) * 512, off + h * 16 * (int)ld);
    };
    // the half tiles of step s into place i of their ring
    auto stage_p = [&](int s, int i) {
        char* dst = lds + i * TP;
        const bool there = s < s1;
        const int t = s >> twice, seg = MODE == kGradX && t >= steps1 ? 1 : 0;
        const int k0 = (t - seg * steps1) * KS;
        const T* p = static_cast<const T*>(a.p[MODE == kGradW ? z : seg]) + ((s & twice) ? a.piece_step : 0);
        if constexpr (PT)
            stage_cols(there, p, ldp, i0, a.pm, k0, dst);
        else
            stage_rows(there, p, ldp, i0, a.m, a.pk, k0, dst, std::integral_constant<int, FP / 2>{});
    };
    auto stage_q = [&](int s, int i) {
        char* dst = lds + NPP * TP + i * TQ;
        const bool there = s < s1;
        const int t = s >> twice, seg = MODE == kGradX && t >= steps1 ? 1 : 0;
        const int k0 = (t - seg * steps1) * KS;
        if constexpr (MODE == kGated) {
            stage_rows(there, a.q[0], ldq, j0, a.n, a.qk, k0, dst, std::integral_constant<int, 2>{});
            stage_rows(there, a.q[1], ldq, j0, a.n, a.qk, k0, dst + TQ / 2, std::integral_constant<int, 2>{});
        } else if constexpr (QT) {
            stage_cols(there, a.q[seg], ldq, j0, a.qn, k0, dst);
        } else {
            stage_rows(there, a.q[0], ldq, j0, a.n, a.qk, k0, dst, std::integral_constant<int, 4>{});
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
    struct Frags { u32x4 p[FP], q[4]; };
    // the reads are issued here, ahead of the matrix instructions that follow (the compiler
    // would move each next to its use)
    auto read = [&](int ip, int iq, int half, Frags& f) {
        const char* tp = lds + ip * TP;
        const char* tq = lds + NPP * TP + iq * TQ;
#pragma unroll
        for (int j = 0; j < 4; ++j) f.q[j] = QT ? frag_cols(tq, qrow(j), half) : frag_rows(tq, qrow(j), half);
#pragma unroll
        for (int i = 0; i < FP; ++i)
            f.p[i] = PT ? frag_cols(tp, (wm * FP + i) * 16, half) : frag_rows(tp, (wm * FP + i) * 16, half);
        asm volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
    };
    typename MM::Acc acc[FP][4] = {};
    auto multiply = [&](const Frags& f) {
#pragma unroll
        for (int i = 0; i < FP; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = MM::mul(f.q[j], f.p[i], acc[i][j]);
    };
    // this wave's reads are done and all but its newest n loads have landed, then the same
    // of all waves
    auto landed = [&](auto n) {
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(decltype(n)::value) : "memory");
        __builtin_amdgcn_sched_barrier(0);
    };
    // The order of loads: P0 Q0 P1 Q1 ... where the rings are equally long, the last two
    // started in step s being P(s + NPP) Q(s + NPQ); with one more place for P (FP = 8)
    // the prologue ends in P2, and step s starts Q(s + 2) P(s + 3).  `after`: the loads
    // that follow those of step 0 in the prologue, `newer`: those that follow step s + 1's
    // when step s waits for them.
    constexpr bool AHEAD = NPP > NPQ;
    static_assert(NPP == NPQ || NPP == NPQ + 1, "ring lengths");
    constexpr int after = (NPP - 1) * LP + (NPQ - 1) * LQ;
    constexpr int newer = after - (LP + LQ);
    if (s0 < s1) {
        Frags f0, f1;
#pragma unroll
        for (int i = 0; i < NPP; ++i) {
            stage_p(s0 + i, i);
            if (i < NPQ) stage_q(s0 + i, i);
        }
        landed(std::integral_constant<int, after>{});
        int ip = 0, iq = 0;                   // places of step s
        read(0, 0, 0, f0);
        for (int s = s0; s < s1; ++s) {
            const int np = ip + 1 < NPP ? ip + 1 : 0, nq = iq + 1 < NPQ ? iq + 1 : 0;
            read(ip, iq, 1, f1);
            multiply(f0);
            landed(std::integral_constant<int, newer>{});
            if constexpr (AHEAD) stage_q(s + NPQ, iq);
            stage_p(s + NPP, ip);
            if constexpr (!AHEAD) stage_q(s + NPQ, iq);
            read(np, nq, 0, f0);
            multiply(f1);
            ip = np;
            iq = nq;
        }
        // nothing may still be on its way to LDS when the workgroup ends
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    }

    // a lane's results: rows row0 + 16 i, four columns from col0 + 16 j
    typedef typename MM::Acc Acc;
    constexpr int NJ = MODE == kGated ? 2 : 4;
    const int row0 = i0 + wm * FP * 16 + (lane & 15);
    const int col0 = j0 + (MODE == kGated ? wn * 32 : wn * 64) + 4 * (lane >> 4);
    if (MODE != kGradW && a.part) {
#pragma unroll
        for (int i = 0; i < FP; ++i) {
            const int row = row0 + i * 16;
            if (row >= a.m) continue;
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                const int col = col0 + j * 16;
                if (col >= a.n) continue;
                Acc* p = static_cast<Acc*>(a.part) + ((((int64_t)share * a.m + row) * a.part_pitch + col) >> 2);
                p[0] = acc[i][j];
                if constexpr (MODE == kGated) p[a.part_pitch >> 3] = acc[i][j + 2];
            }
        }
    } else if (sizeof(O) == 2 && i0 + BlockShape::rows(FP) <= a.m && j0 + COLS <= a.n) {
        // A whole tile of 16-bit results goes out through LDS, in whole rows of the tile
        // (a wave's own results are 32-byte pieces of 16 rows).  Rows are 16 bytes apart in
        // banks.
        constexpr int RB = COLS * 2, PITCH = RB + 16, LR = RB / 16, RW = 64 / LR;   // lanes a row, rows a wave
        static_assert(BlockShape::rows(FP) * PITCH <= block_lds_bytes(FP), "the tile fits LDS");
        float qs[NJ][4] = {};
        if constexpr (MODE == kInt8) {
#pragma unroll
            for (int j = 0; j < NJ; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) qs[j][e] = a.q_scale[col0 + j * 16 + e];
        }
        struct __attribute__((aligned(8))) Four { O e[4]; };
        struct __attribute__((packed, aligned(2))) Loose { u32x4 v; };
        auto put = [&](void* base, int64_t ld, auto value) {
            landed(std::integral_constant<int, 0>{});     // LDS is no longer read or loaded
#pragma unroll
            for (int i = 0; i < FP; ++i) {
                const float ps = MODE == kInt8 ? a.p_scale[row0 + i * 16] : 0.0f;
#pragma unroll
                for (int j = 0; j < NJ; ++j) {
                    Four f;
#pragma unroll
                    for (int e = 0; e < 4; ++e) f.e[e] = from_f32<O>(value(i, j, e, ps));
                    *reinterpret_cast<Four*>(lds + (row0 - i0 + i * 16) * PITCH + (col0 - j0 + j * 16) * 2) = f;
                }
            }
            __syncthreads();
            const int r = RW * wave + lane / LR, c = lane % LR;
            O* o = static_cast<O*>(base) + (int64_t)(i0 + r) * ld + j0 + c * 8;
#pragma unroll
            for (int h = 0; h < BlockShape::rows(FP) / (8 * RW); ++h) {
                reinterpret_cast<Loose*>(o)->v = *reinterpret_cast<const u32x4*>(lds + (r + h * 8 * RW) * PITCH + c * 16);
                o += 8 * RW * ld;
            }
        };
        put(a.out[z], a.ldo, [&](int i, int j, int e, float ps) {
            if constexpr (MODE == kGated) return activate<ACT>(acc[i][j][e]) * acc[i][j + 2][e];
            if constexpr (MODE == kInt8) return (float)acc[i][j][e] * ps * qs[j][e];
            return (float)acc[i][j][e];
        });
        if constexpr (MODE == kGated)
            if (a.save[0]) {
                put(a.save[0], a.lds, [&](int i, int j, int e, float) { return acc[i][j][e]; });
                put(a.save[1], a.lds, [&](int i, int j, int e, float) { return acc[i][j + 2][e]; });
            }
    } else {
#pragma unroll
        for (int i = 0; i < FP; ++i)
#pragma unroll
            for (int j = 0; j < NJ; ++j)
                if (row0 + i * 16 < a.m && col0 + j * 16 < a.n)
                    finish_at<O, MODE, ACT>(a, z, row0 + i * 16, col0 + j * 16, acc[i][j], acc[i][MODE == kGated ? j + 2 : j]);
    }
}

// grid.x = shares * tiles (kGradW: 2 * tiles); block = 512.
template <typename T, typename O, int MODE, int ACT, int FP>
__global__ void __launch_bounds__(BlockShape::kThreads)
block_product(ProductArgs a)
{
    __shared__ __align__(1024) char lds[block_lds_bytes(FP)];
    block_tile_product<T, O, MODE, ACT, FP>(a, blockIdx.x, lds);
}

// Both products of the gated gradient in one launch, the first nx workgroups grad_x's: they
// share no result, and small ones fill the chip together.
//   grid.x = nx + 2 * tiles of the weight gradients; block = 512.
template <typename T, int FP>
__global__ void __launch_bounds__(BlockShape::kThreads)
gradient_products(ProductArgs x, ProductArgs w, int nx)
{
    __shared__ __align__(1024) char lds[block_lds_bytes(8) > block_lds_bytes(FP) ? block_lds_bytes(8) : block_lds_bytes(FP)];
    const int b = blockIdx.x;
    if (b < nx)
        block_tile_product<T, T, kGradX, 0, FP>(x, b, lds);
    else
        block_tile_product<T, T, kGradW, 0, 8>(w, b - nx, lds);
}

}  // namespace qtcq
