// fp8_block.hpp -- the product of e4m3 matrices with block scales for any number of rows, in
// workgroup tiles of 32 FP x 64 QG (256 or 128 columns), for operands whose rows start on 16
// bytes and hold whole 16-byte chunks, gfx950.
//
// Eight waves, 2 x 4, each 16 FP rows of a by 16 QG rows of w.  A step is one block of 128 of
// k.  Its tiles (a's 4 FP KB, w's 8 QG KB) and its scales go from memory straight to LDS, into a
// ring of 2 to 4 places, so the next one to three steps are on their way during a step.
// LDS rows are 128 bytes, their 16-byte chunk c at place c ^ ((row >> 1) & 7): the 16 lanes
// that read one chunk of 16 rows at once touch 16 different places of the 256-byte bank row.
//
// Within a step a wave holds its QG groups of 16 rows of w in registers and takes its rows of
// a two groups at a time, the next two on their way from LDS meanwhile.  When the last two
// are read, all reads of the step are done: wait until the next step has landed, barrier, and
// between the products that are left start the loads of a later step into the places just
// left and read the next step's first groups, each of w's as this step's is done with.
//
// A block's sums must be scaled before they are added to the result's, which are therefore
// ordinary vector registers: one fused multiply-add an element and block beside the matrix
// instructions (four after each).
//
// Where tiles are fewer than the compute units, k is cut into shares; each writes its sums in
// 32 bits, and join_shares adds them in order.
//
// 4096x28672x8192 to bf16, in calls in a row: 774 us, 2.49 PFLOP/s, the matrix cores 67% busy at 1.7
// to 1.8 GHz (on operands of zeros 615 us at 2.4 GHz): power bounds it.  After a pause launches take
// 766 to 1045 us, until the clock has settled some 30 launches on.  A loop of the instruction with its four
// scaled additions and nothing else reaches 3.75 PFLOP/s on random operands; in tiles of 32 x 32
// 3.34.  93x8192x14336 to fp16: 24 us and 4.5 for the shares, w at 4.9 TB/s.  Smaller tiles are
// bound by the loads to LDS: 128 x 128 tiles take 0.64 us a step, their loads alone 0.45 to 0.58
// (13 to 14 TB/s over the chip), the rest alone 0.5; a second set of registers, read a step
// ahead, did not shorten it.
#pragma once

#include <type_traits>

#include "block_product.hpp"
#include "fp8_product.hpp"

namespace qtcq {

// FP: 32 FP rows a tile; QG: 64 QG columns (a wave's groups of 16 rows of w).
struct Fp8Shape {
    static constexpr int kThreads = 512;
    static constexpr int kScales = 2048;      // bytes of a step's scales: 64 floats a wave
    static constexpr int rows(int fp) { return 32 * fp; }
    static constexpr int cols(int qg) { return 64 * qg; }
    static constexpr int places(int fp, int qg) { return fp == 8 ? 2 : (qg == 4 ? 3 : 4); }
    static constexpr int step_bytes(int fp, int qg) { return (rows(fp) + cols(qg)) * 128 + kScales; }
};

// grid.x = shares * tiles, block = 512
template <typename O, int FP, int QG, bool FAST>
__global__ void __launch_bounds__(Fp8Shape::kThreads)
fp8_block_product(Fp8Args a)
{
    typedef BlockOperand<FAST> Op;
    constexpr int ROWS = Fp8Shape::rows(FP), COLS = Fp8Shape::cols(QG);
    constexpr int R = Fp8Shape::places(FP, QG), STEP = Fp8Shape::step_bytes(FP, QG);
    constexpr int TP = ROWS * 128, TQ = COLS * 128;
    constexpr int LP = FP / 2, LQ = QG, LOADS = LP + LQ + 1;     // loads of a step by one wave
    constexpr int PAIRS = FP / 2;
    __shared__ __align__(1024) char lds[R * STEP];

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave >> 2, wn = wave & 3;
    int share, ti, tj;
    block_tile(blockIdx.x, a.shares, (a.m + ROWS - 1) / ROWS, (a.n + COLS - 1) / COLS, share, ti, tj);
    const int i0 = ti * ROWS, j0 = tj * COLS;
    const int steps = (a.k + 127) / 128;
    const int s0 = share * a.share_steps, s1 = s0 + a.share_steps < steps ? s0 + a.share_steps : steps;

    // What the loads of the step to be started next read: raw buffer descriptors of each
    // operand from its tile's row i0 (j0) and the step's k on, and of the scales, moved on by
    // one step at a time.  Their sizes end with the last row's last byte, or are 0 past the
    // last step.
    const int a_rows = a.m - i0 < ROWS ? a.m - i0 : ROWS, w_rows = a.n - j0 < COLS ? a.n - j0 : COLS;
    const bool of_w = wave == 4;               // its floats are w's two scales, waves 0 .. FP / 2 - 1 have a's
    const int s_rows = of_w ? (w_rows > 128 ? 2 : 1) : (wave < FP / 2 ? a_rows : 0);
    const int s_ld = (int)(of_w ? a.ws_row : a.as_row) * 4;
    const int64_t s_step = (of_w ? a.ws_col : a.as_col) * 4;
    auto rsrc = [](const void* p, int bytes) {
        const uint64_t at = reinterpret_cast<uint64_t>(p);
        return u32x4{(uint32_t)at, (uint32_t)(at >> 32) & 0xFFFFu, (uint32_t)bytes, (uint32_t)kRawBufferWord3};
    };
    u32x4 src_a = rsrc(a.a + i0 * a.lda + (int64_t)s0 * 128, (a_rows - 1) * (int)a.lda + a.ak - s0 * 128);
    u32x4 src_w = rsrc(a.w + j0 * a.ldw + (int64_t)s0 * 128, (w_rows - 1) * (int)a.ldw + a.wk - s0 * 128);
    u32x4 src_s = rsrc(reinterpret_cast<const char*>(of_w ? a.w_scale + (j0 >> 7) * a.ws_row : a.a_scale + i0 * a.as_row) + s0 * s_step,
                       s_rows > 0 ? (s_rows - 1) * s_ld + 4 : 0);
    // where a lane's chunks come from: row 64 h + 8 wave + lane / 8 of a tile
    const int from_row = 8 * wave + (lane >> 3);
    const int from_chunk = ((lane & 7) ^ (((wave & 1) << 2) | (lane >> 4))) * 16;
    int off_a[LP], off_w[LQ];
#pragma unroll
    for (int h = 0; h < LP; ++h) off_a[h] = (from_row + 64 * h) * (int)a.lda + from_chunk;
#pragma unroll
    for (int h = 0; h < LQ; ++h) off_w[h] = (from_row + 64 * h) * (int)a.ldw + from_chunk;
    // a's scales lie as the lanes take them: FP groups' of one row of 16 together
    const int s_at = wave * 64 + lane, s_row = of_w ? lane : s_at / (16 * FP) * (16 * FP) + s_at % FP * 16 + s_at / FP % 16;
    const int off_s = s_row < s_rows ? s_row * s_ld : 0x7FFFFFFF;
    // where k ends inside step s, chunks past the rows' ends go out of range
    auto mask_end = [&](int s) {
        const bool in_a = from_chunk < a.ak - s * 128, in_w = from_chunk < a.wk - s * 128;
#pragma unroll
        for (int h = 0; h < LP; ++h) off_a[h] = in_a ? off_a[h] : 0x7FFFFFFF;
#pragma unroll
        for (int h = 0; h < LQ; ++h) off_w[h] = in_w ? off_w[h] : 0x7FFFFFFF;
    };
    // the descriptors on to step s, which may be past the last
    auto advance = [&](int s) {
        auto add = [](u32x4& r, int64_t n) {
            const uint64_t at = (r.x | (uint64_t)r.y << 32) + n;
            r.x = (uint32_t)at;
            r.y = (uint32_t)(at >> 32) & 0xFFFFu;
        };
        add(src_a, 128);
        add(src_w, 128);
        add(src_s, s_step);
        const bool there = s < s1;
        src_a.z = there ? src_a.z - 128 : 0;
        src_w.z = there ? src_w.z - 128 : 0;
        src_s.z = there ? src_s.z : 0;
        mask_end(s);
    };
    // Load l of a step: 16 bytes a lane of a's tile, then of w's, then a float of the scales,
    // from the descriptors to the places of LDS that start at `place` + 1 KB a wave.  Counted
    // by `landed`.
    const uint32_t lds0 = (uint32_t)reinterpret_cast<uintptr_t>((lds_char*)lds);
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
    auto stage = [&](int i, int l) {
        const uint32_t at = lds0 + i * STEP + (l < LP + LQ ? wave * 1024 : wave * 256);
        if (l < LP + LQ)
            asm volatile("s_add_u32 m0, %0, %3\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                         ::"s"(at), "v"(l < LP ? off_a[l] : off_w[l - LP]), "s"(l < LP ? src_a : src_w),
                         "i"(l < LP ? l * 8192 : TP + (l - LP) * 8192) : "m0", "scc", "memory");
        else
            asm volatile("s_add_u32 m0, %0, %3\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds"
                         ::"s"(at), "v"(off_s), "s"(src_s), "i"(TP + TQ) : "m0", "scc", "memory");
    };
#pragma clang diagnostic pop

    // LDS address of a lane's two chunks of a row group
    const int at0 = (lane & 15) * 128 + (((lane >> 4) ^ ((lane >> 1) & 7)) * 16), at1 = at0 ^ 64;
    auto read = [&](const char* tile, int row) {
        return Op(*reinterpret_cast<const u32x4*>(tile + row * 128 + at0), *reinterpret_cast<const u32x4*>(tile + row * 128 + at1));
    };
    auto read_a = [&](int i, int g) { return read(lds + i * STEP, (wm * FP + g) * 16); };
    auto read_w = [&](int i, int g) { return read(lds + i * STEP + TP, wn * 16 * QG + g * 16); };
    // a step's scales as they lie in LDS: of a lane's FP rows of a, and of the wave's block of w
    struct __attribute__((aligned(FP < 4 ? 8 : 16))) RowScales { float f[FP]; };
    struct Scales { RowScales a; float w; };
    auto read_scales = [&](int i) {
        const char* s = lds + i * STEP + TP + TQ;
        return Scales{reinterpret_cast<const RowScales*>(s)[wm * 16 + (lane & 15)], reinterpret_cast<const float*>(s)[256 + (wn * 16 * QG >> 7)]};
    };
    // reads are issued ahead of the matrix instructions that follow
    auto fence = [] {
        asm volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
    };
    // this wave's reads are done and all but its newest n loads have landed, then the same of
    // all waves
    auto landed = [&](auto n) {
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(decltype(n)::value) : "memory");
        __builtin_amdgcn_sched_barrier(0);
    };
    // Product n of a step's QG FP: rows' group 2 (n / PAIR) + n % 2 by w's group n % PAIR / 2, so
    // that a group of w is needed as late as can be after it was read.  Its scaled addition follows
    // LAG products later (into the next step for the last ones), when its result has come out:
    // no wait for it, and between the issue of others.
    constexpr int LAG = 3, PAIR = 2 * QG, TOTAL = QG * FP, TAIL = TOTAL - PAIR;
    f32x4 acc[FP][QG] = {}, sums[LAG + 1] = {};
    float f[FP], late[2] = {0.0f, 0.0f};          // scales, and the last two of the step before
    auto issue = [&](int n, const Op& q, const Op& p) { sums[n % (LAG + 1)] = Op::mul(q, p); };
    auto add = [&](int n, float scale) {
        const int g = 2 * (n / PAIR) + n % 2, j = n % PAIR / 2;
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[g][j][e] = __builtin_fmaf(sums[n % (LAG + 1)][e], scale, acc[g][j][e]);
    };
    // what follows product n
    auto retire = [&](int n) {
        if (n >= LAG)
            add(n - LAG, f[2 * ((n - LAG) / PAIR) + (n - LAG) % 2]);
        else
            add(TOTAL + n - LAG, late[(TOTAL + n - LAG) % 2]);
        __builtin_amdgcn_sched_barrier(0);
    };
    if (s0 < s1) {
        mask_end(s0);
#pragma unroll
        for (int i = 0; i < R; ++i) {
#pragma unroll
            for (int l = 0; l < LOADS; ++l) stage(i, l);
            advance(s0 + i + 1);
        }
        landed(std::integral_constant<int, (R - 1) * LOADS>{});
        Op q[QG];
#pragma unroll
        for (int j = 0; j < QG; ++j) q[j] = read_w(0, j);
        Op p[2][2] = {{read_a(0, 0), read_a(0, 1)}, {read_a(0, 0), read_a(0, 1)}};
        {
            const Scales c = read_scales(0);
#pragma unroll
            for (int g = 0; g < FP; ++g) f[g] = c.a.f[g] * c.w;
        }
        // product AT is the first behind the barrier: six after the reads of the last pair
        constexpr int AT = TOTAL > 10 ? TOTAL - 10 : 0;
        int at = 0;                               // place of step s
        for (int s = s0; s < s1; ++s) {
            const int next = at + 1 < R ? at + 1 : 0;
            Op n0 = p[0][0], n1 = p[0][1];
            Scales c = {};
#pragma unroll
            for (int n = 0; n < TOTAL; ++n) {
                const int u = n / PAIR, i = n % PAIR;
                if (i == 0 && u < PAIRS - 1) {
                    p[(u + 1) & 1][0] = read_a(at, 2 * u + 2);
                    p[(u + 1) & 1][1] = read_a(at, 2 * u + 3);
                    fence();
                }
                if (n == AT) landed(std::integral_constant<int, (R - 2) * LOADS>{});
                issue(n, q[i / 2], p[u & 1][i % 2]);
                // beside the products: the loads of a later step into the places just left, and the
                // reads of the next step, a group of w as the one of this step is done with
#pragma unroll
                for (int l = 0; l < LOADS; ++l)
                    if (n == AT + l * (TOTAL - AT) / LOADS) stage(at, l);
                if (n == TAIL + 1) {
                    n0 = read_a(next, 0);
                    n1 = read_a(next, 1);
                    c = read_scales(next);
                }
                if (n >= TAIL && i % 2 == 1) q[i / 2] = read_w(next, i / 2);
                asm volatile("" ::: "memory");
                retire(n);
            }
            advance(s + R + 1);
            late[0] = f[FP - 2];
            late[1] = f[FP - 1];
#pragma unroll
            for (int g = 0; g < FP; ++g) f[g] = c.a.f[g] * c.w;
            p[0][0] = n0;
            p[0][1] = n1;
            at = next;
        }
#pragma unroll
        for (int n = 0; n < LAG; ++n) add(TOTAL + n - LAG, late[(TOTAL + n - LAG) % 2]);
        // nothing may still be on its way to LDS when the workgroup ends
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    }

    // a lane's results: rows row0 + 16 g, four columns from col0 + 16 j
    const int row0 = i0 + wm * FP * 16 + (lane & 15), col0 = j0 + wn * 16 * QG + 4 * (lane >> 4);
    if (a.part) {
#pragma unroll
        for (int g = 0; g < FP; ++g) {
            const int row = row0 + g * 16;
            if (row >= a.m) continue;
#pragma unroll
            for (int j = 0; j < QG; ++j) {
                const int col = col0 + j * 16;
                if (col < a.n)
                    *reinterpret_cast<f32x4*>(a.part + ((int64_t)share * a.m + row) * a.part_pitch + col) = acc[g][j];
            }
        }
    } else if (j0 + COLS <= a.n) {
        // results of all the tile's columns go out through LDS, in whole rows of the tile
        constexpr int E = 16 / (int)sizeof(O), PITCH = COLS * (int)sizeof(O) + 16;
        static_assert(ROWS * PITCH <= R * STEP, "the tile fits LDS");
        struct __attribute__((aligned(4 * sizeof(O)))) Four { O e[4]; };
        struct __attribute__((packed, aligned(sizeof(O)))) Loose { u32x4 v; };
        landed(std::integral_constant<int, 0>{});         // LDS is no longer read or loaded
#pragma unroll
        for (int g = 0; g < FP; ++g)
#pragma unroll
            for (int j = 0; j < QG; ++j) {
                Four o;
#pragma unroll
                for (int e = 0; e < 4; ++e) o.e[e] = from_f32<O>(acc[g][j][e]);
                *reinterpret_cast<Four*>(lds + (row0 - i0 + g * 16) * PITCH + (col0 - j0 + j * 16) * (int)sizeof(O)) = o;
            }
        __syncthreads();
        constexpr int LR = COLS / E, RW = 64 / LR;        // lanes a row, rows a wave
        const int r = RW * wave + lane / LR, c = lane % LR;
        O* o = static_cast<O*>(a.y) + (int64_t)(i0 + r) * a.ldy + j0 + c * E;
#pragma unroll
        for (int h = 0; h < ROWS / (8 * RW); ++h) {
            if (i0 + r + h * 8 * RW < a.m)
                reinterpret_cast<Loose*>(o)->v = *reinterpret_cast<const u32x4*>(lds + (r + h * 8 * RW) * PITCH + c * 16);
            o += 8 * RW * a.ldy;
        }
    } else {
#pragma unroll
        for (int g = 0; g < FP; ++g)
#pragma unroll
            for (int j = 0; j < QG; ++j)
                if (row0 + g * 16 < a.m && col0 + j * 16 < a.n) {
                    const float v[4] = {acc[g][j][0], acc[g][j][1], acc[g][j][2], acc[g][j][3]};
                    store4(static_cast<O*>(a.y) + (int64_t)(row0 + g * 16) * a.ldy + col0 + j * 16, v, a.n - (col0 + j * 16));
                }
    }
}

}  // namespace qtcq
