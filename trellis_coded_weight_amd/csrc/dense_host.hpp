// dense_host.hpp -- host-side declarations of the dense operators, shared by their C ABI
// (qtcq_dense.hip) and their launch units (launch_rows.hip, launch_int8.hip,
// launch_gated.hip, launch_gated_vjp.hip).
#pragma once

#include "host.hpp"

namespace qtcq {
namespace host {

// Lengths a call may have: tile counts, row offsets inside a tile and element indices
// inside a row stay within 32 bits.
constexpr int kDenseMaxDim = 1 << 24;
// rows of the 16-bit products, in elements: 4 MB, so that a tile's offsets stay below 2^31
constexpr int kHalfMaxRow = 1 << 21;
// 2^14 K, the largest magnitude of a sum of K products of 8-bit integers, below 2^31
constexpr int kInt8MaxK = 131071;
// results of at most this many pieces of 8192 elements (the smallest tile of the block
// kernel): its threads stay below the 2^32 of a launch
constexpr int64_t kDenseMaxTiles = (int64_t)1 << 22;

// whole 16-byte chunks, in elements
inline int chunk_pitch(int cols, int size) { return (cols + 16 / size - 1) / (16 / size) * (16 / size); }
inline size_t round256(size_t n) { return (n + 255) / 256 * 256; }

// row stride of the two slope matrices of the gated gradient, in elements: whole steps
// of its products, zero-filled past F
inline int slope_pitch(int F) { return (F + 63) / 64 * 64; }

// ---- which kernel a product takes, and its scratch (product_launch.hpp) ----------------------
enum : int { kPlanInt8 = 0, kPlanGated = 1, kPlanGradX = 2, kPlanGradW = 3 };

struct ProductPlan {
    bool skinny;             // the kernel for few rows, which takes no scratch
    int fp;                  // block kernel: 32 fp rows a tile
    int shares, share_steps; // shares of k, and the steps of each
    int part_pitch;          // row pitch of the shares' sums
    size_t part_bytes;       // the shares' sums
    size_t p_bytes, q_bytes; // padded copies of the operands
};

// The compute units of the chip the tile and share counts are chosen for.
constexpr int kComputeUnits = 256;

// Whether the kernel for few rows, at most 64, takes a product.  It reads Q once at the memory's rate and
// P once for every 16 columns, so its time grows with m n k; the block kernel's hardly does
// up to 128 rows, but it pays for shares of k and a second launch.  Measured (us, few rows
// against block; m n k in bytes of the multiplied elements): 8-bit 8192x28672 at m = 1 44.5
// against 49.1, m = 8 (2^30.8) 51.8 / 48.2, m = 16 63.8 / 48.1; 28672x8192 at m = 8 52.7 /
// 52.2, 16 (2^31.8) 64.7 / 53.0; gated 14336x4096 at m = 8 (2^30.8) 51.5 / 51.9, 24 69.6 /
// 53.4; gated 4096x4096 at m = 32 (2^31) 22.8 / 23.0, 64 30.5 / 25.2.  Rows that are not whole
// chunks cost the block kernel a copy and this one slower loads: 28672x8193 at m = 1 106.8 /
// 143.9, 8 (2^30.8) 160.8 / 145.1; gated 4096x4097 at m = 16 (just past 2^30) 41.3 / 46.6, 32
// 53.2 / 48.0.
inline bool few_rows(int mode, int size, int m, int n, int k, bool whole)
{
    if (mode != kPlanInt8 && mode != kPlanGated) return false;
    const double work = (double)m * n * k * size * (mode == kPlanGated ? 2 : 1);
    return whole ? m <= 4 || (m <= 64 && work <= 0x1p31) : m <= 2 || (m <= 64 && work <= 0x1.1p30);
}

// mode, bytes of an element, rows and columns of the result, length of a sum; `whole`: the
// operands are whole 16-byte chunks as they are
inline ProductPlan plan_product(int mode, int size, int m, int n, int k, bool whole)
{
    ProductPlan p = {};
    if (few_rows(mode, size, m, n, k, whole)) {
        p.skinny = true;
        return p;
    }
    const int quads = (n + 3) / 4 * 4;
    p.part_pitch = mode == kPlanGated ? 2 * quads : quads;
    const int64_t cols = mode == kPlanGated ? 128 : 256;
    const int per = 128 / size;
    const int steps = (k + per - 1) / per * (mode == kPlanGradX ? 2 : 1);
    // The tile's rows and the shares of k by the shortest estimate, in us: rounds of
    // workgroups (one a compute unit) times a share's steps, each 0.7, 1.0 or 1.7 with 64, 128
    // or 256 rows (8-bit 8192x28672 at m = 2048: 616, 435 and 390 us in 4, 2 and 1 rounds of
    // 224 steps); shares cost a second launch, and their sums' way out and back at 4 TB/s.
    // [k][row] tiles of P are 256 rows wide.
    double best = 0;
    for (int fp = mode == kPlanGradW ? 8 : 2; fp <= 8; fp *= 2) {
        const int64_t tiles = ((int64_t)m + 32 * fp - 1) / (32 * fp) * ((n + cols - 1) / cols);
        const double step = fp == 2 ? 0.7 : (fp == 4 ? 1.0 : 1.7);
        int64_t most = mode == kPlanGradW || tiles == 0 ? 1 : kComputeUnits / tiles;
        if (most > steps / 4) most = steps / 4;
        for (int s = 1; s == 1 || s <= most; ++s) {
            const int share = steps > 0 ? (steps + s - 1) / s : 1, shares = steps > 0 ? (steps + share - 1) / share : 1;
            double t = (double)((tiles * shares + kComputeUnits - 1) / kComputeUnits) * (share + 2) * step;
            if (shares > 1) t += 6.0 + 8.0 * shares * m * p.part_pitch / 4e6;
            if (p.fp == 0 || t < best) best = t, p.fp = fp, p.shares = shares, p.share_steps = share;
        }
    }
    if (p.shares > 1) p.part_bytes = round256((size_t)p.shares * m * p.part_pitch * 4);
    if (mode == kPlanInt8 || mode == kPlanGated) {
        const size_t row = (size_t)chunk_pitch(k, size) * size;
        p.p_bytes = round256((size_t)m * row);
        p.q_bytes = round256((size_t)n * row) * (mode == kPlanGated ? 2 : 1);
    }
    return p;
}

inline size_t rows_product_bytes(int mode, int size, int m, int n, int k, bool whole)
{
    const ProductPlan p = plan_product(mode, size, m, n, k, whole);
    return p.part_bytes + (whole ? 0 : p.p_bytes + p.q_bytes);
}

// The gated gradient's scratch: d_gate and d_up, one after the other, in one or two parts, the shares of grad_x,
// copies of w_gate and w_up, and of x.
struct VjpPlan {
    size_t slopes, part, w_copy, x_copy;
    size_t bytes(bool w_whole, bool x_whole, bool want_x, bool want_w) const
    {
        return slopes + (want_x ? part + (w_whole ? 0 : 2 * w_copy) : 0) + (want_w && !x_whole ? x_copy : 0);
    }
};
inline VjpPlan plan_vjp(int M, int F, int K, int pieces)
{
    VjpPlan v;
    const size_t row = (size_t)chunk_pitch(K, 2) * 2;
    v.slopes = round256((size_t)2 * 2 * pieces * M * slope_pitch(F));
    v.w_copy = round256((size_t)F * row);
    v.x_copy = round256((size_t)M * row);
    v.part = plan_product(kPlanGradX, 2, M, K, F, true).part_bytes;
    return v;
}

struct GatedCall {
    const void *x, *w_gate, *w_up;
    int64_t ldx, ldw;
    int dtype, M, F, K, act;
    void* h;
    int64_t ldh;
    void *gate, *up;
    int64_t ldg;
};

struct GatedVjpCall {
    const void *x, *w_gate, *w_up, *gate, *up, *grad_h;
    int64_t ldx, ldw, ldg, ldgh;
    int dtype, M, F, K, act;
    int pieces;              // parts that d_gate and d_up are held in
    void *grad_x, *grad_w_gate, *grad_w_up;
    int64_t ldgx, ldgw;
};

qtcq_status launch_quantize_rows(const void* x, int dtype, int64_t rows, int cols, int64_t ldx, int8_t* q, int64_t ldq,
                                 float* scale, hipStream_t st);
qtcq_status launch_decode_matrix(int L, const CodeSel& code, bool tb, const uint32_t* bits, int M, int N, int dtype,
                                 void* w, int64_t ldw, float* scale, hipStream_t st);
qtcq_status launch_matmul_int8(const int8_t* a, int64_t lda, const float* a_scale, const int8_t* w, int64_t ldw,
                               const float* w_scale, int M, int N, int K, int dtype, void* y, int64_t ldy,
                               void* ws, size_t wsb, hipStream_t st);
// these check the workspace against what the call's pointers and strides need
qtcq_status launch_gated_forward(const GatedCall& c, void* ws, size_t wsb, hipStream_t st);
qtcq_status launch_gated_vjp(const GatedVjpCall& c, void* ws, size_t wsb, hipStream_t st);

}  // namespace host
}  // namespace qtcq
