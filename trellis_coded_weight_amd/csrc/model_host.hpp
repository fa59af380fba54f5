// model_host.hpp -- host-side declarations of the model operators (8-bit floating point with
// block scales, layer norm, distillation), shared by their C ABI (qtcq_model.hip) and their
// launch units (launch_blocks.hip, launch_fp8.hip, launch_norm.hip, launch_distill.hip).
#pragma once

#include "dense_host.hpp"
#include "model_args.hpp"

namespace qtcq {

namespace host {

// row strides of the scales a product takes, in elements: 256 rows of them stay within 31
// bits of bytes
constexpr int64_t kScaleMaxStride = (int64_t)1 << 20;
// K of the e4m3 product: rows of 4 MB, so that a tile's offsets stay below 2^31
constexpr int kFp8MaxK = 1 << 22;

// elements of a matrix to be quantized: its pieces are counted in 32 bits
constexpr int64_t kBlocksMaxElements = (int64_t)1 << 40;

inline int scale_blocks(int n) { return n / 128 + (n % 128 != 0); }

// Which kernel a product takes, and its scratch (launch_fp8.hip).
struct Fp8Plan {
    bool skinny;             // the kernel for few rows, which takes no scratch
    int fp, qg;              // block kernel: 32 fp rows by 64 qg columns a tile
    int shares, share_steps; // shares of k, and the blocks of each
    int part_pitch;          // row pitch of the shares' sums
    size_t part_bytes;       // the shares' sums
    size_t a_bytes, w_bytes; // padded copies of the operands
};

// Whether the kernel for few rows takes a product.  It reads w once at the memory's rate and a
// once for every 16 columns, in a wave's registers, so its time grows with the groups of 16
// rows and their length; the tiles pay for shares of k and a second launch, which many columns
// need not (us, few rows against tiles: 28672x8192 at m = 8 48.5 / 50.8, 16 59.8 / 49.7; 8192x8192
// at m = 12 (1.5 2^29) 16.4 / 16.9, 16 17.6 / 16.9; 4096x8192 at m = 24 (1.5 2^29) 12.3 / 13.8;
// 8192x4096 at m = 32 (2^30) 14.5 / 13.7; 4096x4096 at m = 64 12.8 / 14.3; 1024x8192 at m = 64
// 21.3 / 13.9; 14336x1024 at m = 48 14.3 / 10.9).  Rows that are not whole chunks cost the tiles
// a copy and this kernel slower loads: 8192x8193 at m = 4 43.4 / 43.5, 8 48.7 / 43.7; 4096x4097 at
// m = 24 (1.5 2^28) 21.4 / 22.3; 4096x2047 at m = 40 16.7 / 19.2; 2000x2047 at m = 64 20.5 / 16.6.
// Past 22528 columns the groups of 16 columns a compute unit takes in turn are the time, and a
// tile of 128 needs no shares (16 bits: 16x20480x2048 12.8 / 14.6, 24x20480x1024 11.6 / 11.0, 9x24576x2048
// 13.0 / 11.4, 32x24576x1024 14.2 / 11.2, 9x28672x2048 15.2 / 11.9, 16x28672x1536 13.8 / 11.3); float32 tiles,
// at half the rate, from 17 rows on (16x24576x2048 14.9 / 16.8, 16x28672x1536 14.1 / 14.3, 24x24576x1024
// 13.5 / 11.4, 32x24576x1024 14.7 / 11.4).
inline bool fp8_few_rows(int m, int n, int k, bool whole, bool precise)
{
    const double work = (double)m * n * k;
    if (!whole) return m <= 4 || (m <= 48 && work <= 0x1.9p28);
    if (n > 22 << 10 && m > (precise ? 16 : 8)) return false;
    return m <= 8 || (m <= 32 && work <= 0x1.8p29) || (m <= 64 && n <= 8192 && k <= 4096 && (double)n * k <= 0x1p24);
}

// `whole`: the operands are whole 16-byte chunks as they are; `precise`: the result is binary32
inline Fp8Plan plan_fp8(int m, int n, int k, bool whole, bool precise)
{
    Fp8Plan p = {};
    if (m == 0 || n == 0 || fp8_few_rows(m, n, k, whole, precise)) {
        p.skinny = true;
        return p;
    }
    p.part_pitch = (n + 3) / 4 * 4;
    const int steps = scale_blocks(k);
    // The tile and the shares of k by the shortest estimate, in us: rounds of workgroups (one a
    // compute unit) times a share's steps, each as long as on large products, but no less than
    // the operands take from memory (w somewhat longer for each further row of tiles that reads
    // it, all of it with fewer workgroups than compute units); shares cost a second launch, and
    // their sums' way out and back.  (us of 64x128 / 64x256 / 128x128 / 128x256 / 256x256, n x k =
    // 28672x8192: 64 rows 49 / 57 / 51 / 58 / 67, 128 72 / 64 / 58 / 65 / 73, 256 125 / 103 / 90 /
    // 75 / 88, 1024 412 / 330 / 299 / 252 / 219; 93 rows of 14336x4096 19 / 28 / 22 / 24 / 27.)
    struct Shape { int fp, qg; double step, precise; };
    constexpr Shape shapes[] = {{2, 2, 0.46, 0.78}, {2, 4, 0.70, 1.20}, {4, 2, 0.64, 1.15}, {4, 4, 0.95, 1.75}, {8, 4, 1.65, 0}};
    double best = 0;
    for (const Shape& c : shapes) {
        if (precise && c.precise == 0) continue;
        const int64_t down = ((int64_t)m + 32 * c.fp - 1) / (32 * c.fp), tiles = down * (((int64_t)n + 64 * c.qg - 1) / (64 * c.qg));
        const double memory = (m + n * (0.85 + 0.15 * down)) * k / 5e6;
        int64_t most = kComputeUnits / tiles;
        if (most > steps / 4) most = steps / 4;
        for (int s = 1; s == 1 || s <= most; ++s) {
            const int share = steps > 0 ? (steps + s - 1) / s : 1, shares = steps > 0 ? (steps + share - 1) / share : 1;
            const int64_t groups = tiles * shares;
            double t = (double)((groups + kComputeUnits - 1) / kComputeUnits) * (share + 2) * (precise ? c.precise : c.step);
            const double least = groups < kComputeUnits ? memory * kComputeUnits / groups : memory;
            if (t < least) t = least + 0.1 * t;
            if (shares > 1) t += 3.0 + 8.0 * shares * m * p.part_pitch / 8e6;
            if (p.fp == 0 || t < best) best = t, p.fp = c.fp, p.qg = c.qg, p.shares = shares, p.share_steps = share;
        }
    }
    if (p.shares > 1) p.part_bytes = round256((size_t)p.shares * m * p.part_pitch * 4);
    const size_t row = (size_t)chunk_pitch(k, 1);
    p.a_bytes = round256((size_t)m * row);
    p.w_bytes = round256((size_t)n * row);
    return p;
}

// For either kind of result; without `whole`, for any operands: where the kernel for few rows takes
// those that are not whole chunks, others may go to the tiles, with shares of k (40x512x8192).
inline size_t fp8_workspace_bytes(int M, int N, int K, bool whole)
{
    size_t most = 0;
    for (int precise = 0; precise < 2; ++precise) {
        Fp8Plan p = plan_fp8(M, N, K, whole, precise != 0);
        if (!whole && p.skinny) p = plan_fp8(M, N, K, true, precise != 0), p.a_bytes = p.w_bytes = 0;
        const size_t need = p.part_bytes + (whole ? 0 : p.a_bytes + p.w_bytes);
        most = need > most ? need : most;
    }
    return most;
}

// size: bytes of an element; float32 needs no less than 16 bits do
size_t norm_grad_workspace_bytes(int64_t rows, int cols, size_t size);
size_t distill_workspace_bytes(int64_t rows, int vocab);

qtcq_status launch_quantize_blocks(const void* x, int dtype, int64_t rows, int cols, int64_t ldx, int block_rows, uint8_t* q,
                                   int64_t ldq, float* scale, int64_t scale_row, int64_t scale_col, hipStream_t st);
// checks the workspace against what the call's pointers and strides need
qtcq_status launch_matmul_fp8(const Fp8Args& a, int dtype, void* ws, size_t wsb, hipStream_t st);
qtcq_status launch_layer_norm(const NormArgs& a, int dtype, int weight_dtype, hipStream_t st);
qtcq_status launch_layer_norm_vjp(const NormGradArgs& a, int dtype, int weight_dtype, void* grad_weight, void* grad_bias,
                                  void* ws, hipStream_t st);
qtcq_status launch_distill(DistillArgs a, int dtype, void* ws, hipStream_t st);
qtcq_status launch_distill_grad(DistillArgs a, int dtype, hipStream_t st);

}  // namespace host
}  // namespace qtcq
