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

// `whole`: the operands are whole 16-byte chunks as they are; `precise`: the result is binary32
inline Fp8Plan plan_fp8(int m, int n, int k, bool whole, bool precise)
{
    Fp8Plan p = {};
    const double work = (double)m * n * k;
    if (whole ? m <= 4 || (m <= 64 && work <= 0x1p31) : m <= 2 || (m <= 64 && work <= 0x1.1p30)) {
        p.skinny = true;
        return p;
    }
    p.part_pitch = (n + 3) / 4 * 4;
    const int steps = scale_blocks(k);
    double best = 0;
    for (int c = 0; c < (precise ? 4 : 5); ++c) {
        const int fp = c < 2 ? 2 : (c < 4 ? 4 : 8), qg = c < 4 && c % 2 == 0 ? 2 : 4;
        const int64_t tiles = ((int64_t)m + 32 * fp - 1) / (32 * fp) * (((int64_t)n + 64 * qg - 1) / (64 * qg));
        const double step = precise ? (fp == 2 ? 1.1 : 1.8) : (fp == 2 ? 0.7 : (fp == 4 ? 1.0 : 1.7));
        int64_t most = kComputeUnits / tiles;
        if (most > steps / 4) most = steps / 4;
        for (int s = 1; s == 1 || s <= most; ++s) {
            const int share = steps > 0 ? (steps + s - 1) / s : 1, shares = steps > 0 ? (steps + share - 1) / share : 1;
            double t = (double)((tiles * shares + kComputeUnits - 1) / kComputeUnits) * (share + 2) * step;
            if (shares > 1) t += 6.0 + 8.0 * shares * m * p.part_pitch / 4e6;
            if (p.fp == 0 || t < best) best = t, p.fp = fp, p.qg = qg, p.shares = shares, p.share_steps = share;
        }
    }
    if (p.shares > 1) p.part_bytes = round256((size_t)p.shares * m * p.part_pitch * 4);
    const size_t row = (size_t)chunk_pitch(k, 1);
    p.a_bytes = round256((size_t)m * row);
    p.w_bytes = round256((size_t)n * row);
    return p;
}

// for either kind of result
inline size_t fp8_workspace_bytes(int M, int N, int K, bool whole)
{
    size_t most = 0;
    for (int precise = 0; precise < 2; ++precise) {
        const Fp8Plan p = plan_fp8(M, N, K, whole, precise != 0);
        const size_t need = p.part_bytes + (whole ? 0 : p.a_bytes + p.w_bytes);
        most = need > most ? need : most;
    }
    return most;
}

size_t norm_grad_workspace_bytes(int64_t rows, int cols);
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
