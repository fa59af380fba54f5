// model_args.hpp -- the arguments of the model operators' kernels, filled by their C ABI
// (qtcq_model.hip) and their launch units.
#pragma once

#include <stdint.h>

namespace qtcq {

// The product of e4m3 matrices with block scales (fp8_skinny.hpp, fp8_block.hpp).
// strides of the scales in elements
struct Fp8Args {
    const uint8_t* a;
    const uint8_t* w;
    int64_t lda, ldw;
    const float* a_scale;
    const float* w_scale;
    int64_t as_row, as_col, ws_row, ws_col;
    int m, n, k;
    int ak, wk;              // k of a and w with their zero padding
    void* y;
    int64_t ldy;
    float* part;             // the shares' sums [shares][m][part_pitch], or NULL
    int part_pitch;
    int shares, share_steps; // shares of k, and the blocks of each
};

// Layer norm and its gradients (norm.hpp).
struct NormArgs {
    const void* x;
    int64_t rows, ldx;
    int cols;
    const void* weight;      // [cols], or NULL: ones
    const void* bias;        // [cols], or NULL: zeros
    float eps;
    void* y;
    int64_t ldy;
    float* mean;             // [rows], or NULL
    float* rstd;
};

struct NormGradArgs {
    const void* x;
    const void* grad_y;
    int64_t rows, ldx, ldgy;
    int cols;
    const void* weight;
    const float* mean;
    const float* rstd;
    void* grad_x;            // or NULL
    int64_t ldgx;
    float* part;             // [row groups][2][part_pitch]: sums of dw, then of db
    int part_pitch;
};

// Distillation from top logits (distill.hpp).
constexpr int kDistillMaxK = 1024;
constexpr int kDistillStats = 5;

struct DistillArgs {
    const void* logits;
    int64_t rows, ldl;
    int vocab;
    const void* index;       // [rows][k] int32, or int64 where wide
    int64_t ldi;
    bool wide;
    const void* teacher;     // [rows][k]
    int64_t ldt;
    int teacher_type;        // qtcq_dtype: float32, bfloat16, float16
    int k;
    float tau;
    const float* teacher_log_z;  // [rows], or NULL: the sum over the entries
    float* loss;             // [rows]
    float* stats;            // [rows][kDistillStats], or NULL
    const float* grad_loss;  // [rows]
    void* grad;              // [rows][vocab], or NULL
    int64_t ldg;
    float* part;             // [rows][segments][2]: m and s of each segment
    int segments, segment;   // a row's segments and their length
};

}  // namespace qtcq
