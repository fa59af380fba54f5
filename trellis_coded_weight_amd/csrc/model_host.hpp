// model_host.hpp -- host-side declarations of the model operators (8-bit floating point with
// block scales, layer norm, distillation), shared by their C ABI (qtcq_model.hip) and their
// launch units (launch_blocks.hip, launch_fp8.hip, launch_norm.hip, launch_distill.hip).
#pragma once

#include "dense_host.hpp"

namespace qtcq {

struct Fp8Args;
struct NormArgs;
struct NormGradArgs;
struct DistillArgs;

namespace host {

// row strides of the scales a product takes, in elements: 256 rows of them stay within 31
// bits of bytes
constexpr int64_t kScaleMaxStride = (int64_t)1 << 20;
// K of the e4m3 product: rows of 4 MB, so that a tile's offsets stay below 2^31
constexpr int kFp8MaxK = 1 << 22;

inline int scale_blocks(int n) { return n / 128 + (n % 128 != 0); }

size_t fp8_workspace_bytes(int M, int N, int K, bool whole);
size_t norm_grad_workspace_bytes(int64_t rows, int cols);
size_t distill_workspace_bytes(int64_t rows, int vocab);

qtcq_status launch_quantize_blocks(const void* x, int dtype, int64_t rows, int cols, int64_t ldx, int block_rows, uint8_t* q,
                                   int64_t ldq, float* scale, int64_t scale_row, int64_t scale_col, hipStream_t st);
// checks the workspace against what the call's pointers and strides need
qtcq_status launch_matmul_fp8(Fp8Args a, int dtype, void* ws, size_t wsb, hipStream_t st);
qtcq_status launch_layer_norm(const NormArgs& a, int dtype, int weight_dtype, hipStream_t st);
qtcq_status launch_layer_norm_vjp(const NormGradArgs& a, int dtype, int weight_dtype, void* grad_weight, void* grad_bias,
                                  void* ws, hipStream_t st);
qtcq_status launch_distill(DistillArgs a, int dtype, void* ws, hipStream_t st);
qtcq_status launch_distill_grad(DistillArgs a, int dtype, hipStream_t st);

}  // namespace host
}  // namespace qtcq
