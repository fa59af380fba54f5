// launch_blocks.hip -- launches of the e4m3 quantization (block_quantize.hpp).
#include "model_host.hpp"
#include "block_quantize.hpp"

namespace qtcq {
namespace host {
namespace {

template <typename T>
qtcq_status blocks_impl(const void* x, int64_t rows, int cols, int64_t ldx, int block_rows, uint8_t* q, int64_t ldq,
                        float* scale, int64_t scale_row, int64_t scale_col, hipStream_t st)
{
    // at most 2^22 workgroups a launch, which then take several pieces each
    constexpr int64_t most = (int64_t)1 << 22;
    const int per = block_rows == 1 ? BlockQuantShape::kRows : 128;
    const int wide = block_rows == 1 ? BlockQuantShape::kCols : 128;
    const int64_t groups = (rows + per - 1) / per * ((cols + wide - 1) / wide);
    const dim3 grid((unsigned)(groups < most ? groups : most)), block(BlockQuantShape::kThreads);
    if (block_rows == 1)
        hipLaunchKernelGGL(quantize_row_blocks<T>, grid, block, 0, st, static_cast<const T*>(x), rows, cols, ldx, q, ldq,
                           scale, scale_row, scale_col, (unsigned)groups);
    else
        hipLaunchKernelGGL(quantize_square_blocks<T>, grid, block, 0, st, static_cast<const T*>(x), rows, cols, ldx, q, ldq,
                           scale, scale_row, scale_col, (unsigned)groups);
    return launch_status();
}

}  // namespace

qtcq_status launch_quantize_blocks(const void* x, int dtype, int64_t rows, int cols, int64_t ldx, int block_rows, uint8_t* q,
                                   int64_t ldq, float* scale, int64_t scale_row, int64_t scale_col, hipStream_t st)
{
    switch (dtype) {
    case QTCQ_BF16: return blocks_impl<__bf16>(x, rows, cols, ldx, block_rows, q, ldq, scale, scale_row, scale_col, st);
    case QTCQ_F16: return blocks_impl<_Float16>(x, rows, cols, ldx, block_rows, q, ldq, scale, scale_row, scale_col, st);
    default: return blocks_impl<float>(x, rows, cols, ldx, block_rows, q, ldq, scale, scale_row, scale_col, st);
    }
}

}  // namespace host
}  // namespace qtcq
