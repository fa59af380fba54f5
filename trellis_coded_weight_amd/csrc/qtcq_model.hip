// qtcq_model.hip -- the C ABI of the model operators (include/qtcq.h, "Model operators on coded
// weights"): argument validation; accepted calls go to launch_blocks.hip, launch_fp8.hip,
// launch_norm.hip and launch_distill.hip.
#include "model_host.hpp"

namespace host = qtcq::host;
using namespace qtcq::host;

namespace {

bool aligned_to(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool float_type(int dtype) { return dtype == QTCQ_F32 || dtype == QTCQ_BF16 || dtype == QTCQ_F16; }
size_t type_size(int dtype) { return dtype == QTCQ_F32 ? 4 : 2; }

// an operand or result of `rows` rows and `cols` columns: there, and aligned to its
// element; one without elements may be NULL
bool there(const void* p, int64_t rows, int64_t cols, size_t size)
{
    return rows == 0 || cols == 0 || (p != nullptr && aligned_to(p, size));
}

bool optional(const void* p, size_t size) { return p == nullptr || aligned_to(p, size); }

// strides of written scales [r][c]: no two at one place
bool distinct(int64_t r, int64_t c, int64_t row, int64_t col)
{
    return (r <= 1 && c <= 1) || (col >= 1 && (r <= 1 || row / col >= c)) || (row >= 1 && (c <= 1 || col / row >= r));
}

// strides of read scales
bool readable(int64_t row, int64_t col) { return row >= 0 && col >= 0; }

bool workspace_ok(const void* ws, size_t wsb, size_t need) { return need == 0 || (ws && aligned16(ws) && wsb >= need); }

bool fp8_sizes_ok(int M, int N, int K)
{
    return M >= 0 && N >= 0 && K >= 0 && M <= kDenseMaxDim && N <= kDenseMaxDim && K <= kFp8MaxK &&
           ((int64_t)M + 127) / 128 * (((int64_t)N + 63) / 64) <= kDenseMaxTiles;
}

// a temperature whose reciprocal is a normal number too
bool temperature_ok(float t) { return t >= 0x1p-100f && t <= 0x1p100f; }

bool weight_type_ok(int dtype, int weight_dtype) { return weight_dtype == QTCQ_F32 || weight_dtype == dtype; }

// what both directions of the distillation share
qtcq_status distill_args(const void* logits, int dtype, int64_t rows, int vocab, int64_t ldl, const void* index,
                         int index_bytes, int64_t ldi, const void* teacher, int teacher_dtype, int64_t ldt, int k,
                         float temperature)
{
    if (rows < 0 || vocab < 0 || k < 0 || ldl < vocab || ldi < k || ldt < k || !(temperature > 0.0f))
        return QTCQ_ERR_INVALID_ARG;
    if (!float_type(dtype) || !float_type(teacher_dtype) || (index_bytes != 4 && index_bytes != 8) || rows > kDenseMaxDim ||
        vocab > kDenseMaxDim || k > qtcq::kDistillMaxK || !temperature_ok(temperature))
        return QTCQ_ERR_UNSUPPORTED;
    if (!there(logits, rows, vocab, type_size(dtype)) || !there(index, rows, k, index_bytes) ||
        !there(teacher, rows, k, type_size(teacher_dtype)))
        return QTCQ_ERR_INVALID_ARG;
    return QTCQ_OK;
}

}  // namespace

extern "C" {

qtcq_status qtcq_quantize_blocks(const void* x, int dtype, int64_t rows, int cols, int64_t ldx, int block_rows, uint8_t* q,
                                 int64_t ldq, float* scale, int64_t scale_row, int64_t scale_col, void* stream)
{
    if (rows < 0 || cols < 0 || ldx < cols || ldq < cols) return QTCQ_ERR_INVALID_ARG;
    if (!float_type(dtype) || (block_rows != 1 && block_rows != 128) || rows > kDenseMaxDim || cols > kDenseMaxDim ||
        rows * cols > kBlocksMaxElements)
        return QTCQ_ERR_UNSUPPORTED;
    const int64_t r = block_rows == 1 ? rows : scale_blocks((int)rows), c = scale_blocks(cols);
    if (!distinct(r, c, scale_row, scale_col)) return QTCQ_ERR_INVALID_ARG;
    if (rows == 0 || cols == 0) return QTCQ_OK;
    if (!there(scale, r, c, 4) || !there(x, rows, cols, type_size(dtype)) || !there(q, rows, cols, 1))
        return QTCQ_ERR_INVALID_ARG;
    return host::launch_quantize_blocks(x, dtype, rows, cols, ldx, block_rows, q, ldq, scale, scale_row, scale_col,
                                        as_stream(stream));
}

size_t qtcq_matmul_fp8_workspace_bytes(int M, int N, int K, int whole_rows)
{
    return fp8_sizes_ok(M, N, K) ? host::fp8_workspace_bytes(M, N, K, whole_rows != 0) : 0;
}

qtcq_status qtcq_matmul_fp8(const uint8_t* a, int64_t lda, const float* a_scale, int64_t as_row, int64_t as_col,
                            const uint8_t* w, int64_t ldw, const float* w_scale, int64_t ws_row, int64_t ws_col, int M, int N,
                            int K, int dtype, void* y, int64_t ldy, void* workspace, size_t workspace_bytes, void* stream)
{
    if (M < 0 || N < 0 || K < 0 || lda < K || ldw < K || ldy < N || !readable(as_row, as_col) || !readable(ws_row, ws_col))
        return QTCQ_ERR_INVALID_ARG;
    if (!float_type(dtype) || !fp8_sizes_ok(M, N, K) || as_row > kScaleMaxStride ||
        ws_row > kScaleMaxStride)
        return QTCQ_ERR_UNSUPPORTED;
    if (M == 0 || N == 0) return QTCQ_OK;
    if (!there(a, M, K, 1) || !there(w, N, K, 1) || !there(a_scale, M, K, 4) || !there(w_scale, N, K, 4) ||
        !there(y, M, N, type_size(dtype)))
        return QTCQ_ERR_INVALID_ARG;
    qtcq::Fp8Args p = {};
    p.a = a;
    p.w = w;
    p.lda = lda;
    p.ldw = ldw;
    p.a_scale = a_scale;
    p.w_scale = w_scale;
    p.as_row = as_row;
    p.as_col = as_col;
    p.ws_row = ws_row;
    p.ws_col = ws_col;
    p.m = M;
    p.n = N;
    p.k = K;
    p.y = y;
    p.ldy = ldy;
    return host::launch_matmul_fp8(p, dtype, workspace, workspace_bytes, as_stream(stream));
}

qtcq_status qtcq_layer_norm(const void* x, int dtype, int64_t rows, int cols, int64_t ldx, const void* weight,
                            const void* bias, int weight_dtype, float eps, void* y, int64_t ldy, float* mean, float* rstd,
                            void* stream)
{
    if (rows < 0 || cols < 0 || ldx < cols || ldy < cols || (mean == nullptr) != (rstd == nullptr) || !(eps >= 0.0f))
        return QTCQ_ERR_INVALID_ARG;
    if (!float_type(dtype) || !weight_type_ok(dtype, weight_dtype) || rows > kDenseMaxDim || cols > kDenseMaxDim)
        return QTCQ_ERR_UNSUPPORTED;
    if (rows == 0 || cols == 0) return QTCQ_OK;
    const size_t w = type_size(weight_dtype);
    if (!there(x, rows, cols, type_size(dtype)) || !there(y, rows, cols, type_size(dtype)) || !optional(weight, w) ||
        !optional(bias, w) || !optional(mean, 4) || !optional(rstd, 4))
        return QTCQ_ERR_INVALID_ARG;
    const qtcq::NormArgs a = {x, rows, ldx, cols, weight, bias, eps, y, ldy, mean, rstd};
    return host::launch_layer_norm(a, dtype, weight_dtype, as_stream(stream));
}

size_t qtcq_layer_norm_vjp_workspace_bytes(int64_t rows, int cols)
{
    if (rows < 0 || cols < 0 || rows > kDenseMaxDim || cols > kDenseMaxDim) return 0;
    return host::norm_grad_workspace_bytes(rows, cols, 4);
}

qtcq_status qtcq_layer_norm_vjp(const void* x, int dtype, int64_t rows, int cols, int64_t ldx, const void* weight,
                                int weight_dtype, const float* mean, const float* rstd, const void* grad_y, int64_t ldgy,
                                void* grad_x, int64_t ldgx, void* grad_weight, void* grad_bias, void* workspace,
                                size_t workspace_bytes, void* stream)
{
    if (rows < 0 || cols < 0 || ldx < cols || ldgy < cols || (grad_x && ldgx < cols)) return QTCQ_ERR_INVALID_ARG;
    if (!float_type(dtype) || !weight_type_ok(dtype, weight_dtype) || rows > kDenseMaxDim || cols > kDenseMaxDim)
        return QTCQ_ERR_UNSUPPORTED;
    const bool want_x = grad_x && rows > 0, want_w = grad_weight || grad_bias;
    if (cols == 0 || (!want_x && !want_w)) return QTCQ_OK;
    const size_t t = type_size(dtype), w = type_size(weight_dtype);
    if (!there(x, rows, cols, t) || !there(grad_y, rows, cols, t) || !there(mean, rows, 1, 4) || !there(rstd, rows, 1, 4) ||
        !optional(grad_x, t) || !optional(weight, w) || !optional(grad_weight, w) || !optional(grad_bias, w))
        return QTCQ_ERR_INVALID_ARG;
    if (want_w && !workspace_ok(workspace, workspace_bytes, host::norm_grad_workspace_bytes(rows, cols, t)))
        return QTCQ_ERR_WORKSPACE;
    qtcq::NormGradArgs a = {};
    a.x = x;
    a.grad_y = grad_y;
    a.rows = rows;
    a.ldx = ldx;
    a.ldgy = ldgy;
    a.cols = cols;
    a.weight = weight;
    a.mean = mean;
    a.rstd = rstd;
    a.grad_x = want_x ? grad_x : nullptr;
    a.ldgx = ldgx;
    return host::launch_layer_norm_vjp(a, dtype, weight_dtype, grad_weight, grad_bias, workspace, as_stream(stream));
}

size_t qtcq_distill_topk_workspace_bytes(int64_t rows, int vocab)
{
    if (rows < 0 || vocab < 0 || rows > kDenseMaxDim || vocab > kDenseMaxDim) return 0;
    return host::distill_workspace_bytes(rows, vocab);
}

qtcq_status qtcq_distill_topk(const void* logits, int dtype, int64_t rows, int vocab, int64_t ldl, const void* index,
                              int index_bytes, int64_t ldi, const void* teacher, int teacher_dtype, int64_t ldt, int k,
                              float temperature, const float* teacher_log_z, float* loss, float* stats,
                              const float* grad_loss, void* grad_logits, int64_t ldg, void* workspace,
                              size_t workspace_bytes, void* stream)
{
    const qtcq_status s = distill_args(logits, dtype, rows, vocab, ldl, index, index_bytes, ldi, teacher, teacher_dtype, ldt,
                                       k, temperature);
    if (s != QTCQ_OK) return s;
    if (grad_logits && ldg < vocab) return QTCQ_ERR_INVALID_ARG;
    if (rows == 0) return QTCQ_OK;
    if (!loss || !aligned_to(loss, 4) || !optional(teacher_log_z, 4) || !optional(stats, 4) ||
        !optional(grad_logits, type_size(dtype)) || (grad_logits && (!grad_loss || !aligned_to(grad_loss, 4))))
        return QTCQ_ERR_INVALID_ARG;
    if (!workspace_ok(workspace, workspace_bytes, host::distill_workspace_bytes(rows, vocab))) return QTCQ_ERR_WORKSPACE;
    const qtcq::DistillArgs a = {logits, rows, ldl, vocab, index, ldi, index_bytes == 8, teacher, ldt, teacher_dtype, k,
                                 temperature, teacher_log_z, loss, stats, grad_loss, grad_logits, ldg, nullptr, 1, vocab};
    return host::launch_distill(a, dtype, workspace, as_stream(stream));
}

qtcq_status qtcq_distill_topk_vjp(const void* logits, int dtype, int64_t rows, int vocab, int64_t ldl, const void* index,
                                  int index_bytes, int64_t ldi, const void* teacher, int teacher_dtype, int64_t ldt, int k,
                                  float temperature, const float* stats, const float* grad_loss, void* grad_logits,
                                  int64_t ldg, void* stream)
{
    const qtcq_status s = distill_args(logits, dtype, rows, vocab, ldl, index, index_bytes, ldi, teacher, teacher_dtype, ldt,
                                       k, temperature);
    if (s != QTCQ_OK) return s;
    if (ldg < vocab) return QTCQ_ERR_INVALID_ARG;
    if (rows == 0 || vocab == 0) return QTCQ_OK;
    if (!there(stats, rows, 1, 4) || !there(grad_loss, rows, 1, 4) || !there(grad_logits, rows, vocab, type_size(dtype)))
        return QTCQ_ERR_INVALID_ARG;
    qtcq::DistillArgs a = {logits, rows, ldl, vocab, index, ldi, index_bytes == 8, teacher, ldt, teacher_dtype, k,
                           temperature, nullptr, nullptr, const_cast<float*>(stats), grad_loss, grad_logits, ldg, nullptr, 1,
                           vocab};
    return host::launch_distill_grad(a, dtype, as_stream(stream));
}

}  // extern "C"
