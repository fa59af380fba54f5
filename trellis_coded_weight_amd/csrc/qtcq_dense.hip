// qtcq_dense.hip -- the C ABI of the dense operators (include/qtcq.h, "Dense operators
// around the codec"): argument validation; accepted calls go to launch_rows.hip,
// launch_int8.hip, launch_gated.hip and launch_gated_vjp.hip.
#include "dense_host.hpp"

namespace host = qtcq::host;
using namespace qtcq::host;

namespace {

bool aligned_to(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool half_type(int dtype) { return dtype == QTCQ_BF16 || dtype == QTCQ_F16; }
bool float_type(int dtype) { return dtype == QTCQ_F32 || half_type(dtype); }
size_t type_size(int dtype) { return dtype == QTCQ_F32 ? 4 : dtype == QTCQ_I8 ? 1 : 2; }

// an operand or result of `rows` rows and `cols` columns: there, and aligned to its
// element; one without elements may be NULL
bool there(const void* p, int64_t rows, int64_t cols, size_t size)
{
    return rows == 0 || cols == 0 || (p != nullptr && aligned_to(p, size));
}

bool tiles_ok(int64_t rows, int64_t cols)
{
    return ((rows + 127) / 128) * ((cols + 63) / 64) <= kDenseMaxTiles;
}

bool gated_sizes_ok(int M, int F, int K)
{
    return M >= 0 && F >= 0 && K >= 0 && M <= kDenseMaxDim && F <= kHalfMaxRow && K <= kHalfMaxRow && tiles_ok(M, F);
}

bool vjp_sizes_ok(int M, int F, int K)
{
    // the elementwise kernel's grid: one thread per 8 of M slope_pitch(F) elements
    return gated_sizes_ok(M, F, K) && (int64_t)M * slope_pitch(F) <= (int64_t)1 << 34 && tiles_ok(M, K) && tiles_ok(F, K);
}

}  // namespace

extern "C" {

qtcq_status qtcq_quantize_rows(const void* x, int dtype, int64_t rows, int cols, int64_t ldx, int8_t* q, int64_t ldq,
                               float* scale, void* stream)
{
    if (rows < 0 || cols < 0 || ldx < cols || ldq < cols) return QTCQ_ERR_INVALID_ARG;
    if (!float_type(dtype) || rows > kDenseMaxDim || cols > kDenseMaxDim) return QTCQ_ERR_UNSUPPORTED;
    if (rows == 0) return QTCQ_OK;
    if (!scale || !aligned_to(scale, 4) || !there(x, rows, cols, type_size(dtype)) || !there(q, rows, cols, 1))
        return QTCQ_ERR_INVALID_ARG;
    return host::launch_quantize_rows(x, dtype, rows, cols, ldx, q, ldq, scale, as_stream(stream));
}

qtcq_status qtcq_decode_matrix(const uint32_t* bits, int M, int N, int L, int k, qtcq_code code, int tailbiting,
                               int dtype, void* w, int64_t ldw, float* scale, void* stream)
{
    if (M < 0 || N < 0 || (M % 16) != 0 || (N % 16) != 0 || ldw < N) return QTCQ_ERR_INVALID_ARG;
    if (!supported_trellis(L, k)) return QTCQ_ERR_UNSUPPORTED;
    CodeSel cs;
    if (const qtcq_status pc = parse_code(code, L, &cs); pc != QTCQ_OK) return pc;
    if ((!float_type(dtype) && dtype != QTCQ_I8) || M > kDenseMaxDim || N > kDenseMaxDim) return QTCQ_ERR_UNSUPPORTED;
    if ((ldw * (int64_t)type_size(dtype)) % 16 != 0) return QTCQ_ERR_INVALID_ARG;
    if (M == 0) return QTCQ_OK;
    if (!there(bits, M, N, 4) || !there(w, M, N, 16)) return QTCQ_ERR_INVALID_ARG;
    if (dtype == QTCQ_I8 && (!scale || !aligned_to(scale, 4))) return QTCQ_ERR_INVALID_ARG;
    if (N == 0 && dtype != QTCQ_I8) return QTCQ_OK;
    return host::launch_decode_matrix(L, cs, tailbiting != 0, bits, M, N, dtype, w, ldw, scale, as_stream(stream));
}

size_t qtcq_matmul_int8_workspace_bytes(int M, int N, int K, int whole_rows)
{
    if (M < 0 || N < 0 || K < 0 || M > kDenseMaxDim || N > kDenseMaxDim || K > kInt8MaxK || !tiles_ok(M, N)) return 0;
    return rows_product_bytes(kPlanInt8, 1, M, N, K, whole_rows != 0);
}

qtcq_status qtcq_matmul_int8(const int8_t* a, int64_t lda, const float* a_scale, const int8_t* w, int64_t ldw,
                             const float* w_scale, int M, int N, int K, int dtype, void* y, int64_t ldy, void* workspace,
                             size_t workspace_bytes, void* stream)
{
    if (M < 0 || N < 0 || K < 0 || lda < K || ldw < K || ldy < N) return QTCQ_ERR_INVALID_ARG;
    if (!float_type(dtype) || M > kDenseMaxDim || N > kDenseMaxDim || K > kInt8MaxK || !tiles_ok(M, N))
        return QTCQ_ERR_UNSUPPORTED;
    if (M == 0 || N == 0) return QTCQ_OK;
    if (!there(a, M, K, 1) || !there(w, N, K, 1) || !there(a_scale, M, 1, 4) || !there(w_scale, N, 1, 4) ||
        !there(y, M, N, type_size(dtype)))
        return QTCQ_ERR_INVALID_ARG;
    return host::launch_matmul_int8(a, lda, a_scale, w, ldw, w_scale, M, N, K, dtype, y, ldy, workspace, workspace_bytes,
                                    as_stream(stream));
}

size_t qtcq_gated_workspace_bytes(int M, int F, int K, int whole_rows)
{
    if (!gated_sizes_ok(M, F, K)) return 0;
    return rows_product_bytes(kPlanGated, 2, M, F, K, whole_rows != 0);
}

qtcq_status qtcq_gated_forward(const void* x, int64_t ldx, const void* w_gate, const void* w_up, int64_t ldw, int dtype,
                               int M, int F, int K, int activation, void* h, int64_t ldh, void* gate, void* up,
                               int64_t ldg, void* workspace, size_t workspace_bytes, void* stream)
{
    if (M < 0 || F < 0 || K < 0 || ldx < K || ldw < K || ldh < F) return QTCQ_ERR_INVALID_ARG;
    if ((gate == nullptr) != (up == nullptr) || (gate && ldg < F)) return QTCQ_ERR_INVALID_ARG;
    if (!half_type(dtype) || activation < QTCQ_ACT_SILU || activation > QTCQ_ACT_SIGMOID) return QTCQ_ERR_UNSUPPORTED;
    if (!gated_sizes_ok(M, F, K)) return QTCQ_ERR_UNSUPPORTED;
    if (M == 0 || F == 0) return QTCQ_OK;
    if (!there(x, M, K, 2) || !there(w_gate, F, K, 2) || !there(w_up, F, K, 2) || !there(h, M, F, 2) ||
        !aligned_to(gate, 2) || !aligned_to(up, 2))
        return QTCQ_ERR_INVALID_ARG;
    const GatedCall c = {x, w_gate, w_up, ldx, ldw, dtype, M, F, K, activation, h, ldh, gate, up, ldg};
    return host::launch_gated_forward(c, workspace, workspace_bytes, as_stream(stream));
}

size_t qtcq_gated_vjp_workspace_bytes(int M, int F, int K, int whole_rows)
{
    if (!vjp_sizes_ok(M, F, K)) return 0;
    return plan_vjp(M, F, K, 2).bytes(whole_rows != 0, whole_rows != 0, true, true);
}

qtcq_status qtcq_gated_vjp(const void* x, int64_t ldx, const void* w_gate, const void* w_up, int64_t ldw,
                           const void* gate, const void* up, int64_t ldg, const void* grad_h, int64_t ldgh, int dtype,
                           int M, int F, int K, int activation, void* grad_x, int64_t ldgx, void* grad_w_gate,
                           void* grad_w_up, int64_t ldgw, void* workspace, size_t workspace_bytes, void* stream)
{
    if (M < 0 || F < 0 || K < 0 || ldg < F || ldgh < F) return QTCQ_ERR_INVALID_ARG;
    if ((grad_w_gate == nullptr) != (grad_w_up == nullptr)) return QTCQ_ERR_INVALID_ARG;
    if (grad_x && (ldw < K || ldgx < K)) return QTCQ_ERR_INVALID_ARG;
    if (grad_w_gate && (ldx < K || ldgw < K)) return QTCQ_ERR_INVALID_ARG;
    const int pieces = activation >= 0 && (activation & QTCQ_ACT_ROUND_SLOPES) ? 1 : 2;
    if (pieces == 1) activation &= ~QTCQ_ACT_ROUND_SLOPES;
    if (!half_type(dtype) || activation < QTCQ_ACT_SILU || activation > QTCQ_ACT_SIGMOID) return QTCQ_ERR_UNSUPPORTED;
    if (!vjp_sizes_ok(M, F, K)) return QTCQ_ERR_UNSUPPORTED;
    // what is left to write: grad_x [M][K], the weight gradients [F][K]
    const bool want_x = grad_x && M > 0 && K > 0, want_w = grad_w_gate && F > 0 && K > 0;
    if (!want_x && !want_w) return QTCQ_OK;
    if (!there(gate, M, F, 2) || !there(up, M, F, 2) || !there(grad_h, M, F, 2)) return QTCQ_ERR_INVALID_ARG;
    if (want_x && (!aligned_to(grad_x, 2) || !there(w_gate, F, K, 2) || !there(w_up, F, K, 2)))
        return QTCQ_ERR_INVALID_ARG;
    if (want_w && (!aligned_to(grad_w_gate, 2) || !aligned_to(grad_w_up, 2) || !there(x, M, K, 2)))
        return QTCQ_ERR_INVALID_ARG;
    const GatedVjpCall c = {x, w_gate, w_up, gate, up, grad_h, ldx, ldw, ldg, ldgh, dtype, M, F, K, activation, pieces,
                            want_x ? grad_x : nullptr, want_w ? grad_w_gate : nullptr, want_w ? grad_w_up : nullptr,
                            ldgx, ldgw};
    return host::launch_gated_vjp(c, workspace, workspace_bytes, as_stream(stream));
}

}  // extern "C"
