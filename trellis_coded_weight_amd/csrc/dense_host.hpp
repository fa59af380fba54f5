// dense_host.hpp -- host-side declarations of the dense operators, shared by their C ABI
// (qtcq_dense.hip) and their launch units (launch_rows.hip, launch_products.hip).
#pragma once

#include "host.hpp"

namespace qtcq {
namespace host {

// Lengths a call may have: tile counts, row offsets inside a tile and element indices
// inside a row stay within 32 bits.
constexpr int kDenseMaxDim = 1 << 24;
// 2^14 K, the largest magnitude of a sum of K products of 8-bit integers, below 2^31
constexpr int kInt8MaxK = 131071;
// the largest grid of 128-wide tiles of 256 threads a launch can hold
constexpr int64_t kDenseMaxTiles = (int64_t)1 << 23;

// row stride of the two slope matrices of the gated gradient, in elements: whole steps
// of its products, zero-filled past F
inline int slope_pitch(int F) { return (F + 63) / 64 * 64; }
inline size_t gated_vjp_bytes(int M, int F)
{
    return ((size_t)2 * 2 * (size_t)M * (size_t)slope_pitch(F) + 255) / 256 * 256;
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
    void *grad_x, *grad_w_gate, *grad_w_up;
    int64_t ldgx, ldgw;
};

qtcq_status launch_quantize_rows(const void* x, int dtype, int64_t rows, int cols, int64_t ldx, int8_t* q, int64_t ldq,
                                 float* scale, hipStream_t st);
qtcq_status launch_decode_matrix(int L, const CodeSel& code, bool tb, const uint32_t* bits, int M, int N, int dtype,
                                 void* w, int64_t ldw, float* scale, hipStream_t st);
qtcq_status launch_matmul_int8(const int8_t* a, int64_t lda, const float* a_scale, const int8_t* w, int64_t ldw,
                               const float* w_scale, int M, int N, int K, int dtype, void* y, int64_t ldy,
                               hipStream_t st);
qtcq_status launch_gated_forward(const GatedCall& c, hipStream_t st);
qtcq_status launch_gated_vjp(const GatedVjpCall& c, void* ws, hipStream_t st);

}  // namespace host
}  // namespace qtcq
