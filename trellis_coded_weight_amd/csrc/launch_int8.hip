// launch_int8.hip -- launches of the 8-bit product.
#include "product_launch.hpp"

namespace qtcq {
namespace host {

qtcq_status launch_matmul_int8(const int8_t* a, int64_t lda, const float* a_scale, const int8_t* w, int64_t ldw,
                               const float* w_scale, int M, int N, int K, int dtype, void* y, int64_t ldy,
                               void* ws, size_t wsb, hipStream_t st)
{
    ProductArgs p = {};
    p.p[0] = a;
    p.q[0] = w;
    p.ldp = lda;
    p.ldq = ldw;
    p.out[0] = y;
    p.ldo = ldy;
    p.m = M;
    p.n = N;
    p.k = K;
    p.p_scale = a_scale;
    p.q_scale = w_scale;
    switch (dtype) {
    case QTCQ_BF16: return rows_product<int8_t, __bf16, kInt8>(p, ws, wsb, st);
    case QTCQ_F16: return rows_product<int8_t, _Float16, kInt8>(p, ws, wsb, st);
    default: return rows_product<int8_t, float, kInt8>(p, ws, wsb, st);
    }
}

}  // namespace host
}  // namespace qtcq
