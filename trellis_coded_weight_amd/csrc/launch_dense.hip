// launch_dense.hip -- launches of the dense operators: row quantization, decode to rows
// (quantize.hpp), the 8-bit product and the gated projections (tile_product.hpp).
#include "dense_host.hpp"
#include "quantize.hpp"
#include "tile_product.hpp"

namespace qtcq {
namespace host {
namespace {

template <typename T, int RT, int NCH>
void quantize_go(bool vec, const void* x, int64_t rows, int cols, int64_t ldx, int8_t* q, int64_t ldq, float* scale,
                 hipStream_t st)
{
    const dim3 grid(blocks_for(rows, QuantShape::kThreads / RT)), block(QuantShape::kThreads);
    if (vec)
        hipLaunchKernelGGL((quantize_rows<T, RT, NCH, true>), grid, block, 0, st, static_cast<const T*>(x), rows, cols,
                           ldx, q, ldq, scale);
    else
        hipLaunchKernelGGL((quantize_rows<T, RT, NCH, false>), grid, block, 0, st, static_cast<const T*>(x), rows, cols,
                           ldx, q, ldq, scale);
}

template <typename T>
qtcq_status quantize_impl(const void* x, int64_t rows, int cols, int64_t ldx, int8_t* q, int64_t ldq, float* scale,
                          hipStream_t st)
{
    constexpr int E = 16 / (int)sizeof(T);
    const bool vec = aligned16(x) && ldx % E == 0 && (reinterpret_cast<uintptr_t>(q) & 7u) == 0 && ldq % 8 == 0;
    const int chunks = (cols + E - 1) / E;
    if (chunks <= 64)
        quantize_go<T, 64, 1>(vec, x, rows, cols, ldx, q, ldq, scale, st);
    else if (chunks <= 256)
        quantize_go<T, 64, 4>(vec, x, rows, cols, ldx, q, ldq, scale, st);
    else if (chunks <= 1024)
        quantize_go<T, 256, 4>(vec, x, rows, cols, ldx, q, ldq, scale, st);
    else
        quantize_go<T, 256, 8>(vec, x, rows, cols, ldx, q, ldq, scale, st);
    return launch_status();
}

template <int L, int CODE, bool TB>
qtcq_status decode_rows_impl(const uint32_t* bits, int M, int N, int dtype, void* w, int64_t ldw, float* scale,
                             const CodeArg& ca, hipStream_t st)
{
    const dim3 grid((unsigned)(M / 16)), block(DecodeRowsShape::kThreads);
    auto go = [&](auto out) {
        hipLaunchKernelGGL((decode_rows<L, CODE, TB, decltype(out)::value>), grid, block, 0, st, bits, N / 16, w, ldw,
                           scale, ca);
        return launch_status();
    };
    switch (dtype) {
    case QTCQ_I8: return go(int_c<0>{});
    case QTCQ_BF16: return go(int_c<1>{});
    case QTCQ_F16: return go(int_c<2>{});
    default: return go(int_c<3>{});
    }
}

template <typename T, typename O, int MODE>
qtcq_status tiles_go(const ProductArgs& a, hipStream_t st)
{
    const int64_t tiles = (int64_t)blocks_for(a.m, TileShape::kRows) * blocks_for(a.n, TileShape::cols(MODE));
    const dim3 grid((unsigned)tiles, 1, MODE == kGradW ? 2 : 1), block(TileShape::kThreads);
    hipLaunchKernelGGL((tile_product<T, O, MODE>), grid, block, 0, st, a);
    return launch_status();
}

template <typename T>
qtcq_status slopes(int act, const GatedVjpCall& c, int ldd, T* dg, T* du, hipStream_t st)
{
    const dim3 grid(blocks_for((int64_t)c.M * (ldd / 8), 256)), block(256);
    auto go = [&](auto act_c) {
        hipLaunchKernelGGL((gated_slopes<T, decltype(act_c)::value>), grid, block, 0, st,
                           static_cast<const T*>(c.gate), static_cast<const T*>(c.up), c.ldg,
                           static_cast<const T*>(c.grad_h), c.ldgh, c.M, c.F, ldd, dg, du);
        return launch_status();
    };
    switch (act) {
    case kActSilu: return go(int_c<kActSilu>{});
    case kActGelu: return go(int_c<kActGelu>{});
    case kActGeluTanh: return go(int_c<kActGeluTanh>{});
    case kActRelu: return go(int_c<kActRelu>{});
    default: return go(int_c<kActSigmoid>{});
    }
}

template <typename T>
qtcq_status gated_vjp_impl(const GatedVjpCall& c, void* ws, hipStream_t st)
{
    const int ldd = slope_pitch(c.F);
    T* dg = static_cast<T*>(ws);
    T* du = dg + (int64_t)c.M * ldd;
    if (c.M > 0 && c.F > 0)
        if (const qtcq_status s = slopes<T>(c.act, c, ldd, dg, du, st); s != QTCQ_OK) return s;
    if (c.grad_x) {
        ProductArgs a = {};
        a.p[0] = dg;
        a.p[1] = du;
        a.q[0] = c.w_gate;
        a.q[1] = c.w_up;
        a.ldp = ldd;
        a.ldq = c.ldw;
        a.out[0] = c.grad_x;
        a.ldo = c.ldgx;
        a.m = c.M;
        a.n = c.K;
        a.k = c.F;
        if (const qtcq_status s = tiles_go<T, T, kGradX>(a, st); s != QTCQ_OK) return s;
    }
    if (c.grad_w_gate) {
        ProductArgs a = {};
        a.p[0] = dg;
        a.p[1] = du;
        a.q[0] = c.x;
        a.ldp = ldd;
        a.ldq = c.ldx;
        a.out[0] = c.grad_w_gate;
        a.out[1] = c.grad_w_up;
        a.ldo = c.ldgw;
        a.m = c.F;
        a.n = c.K;
        a.k = c.M;
        return tiles_go<T, T, kGradW>(a, st);
    }
    return QTCQ_OK;
}

}  // namespace

qtcq_status launch_quantize_rows(const void* x, int dtype, int64_t rows, int cols, int64_t ldx, int8_t* q, int64_t ldq,
                                 float* scale, hipStream_t st)
{
    switch (dtype) {
    case QTCQ_BF16: return quantize_impl<__bf16>(x, rows, cols, ldx, q, ldq, scale, st);
    case QTCQ_F16: return quantize_impl<_Float16>(x, rows, cols, ldx, q, ldq, scale, st);
    default: return quantize_impl<float>(x, rows, cols, ldx, q, ldq, scale, st);
    }
}

qtcq_status launch_decode_matrix(int L, const CodeSel& code, bool tb, const uint32_t* bits, int M, int N, int dtype,
                                 void* w, int64_t ldw, float* scale, hipStream_t st)
{
    return with_L_code(L, code.id, [&](auto l, auto c) {
        return with_bool(tb, [&](auto t) {
            return decode_rows_impl<decltype(l)::value, decltype(c)::value, decltype(t)::value>(
                bits, M, N, dtype, w, ldw, scale, code.arg, st);
        });
    });
}

qtcq_status launch_matmul_int8(const int8_t* a, int64_t lda, const float* a_scale, const int8_t* w, int64_t ldw,
                               const float* w_scale, int M, int N, int K, int dtype, void* y, int64_t ldy,
                               hipStream_t st)
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
    case QTCQ_BF16: return tiles_go<int8_t, __bf16, kInt8>(p, st);
    case QTCQ_F16: return tiles_go<int8_t, _Float16, kInt8>(p, st);
    default: return tiles_go<int8_t, float, kInt8>(p, st);
    }
}

qtcq_status launch_gated_forward(const GatedCall& c, hipStream_t st)
{
    ProductArgs p = {};
    p.p[0] = c.x;
    p.q[0] = c.w_gate;
    p.q[1] = c.w_up;
    p.ldp = c.ldx;
    p.ldq = c.ldw;
    p.out[0] = c.h;
    p.ldo = c.ldh;
    p.m = c.M;
    p.n = c.F;
    p.k = c.K;
    p.save[0] = c.gate;
    p.save[1] = c.up;
    p.lds = c.ldg;
    p.act = c.act;
    return c.dtype == QTCQ_BF16 ? tiles_go<__bf16, __bf16, kGated>(p, st) : tiles_go<_Float16, _Float16, kGated>(p, st);
}

qtcq_status launch_gated_vjp(const GatedVjpCall& c, void* ws, hipStream_t st)
{
    return c.dtype == QTCQ_BF16 ? gated_vjp_impl<__bf16>(c, ws, st) : gated_vjp_impl<_Float16>(c, ws, st);
}

}  // namespace host
}  // namespace qtcq
