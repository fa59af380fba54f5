// launch_products.hip -- launches of the 8-bit product and of the gated projections and
// their gradients (tile_product.hpp, block_product.hpp).
#include "dense_host.hpp"
#include "block_product.hpp"

namespace qtcq {
namespace host {
namespace {

// rows that start on 16 bytes and whose last chunk is whole, `inner` elements long
template <typename T>
bool whole_chunks(const void* p, int64_t ld, int inner)
{
    constexpr int E = 16 / (int)sizeof(T);
    return aligned16(p) && ld % E == 0 && inner % E == 0 && ld * (int64_t)sizeof(T) <= BlockShape::kMaxStride;
}

template <typename T, int MODE>
bool block_ok(const ProductArgs& a)
{
    const int pk = MODE == kGradW ? a.m : (MODE == kGradX ? a.kp : a.k);
    const bool p = whole_chunks<T>(a.p[0], a.ldp, pk) && aligned16(a.p[1]);
    return p && whole_chunks<T>(a.q[0], a.ldq, MODE == kGradX || MODE == kGradW ? a.n : a.k) && aligned16(a.q[1]);
}

template <typename T, typename O, int MODE, int ACT = 0>
qtcq_status tiles_go(const ProductArgs& a, hipStream_t st)
{
    if (block_ok<T, MODE>(a) && a.m > 64) {
        const int64_t n = (int64_t)blocks_for(a.m, BlockShape::kRows) * blocks_for(a.n, BlockShape::cols(MODE));
        hipLaunchKernelGGL((block_product<T, O, MODE, ACT>), dim3((unsigned)n, 1, MODE == kGradW ? 2 : 1),
                           dim3(BlockShape::kThreads), 0, st, a);
        return launch_status();
    }
    const int64_t tiles = (int64_t)blocks_for(a.m, TileShape::kRows) * blocks_for(a.n, TileShape::cols(MODE));
    const dim3 grid((unsigned)tiles, 1, MODE == kGradW ? 2 : 1), block(TileShape::kThreads);
    hipLaunchKernelGGL((tile_product<T, O, MODE, ACT>), grid, block, 0, st, a);
    return launch_status();
}

// f(int_c<ACT>{})
template <typename F>
qtcq_status with_act(int act, F&& f)
{
    switch (act) {
    case kActSilu: return f(int_c<kActSilu>{});
    case kActGelu: return f(int_c<kActGelu>{});
    case kActGeluTanh: return f(int_c<kActGeluTanh>{});
    case kActRelu: return f(int_c<kActRelu>{});
    default: return f(int_c<kActSigmoid>{});
    }
}

template <typename T>
qtcq_status slopes(const GatedVjpCall& c, int ldd, T* dg, T* du, hipStream_t st)
{
    const dim3 grid(blocks_for((int64_t)c.M * (ldd / 8), 256)), block(256);
    return with_act(c.act, [&](auto act) {
        hipLaunchKernelGGL((gated_slopes<T, decltype(act)::value>), grid, block, 0, st,
                           static_cast<const T*>(c.gate), static_cast<const T*>(c.up), c.ldg,
                           static_cast<const T*>(c.grad_h), c.ldgh, c.M, c.F, ldd, dg, du);
        return launch_status();
    });
}

template <typename T>
qtcq_status gated_vjp_impl(const GatedVjpCall& c, void* ws, hipStream_t st)
{
    const int ldd = slope_pitch(c.F);
    T* dg = static_cast<T*>(ws);
    T* du = dg + (int64_t)c.M * ldd;
    if (c.M > 0 && c.F > 0)
        if (const qtcq_status s = slopes<T>(c, ldd, dg, du, st); s != QTCQ_OK) return s;
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
        a.kp = ldd;
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
    return with_act(c.act, [&](auto act) {
        constexpr int ACT = decltype(act)::value;
        return c.dtype == QTCQ_BF16 ? tiles_go<__bf16, __bf16, kGated, ACT>(p, st)
                                    : tiles_go<_Float16, _Float16, kGated, ACT>(p, st);
    });
}

qtcq_status launch_gated_vjp(const GatedVjpCall& c, void* ws, hipStream_t st)
{
    return c.dtype == QTCQ_BF16 ? gated_vjp_impl<__bf16>(c, ws, st) : gated_vjp_impl<_Float16>(c, ws, st);
}

}  // namespace host
}  // namespace qtcq
