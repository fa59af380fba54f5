// launch_gated_vjp.hip -- launches of the gated projections' gradients.
#include "product_launch.hpp"

namespace qtcq {
namespace host {
namespace {

template <typename T>
qtcq_status slopes(const GatedVjpCall& c, int ldd, T* dg, T* du, hipStream_t st)
{
    const dim3 grid((unsigned)RowGrid{ldd / 8}.blocks(c.M)), block(256);
    return with_act(c.act, [&](auto act) {
        hipLaunchKernelGGL((gated_slopes<T, decltype(act)::value>), grid, block, 0, st,
                           static_cast<const T*>(c.gate), static_cast<const T*>(c.up), c.ldg,
                           static_cast<const T*>(c.grad_h), c.ldgh, c.M, c.F, ldd, dg, du);
        return launch_status();
    });
}

template <typename T>
qtcq_status gated_vjp_impl(const GatedVjpCall& c, void* ws, size_t wsb, hipStream_t st)
{
    const VjpPlan v = plan_vjp(c.M, c.F, c.K);
    const bool ww = whole_chunks<T>(c.w_gate, c.ldw, c.K) && aligned16(c.w_up), xw = whole_chunks<T>(c.x, c.ldx, c.K);
    const size_t need = v.bytes(ww, xw, c.grad_x != nullptr, c.grad_w_gate != nullptr);
    if (need > 0 && (!ws || !aligned16(ws) || wsb < need)) return QTCQ_ERR_WORKSPACE;
    const int ldd = slope_pitch(c.F);
    T* dg = static_cast<T*>(ws);
    T* du = dg + (int64_t)c.M * ldd;
    char* more = static_cast<char*>(ws) + v.slopes;
    if (c.M > 0 && c.F > 0)
        if (const qtcq_status s = slopes<T>(c, ldd, dg, du, st); s != QTCQ_OK) return s;
    ProductArgs a = {};
    a.p[0] = dg;
    a.p[1] = du;
    a.ldp = a.pk = a.pm = ldd;
    a.n = c.K;
    if (c.grad_x) {
        const ProductPlan plan = plan_product(kPlanGradX, (int)sizeof(T), c.M, c.K, c.F, true);
        a.q[0] = c.w_gate;
        a.q[1] = c.w_up;
        a.ldq = c.ldw;
        a.qn = c.K;
        if (!ww) {
            char* at = more + v.part;
            PadCopies<T> copies(c.K);
            for (int i = 0; i < 2; ++i) a.q[i] = copies.add(a.q[i], c.ldw, c.F, &at);
            a.ldq = a.qn = copies.a.pitch;
            copies.go(st);
        }
        a.out[0] = c.grad_x;
        a.ldo = c.ldgx;
        a.m = c.M;
        a.k = c.F;
        if (const qtcq_status s = block_go<T, T, kGradX, 0>(a, plan, more, st); s != QTCQ_OK) return s;
    }
    if (c.grad_w_gate) {
        const ProductPlan plan = plan_product(kPlanGradW, (int)sizeof(T), c.F, c.K, c.M, true);
        a.q[0] = c.x;
        a.ldq = c.ldx;
        a.qn = c.K;
        if (!xw) {
            char* at = more;
            PadCopies<T> copies(c.K);
            a.q[0] = copies.add(c.x, c.ldx, c.M, &at);
            a.ldq = a.qn = copies.a.pitch;
            copies.go(st);
        }
        a.out[0] = c.grad_w_gate;
        a.out[1] = c.grad_w_up;
        a.ldo = c.ldgw;
        a.m = c.F;
        a.k = c.M;
        return block_go<T, T, kGradW, 0>(a, plan, nullptr, st);
    }
    return launch_status();
}

}  // namespace

qtcq_status launch_gated_vjp(const GatedVjpCall& c, void* ws, size_t wsb, hipStream_t st)
{
    return c.dtype == QTCQ_BF16 ? gated_vjp_impl<__bf16>(c, ws, wsb, st) : gated_vjp_impl<_Float16>(c, ws, wsb, st);
}

}  // namespace host
}  // namespace qtcq
