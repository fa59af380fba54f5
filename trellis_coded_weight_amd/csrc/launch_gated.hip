// launch_gated.hip -- launches of the gated projections.
#include "product_launch.hpp"

namespace qtcq {
namespace host {

qtcq_status launch_gated_forward(const GatedCall& c, void* ws, size_t wsb, hipStream_t st)
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
        return c.dtype == QTCQ_BF16 ? rows_product<__bf16, __bf16, kGated, ACT>(p, ws, wsb, st)
                                    : rows_product<_Float16, _Float16, kGated, ACT>(p, ws, wsb, st);
    });
}

}  // namespace host
}  // namespace qtcq
