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
                           static_cast<const T*>(c.grad_h), c.ldgh, c.M, c.F, ldd, dg, du, c.pieces,
                           (int64_t)2 * c.M * ldd);
        return launch_status();
    });
}

template <typename T>
qtcq_status gated_vjp_impl(const GatedVjpCall& c, void* ws, size_t wsb, hipStream_t st)
{
    const VjpPlan v = plan_vjp(c.M, c.F, c.K, c.pieces);
    const bool ww = whole_chunks<T>(c.w_gate, c.ldw, c.K) && aligned16(c.w_up), xw = whole_chunks<T>(c.x, c.ldx, c.K);
    const size_t need = v.bytes(ww, xw, c.grad_x != nullptr, c.grad_w_gate != nullptr);
    if (need > 0 && (!ws || !aligned16(ws) || wsb < need)) return QTCQ_ERR_WORKSPACE;
    const int ldd = slope_pitch(c.F);
    T* dg = static_cast<T*>(ws);
    T* du = dg + (int64_t)c.M * ldd;
    char* more = static_cast<char*>(ws) + v.slopes;
    if (c.M > 0 && c.F > 0)
        if (const qtcq_status s = slopes<T>(c, ldd, dg, du, st); s != QTCQ_OK) return s;
    // both products from the slopes and, where the rows are not whole chunks, from copies
    ProductArgs ax = {};
    ax.p[0] = dg;
    ax.p[1] = du;
    ax.ldp = ax.pk = ax.pm = ldd;
    ax.pieces = c.pieces;
    ax.piece_step = (int64_t)2 * c.M * ldd;
    ax.n = ax.qn = c.K;
    ProductArgs aw = ax;
    PadCopies<T> copies(c.K);
    const ProductPlan plan = plan_product(kPlanGradX, (int)sizeof(T), c.M, c.K, c.F, true);
    char* at = more + v.part;
    if (c.grad_x) {
        ax.q[0] = c.w_gate;
        ax.q[1] = c.w_up;
        ax.ldq = c.ldw;
        if (!ww) {
            for (int i = 0; i < 2; ++i) ax.q[i] = copies.add(ax.q[i], c.ldw, c.F, &at);
            ax.ldq = ax.qn = copies.a.pitch;
        }
        ax.out[0] = c.grad_x;
        ax.ldo = c.ldgx;
        ax.m = c.M;
        ax.k = c.F;
        use_plan(ax, plan, more);
    } else {
        at = more;
    }
    if (c.grad_w_gate) {
        aw.q[0] = c.x;
        aw.ldq = c.ldx;
        if (!xw) {
            aw.q[0] = copies.add(c.x, c.ldx, c.M, &at);
            aw.ldq = aw.qn = copies.a.pitch;
        }
        aw.out[0] = c.grad_w_gate;
        aw.out[1] = c.grad_w_up;
        aw.ldo = c.ldgw;
        aw.m = c.F;
        aw.k = c.M;
        use_plan(aw, plan_product(kPlanGradW, (int)sizeof(T), c.F, c.K, c.M, true), nullptr);
    }
    copies.go(st);
    if (!c.grad_w_gate) return block_go<T, T, kGradX, 0>(ax, plan.fp, st);
    if (!c.grad_x) return block_go<T, T, kGradW, 0>(aw, 8, st);
    // One launch for both where they are small enough to fill the chip together (us, one launch
    // against two: 64x4096x1024 32.6 / 41.4, 700x5000x1280 105 / 110, 120x14336x4096 183 / 186;
    // on slopes of one part 28.9 / 36.1, 74 / 77, 147 / 157); beyond that the two are within 3%
    // (512x14336x4096 476 / 492, 4096x14336x4096 3260 both).  The results are the same bits.
    if ((double)c.M * c.F * c.K > 0x1p34) {
        if (const qtcq_status s = block_go<T, T, kGradX, 0>(ax, plan.fp, st); s != QTCQ_OK) return s;
        return block_go<T, T, kGradW, 0>(aw, 8, st);
    }
    const int64_t nx = block_groups<kGradX>(ax, plan.fp), n = nx + block_groups<kGradW>(aw, 8);
    auto go = [&](auto fp) {
        hipLaunchKernelGGL((gradient_products<T, decltype(fp)::value>), dim3((unsigned)n), dim3(BlockShape::kThreads), 0,
                           st, ax, aw, (int)nx);
    };
    if (plan.fp == 2)
        go(int_c<2>{});
    else if (plan.fp == 4)
        go(int_c<4>{});
    else
        go(int_c<8>{});
    join_go<T, T, kGradX, 0>(ax, st);
    return launch_status();
}

}  // namespace

qtcq_status launch_gated_vjp(const GatedVjpCall& c, void* ws, size_t wsb, hipStream_t st)
{
    return c.dtype == QTCQ_BF16 ? gated_vjp_impl<__bf16>(c, ws, wsb, st) : gated_vjp_impl<_Float16>(c, ws, wsb, st);
}

}  // namespace host
}  // namespace qtcq
