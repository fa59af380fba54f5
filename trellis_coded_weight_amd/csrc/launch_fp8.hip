// launch_fp8.hip -- launches of the product of e4m3 matrices with block scales: few rows
// (fp8_skinny.hpp) and tiles (fp8_block.hpp).
#include "model_host.hpp"
#include "fp8_block.hpp"
#include "fp8_skinny.hpp"
#include "product_launch.hpp"

namespace qtcq {
namespace host {
namespace {

template <typename O, int MI>
void skinny_shape(const Fp8Args& a, bool whole, hipStream_t st)
{
    const dim3 grid(blocks_for(a.n, 16)), block(Fp8SkinnyShape::kThreads);
    constexpr int DEPTH = MI == 1 ? 4 : (MI == 2 ? 3 : 2);
    if (whole)
        hipLaunchKernelGGL((fp8_skinny_product<O, MI, DEPTH, true>), grid, block, 0, st, a);
    else
        hipLaunchKernelGGL((fp8_skinny_product<O, MI, DEPTH, false>), grid, block, 0, st, a);
}

template <typename O, int FP, int QG>
void block_shape(const Fp8Args& a, hipStream_t st)
{
    const int64_t tiles = (int64_t)blocks_for(a.m, Fp8Shape::rows(FP)) * blocks_for(a.n, Fp8Shape::cols(QG));
    hipLaunchKernelGGL((fp8_block_product<O, FP, QG, sizeof(O) == 2>), dim3((unsigned)(tiles * a.shares)),
                       dim3(Fp8Shape::kThreads), 0, st, a);
}

template <typename O>
qtcq_status product(Fp8Args a, void* ws, size_t wsb, hipStream_t st)
{
    constexpr bool PRECISE = sizeof(O) == 4;
    const bool aw = whole_chunks<int8_t>(a.a, a.lda, a.k), ww = whole_chunks<int8_t>(a.w, a.ldw, a.k);
    const Fp8Plan plan = plan_fp8(a.m, a.n, a.k, aw && ww, PRECISE);
    if (plan.skinny) {
        if (a.m <= 16)
            skinny_shape<O, 1>(a, aw && ww, st);
        else if (a.m <= 32)
            skinny_shape<O, 2>(a, aw && ww, st);
        else
            skinny_shape<O, 4>(a, aw && ww, st);
        return launch_status();
    }
    const size_t need = plan.part_bytes + (aw ? 0 : plan.a_bytes) + (ww ? 0 : plan.w_bytes);
    if (need > 0 && (!ws || !aligned16(ws) || wsb < need)) return QTCQ_ERR_WORKSPACE;
    char* at = static_cast<char*>(ws) + plan.part_bytes;
    PadCopies<int8_t> copies(a.k);
    a.ak = a.wk = a.k;
    if (!aw) {
        a.a = static_cast<const uint8_t*>(copies.add(a.a, a.lda, a.m, &at));
        a.lda = a.ak = copies.a.pitch;
    }
    if (!ww) {
        a.w = static_cast<const uint8_t*>(copies.add(a.w, a.ldw, a.n, &at));
        a.ldw = a.wk = copies.a.pitch;
    }
    copies.go(st);
    a.part = plan.shares > 1 ? static_cast<float*>(ws) : nullptr;
    a.part_pitch = plan.part_pitch;
    a.shares = plan.shares;
    a.share_steps = plan.share_steps;
    if (plan.fp == 2)
        plan.qg == 2 ? block_shape<O, 2, 2>(a, st) : block_shape<O, 2, 4>(a, st);
    else if (PRECISE || plan.fp == 4)
        plan.qg == 2 ? block_shape<O, 4, 2>(a, st) : block_shape<O, 4, 4>(a, st);
    else if constexpr (!PRECISE)
        block_shape<O, 8, 4>(a, st);
    // the shares' sums as those of any product
    ProductArgs j = {};
    j.out[0] = a.y;
    j.ldo = a.ldy;
    j.m = a.m;
    j.n = a.n;
    j.part = a.part;
    j.part_pitch = a.part_pitch;
    j.shares = a.shares;
    join_go<__bf16, O, kGradX, 0>(j, st);
    return launch_status();
}

}  // namespace

qtcq_status launch_matmul_fp8(const Fp8Args& a, int dtype, void* ws, size_t wsb, hipStream_t st)
{
    switch (dtype) {
    case QTCQ_BF16: return product<__bf16>(a, ws, wsb, st);
    case QTCQ_F16: return product<_Float16>(a, ws, wsb, st);
    default: return product<float>(a, ws, wsb, st);
    }
}

}  // namespace host
}  // namespace qtcq
