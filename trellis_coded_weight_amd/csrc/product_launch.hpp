// product_launch.hpp -- which kernel a product takes (skinny_product.hpp or
// block_product.hpp), its workspace and its launch, shared by the products' launch units.
#pragma once

#include "dense_host.hpp"
#include "block_product.hpp"
#include "skinny_product.hpp"

namespace qtcq {
namespace host {

static_assert(kPlanGated == kGated && kPlanInt8 == kInt8 && kPlanGradX == kGradX && kPlanGradW == kGradW, "modes");

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

// Few rows of P: 16 MI rows by 16 NJ columns a workgroup.  DEPTH blocks in flight fill the
// registers that the sums leave.
template <typename T, typename O, int MODE, int ACT, int MI, int NJ, bool ALIGNED>
qtcq_status skinny_shape(const ProductArgs& a, hipStream_t st)
{
    constexpr int frags = 2 * (MI + (MODE == kGated ? 2 * NJ : NJ));
    constexpr int DEPTH = frags <= 8 ? 4 : (frags <= 12 ? 3 : 2);
    const dim3 grid(blocks_for(a.n, 16 * NJ)), block(SkinnyShape::kThreads);
    hipLaunchKernelGGL((skinny_product<T, O, MODE, ACT, MI, NJ, DEPTH, ALIGNED>), grid, block, 0, st, a);
    return launch_status();
}

template <typename T, typename O, int MODE, int ACT>
qtcq_status skinny_go(const ProductArgs& a, bool whole, hipStream_t st)
{
    // Two groups of columns a workgroup halve the reads of P (the gated product has two as it
    // is); worth it once P has rows to read, where that leaves two workgroups a compute unit
    // (us, one group against two: 8-bit 28672x8192 at m = 4 47.2 / 56.1, 16384x4096 at m = 16
    // 20.9 / 18.8, m = 32 30.1 / 23.9).
    const bool wide = a.m > 8 && a.n >= 16 * 2 * 512;
    return with_bool(whole, [&](auto al) {
        constexpr bool ALIGNED = decltype(al)::value;
        auto go = [&](auto mi) {
            constexpr int MI = decltype(mi)::value;
            if constexpr (MODE == kInt8)
                if (wide) return skinny_shape<T, O, MODE, ACT, MI, 2, ALIGNED>(a, st);
            return skinny_shape<T, O, MODE, ACT, MI, 1, ALIGNED>(a, st);
        };
        if (a.m <= 16) return go(int_c<1>{});
        if (a.m <= 32) return go(int_c<2>{});
        return go(int_c<4>{});
    });
}

// workgroups of a product
template <int MODE>
int64_t block_groups(const ProductArgs& a, int fp)
{
    return (int64_t)blocks_for(a.m, BlockShape::rows(fp)) * blocks_for(a.n, BlockShape::cols(MODE)) *
           (MODE == kGradW ? 2 : a.shares);
}

template <typename T, typename O, int MODE, int ACT>
void join_go(const ProductArgs& a, hipStream_t st)
{
    if (a.shares < 2) return;
    const RowGrid g{MODE == kGated ? a.part_pitch / 8 : a.part_pitch / 4};
    hipLaunchKernelGGL((join_shares<T, O, MODE, ACT>), dim3((unsigned)g.blocks(a.m)), dim3(256), 0, st, a);
}

// the plan's shares into the arguments; `part`: p.part_bytes of scratch
inline void use_plan(ProductArgs& a, const ProductPlan& p, void* part)
{
    a.part = p.shares > 1 ? part : nullptr;
    a.part_pitch = p.part_pitch;
    a.shares = p.shares;
    a.share_steps = p.share_steps;
}

template <typename T, typename O, int MODE, int ACT, int FP>
void block_shape(const ProductArgs& a, hipStream_t st)
{
    hipLaunchKernelGGL((block_product<T, O, MODE, ACT, FP>), dim3((unsigned)block_groups<MODE>(a, FP)),
                       dim3(BlockShape::kThreads), 0, st, a);
}

template <typename T, typename O, int MODE, int ACT>
qtcq_status block_go(const ProductArgs& a, int fp, hipStream_t st)
{
    if constexpr (MODE == kGradW) {
        block_shape<T, O, MODE, ACT, 8>(a, st);
    } else {
        if (fp == 2)
            block_shape<T, O, MODE, ACT, 2>(a, st);
        else if (fp == 4)
            block_shape<T, O, MODE, ACT, 4>(a, st);
        else
            block_shape<T, O, MODE, ACT, 8>(a, st);
        join_go<T, O, MODE, ACT>(a, st);
    }
    return launch_status();
}

// Rows that start on 16 bytes and whose last chunk is whole, `inner` elements long, at a
// stride the block kernel's offsets hold.
template <typename T>
bool whole_chunks(const void* p, int64_t ld, int inner)
{
    constexpr int E = 16 / (int)sizeof(T);
    return aligned16(p) && ld % E == 0 && inner % E == 0 && ld * (int64_t)sizeof(T) <= BlockShape::kMaxStride;
}

// Copies of operands with rows of whole chunks, gathered and then launched together.
template <typename T>
struct PadCopies {
    PadArgs a = {};
    int n = 0;
    explicit PadCopies(int cols) { a.cols = cols, a.pitch = chunk_pitch(cols, (int)sizeof(T)); }
    // the copy goes to *at, which moves past it; returns its place
    const void* add(const void* src, int64_t ld, int64_t rows, char** at)
    {
        void* dst = *at;
        a.src[n] = src;
        a.dst[n] = dst;
        a.ld[n] = ld;
        a.rows[n] = rows;
        a.first[n + 1] = a.first[n] + RowGrid{a.pitch / (16 / (int)sizeof(T))}.blocks(rows);
        *at += round256((size_t)rows * a.pitch * sizeof(T));
        ++n;
        return dst;
    }
    void go(hipStream_t st)
    {
        for (int i = n; i < 3; ++i) a.first[i + 1] = a.first[n];
        constexpr int64_t most = 1 << 20;
        if (a.first[n] > 0)
            hipLaunchKernelGGL(pad_rows<T>, dim3((unsigned)(a.first[n] < most ? a.first[n] : most)), dim3(256), 0, st, a);
    }
};

// kInt8 and kGated: both operands stored [row][k].
template <typename T, typename O, int MODE, int ACT = 0>
qtcq_status rows_product(ProductArgs a, void* ws, size_t wsb, hipStream_t st)
{
    constexpr int QS = MODE == kGated ? 2 : 1;
    const bool pw = whole_chunks<T>(a.p[0], a.ldp, a.k);
    const bool qw = whole_chunks<T>(a.q[0], a.ldq, a.k) && (QS == 1 || aligned16(a.q[1]));
    const ProductPlan plan = plan_product(MODE, (int)sizeof(T), a.m, a.n, a.k, pw && qw);
    if (plan.skinny) return skinny_go<T, O, MODE, ACT>(a, pw && qw, st);
    const size_t need = plan.part_bytes + (pw ? 0 : plan.p_bytes) + (qw ? 0 : plan.q_bytes);
    if (need > 0 && (!ws || !aligned16(ws) || wsb < need)) return QTCQ_ERR_WORKSPACE;
    char* at = static_cast<char*>(ws) + plan.part_bytes;
    PadCopies<T> copies(a.k);
    a.pk = a.qk = a.k;
    if (!pw) {
        a.p[0] = copies.add(a.p[0], a.ldp, a.m, &at);
        a.ldp = a.pk = copies.a.pitch;
    }
    if (!qw) {
        for (int i = 0; i < QS; ++i) a.q[i] = copies.add(a.q[i], a.ldq, a.n, &at);
        a.ldq = a.qk = copies.a.pitch;
    }
    copies.go(st);
    use_plan(a, plan, ws);
    return block_go<T, O, MODE, ACT>(a, plan.fp, st);
}

}  // namespace host
}  // namespace qtcq
