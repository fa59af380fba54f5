// launch_fp8.hip -- launches of the product of e4m3 matrices with block scales.
#include "model_host.hpp"
#include "fp8_skinny.hpp"
#include "block_product.hpp"

namespace qtcq {
namespace host {
namespace {

template <typename O, int MI>
void skinny_shape(const Fp8Args& a, bool whole, hipStream_t st)
{
    const dim3 grid(blocks_for(a.n, 16), blocks_for(a.m, 16 * MI)), block(Fp8SkinnyShape::kThreads);
    if (whole)
        hipLaunchKernelGGL((fp8_skinny_product<O, MI, 1, 4, true>), grid, block, 0, st, a);
    else
        hipLaunchKernelGGL((fp8_skinny_product<O, MI, 1, 4, false>), grid, block, 0, st, a);
}

template <typename O>
qtcq_status product(const Fp8Args& a, hipStream_t st)
{
    const bool whole = aligned16(a.a) && aligned16(a.w) && a.lda % 16 == 0 && a.ldw % 16 == 0 && a.k % 16 == 0 &&
                       a.lda <= BlockShape::kMaxStride && a.ldw <= BlockShape::kMaxStride;
    if (a.m <= 16)
        skinny_shape<O, 1>(a, whole, st);
    else
        skinny_shape<O, 2>(a, whole, st);
    return launch_status();
}

}  // namespace

size_t fp8_workspace_bytes(int, int, int, bool) { return 0; }

qtcq_status launch_matmul_fp8(Fp8Args a, int dtype, void*, size_t, hipStream_t st)
{
    switch (dtype) {
    case QTCQ_BF16: return product<__bf16>(a, st);
    case QTCQ_F16: return product<_Float16>(a, st);
    default: return product<float>(a, st);
    }
}

}  // namespace host
}  // namespace qtcq
