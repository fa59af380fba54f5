// fp8_product.hpp -- what the products of e4m3 matrices with block scales share, gfx950.
//
//   y[i][j] = sum over blocks b of 128 of k:  sa[i][b] sw[j / 128][b] sum_{k in b} a[i][k] w[j][k]
//
// v_mfma_f32_16x16x128_f8f6f4 takes one block of k whole: lane l holds 32 bytes of row l % 16
// of each operand, the 16-byte chunks l / 16 and 4 + l / 16 of the block (both operands in the
// same order, so that the sum over k is the same), and its four results are the block's sums of
// four consecutive columns j of row i = l % 16.  Each block's sums start from 0 and are then
// scaled into the binary32 sums of the result by one fused multiply-add an element, the scale
// being fl(sa sw).
#pragma once

#include "codes.hpp"
#include "model_args.hpp"
#include "product.hpp"

namespace qtcq {

typedef int i32x8 __attribute__((ext_vector_type(8)));

// The 8-bit instruction does not keep all of a sum: 8 products next to each other in k are summed
// with each of them cut off, toward zero, at 2^-13 of the largest power of two among them (that of
// a product's two exponents together), and these sums are added in binary32.  (Found with single
// products; sums formed so in 64 bits are the instruction's on random values, to binary32's last
// digits.)  The results are then 1.4e-5 of their norm away from the exact sums on values of a
// Gaussian, 3e-6 where all products have one sign, 6.5e-5 where 3 columns of a in 100 are 64 times
// the others: far below the rounding to bf16 (1.7e-3 of the norm), and a fifteenth to a third of
// that to fp16 (2.1e-4), at twice the rate of the 16-bit instructions.  A group never loses more
// than 7 2^-13 of that power of two, a ninth of a step of bf16 there and most of one of fp16.  Where the
// results are binary32, or the weights' bytes are the work, the e4m3 values go to fp16, which
// holds them exactly, and the sums are those of binary32 (a float32 result at half the rate).
__device__ __forceinline__ f16x8 e4m3_to_f16(uint32_t lo, uint32_t hi)
{
    typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
    const f16x2 v[4] = {__builtin_bit_cast(f16x2, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, false)),
                        __builtin_bit_cast(f16x2, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, true)),
                        __builtin_bit_cast(f16x2, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, false)),
                        __builtin_bit_cast(f16x2, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, true))};
    return f16x8{v[0].x, v[0].y, v[1].x, v[1].y, v[2].x, v[2].y, v[3].x, v[3].y};
}

// The 32 bytes of a block of 128 of k that a lane holds of a row.
template <bool FAST> struct BlockOperand;
template <> struct BlockOperand<true> {
    i32x8 v;
    __device__ __forceinline__ BlockOperand() {}
    __device__ __forceinline__ BlockOperand(u32x4 a, u32x4 b)
        : v(__builtin_bit_cast(i32x8, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7))) {}
    __device__ __forceinline__ static f32x4 mul(const BlockOperand& a, const BlockOperand& b)
    {
        // both e4m3; scales of 0 select the form without the instruction's own scales
        return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a.v, b.v, f32x4{0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0, 0, 0, 0);
    }
};
template <> struct BlockOperand<false> {
    f16x8 v[4];
    __device__ __forceinline__ BlockOperand() {}
    __device__ __forceinline__ BlockOperand(u32x4 a, u32x4 b)
        : v{e4m3_to_f16(a.x, a.y), e4m3_to_f16(a.z, a.w), e4m3_to_f16(b.x, b.y), e4m3_to_f16(b.z, b.w)} {}
    __device__ __forceinline__ static f32x4 mul(const BlockOperand& a, const BlockOperand& b)
    {
        f32x4 c = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_16x16x32_f16(a.v[i], b.v[i], c, 0, 0, 0);
        return c;
    }
};

}  // namespace qtcq
