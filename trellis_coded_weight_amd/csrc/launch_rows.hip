// launch_rows.hip -- launches of the row quantization and of the decode of streams to rows
// (quantize.hpp).
#include "dense_host.hpp"
#include "quantize.hpp"

namespace qtcq {
namespace host {
namespace {

template <typename T>
qtcq_status quantize_impl(const void* x, int64_t rows, int cols, int64_t ldx, int8_t* q, int64_t ldq, float* scale,
                          hipStream_t st)
{
    constexpr int E = 16 / (int)sizeof(T);
    auto go = [&](auto rt, auto nch) {
        constexpr int RT = decltype(rt)::value, NCH = decltype(nch)::value;
        // as many rows a launch as keep its threads below 2^32
        constexpr int64_t most = ((int64_t)1 << 31) / RT;
        for (int64_t r = 0; r < rows; r += most) {
            const int64_t n = rows - r < most ? rows - r : most;
            hipLaunchKernelGGL((quantize_rows<T, RT, NCH>), dim3(blocks_for(n, QuantShape::kThreads / RT)),
                               dim3(QuantShape::kThreads), 0, st, static_cast<const T*>(x) + r * ldx, n, cols, ldx,
                               q + r * ldq, ldq, scale + r);
        }
        return launch_status();
    };
    // A wave a row needs no barrier, a workgroup a row keeps longer rows in registers (us, wave
    // against workgroup, bf16: 65536x1024 38 / 72, 65536x2048 76 / 86, 8192x4096 25 / 20,
    // 16384x8192 108 / 74).
    const int chunks = (cols + E - 1) / E;
    if (chunks <= 64) return go(int_c<64>{}, int_c<1>{});
    if (chunks <= 256) return go(int_c<64>{}, int_c<4>{});
    if (chunks <= 1024) return go(int_c<256>{}, int_c<4>{});
    return go(int_c<256>{}, int_c<8>{});
}

template <int L, int CODE, bool TB>
qtcq_status decode_rows_impl(const uint32_t* bits, int M, int N, int dtype, void* w, int64_t ldw, float* scale,
                             const CodeArg& ca, hipStream_t st)
{
    const dim3 grid((unsigned)(M / 4)), block(DecodeRowsShape::kThreads);
    auto go = [&](auto out, auto hold) {
        hipLaunchKernelGGL((decode_rows<L, CODE, TB, decltype(out)::value, decltype(hold)::value>), grid, block, 0, st,
                           bits, M / 16, N / 16, w, ldw, scale, ca);
        return launch_status();
    };
    switch (dtype) {
    // codes held between the passes: 32 registers for up to 4096 columns, 64 beyond (3INST,
    // us, 32 against 64: 4096x4096 14.1 / 14.0, 28672x8192 115 / 107).  Columns past 4096 or
    // 8192 of a row are decoded twice (4096x14336 47 / 45, 8192x28672 150 / 146).
    case QTCQ_I8: return N <= 16 * DecodeRowsShape::kTiles ? go(int_c<0>{}, int_c<1>{}) : go(int_c<0>{}, int_c<2>{});
    case QTCQ_BF16: return go(int_c<1>{}, int_c<1>{});
    case QTCQ_F16: return go(int_c<2>{}, int_c<1>{});
    default: return go(int_c<3>{}, int_c<1>{});
    }
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

}  // namespace host
}  // namespace qtcq
