// Host-side check of the dense operators' validation layer (csrc/qtcq_dense.hip) and of the
// choice of kernel and workspace (csrc/dense_host.hpp), built host-only with
// AddressSanitizer and UndefinedBehaviorSanitizer by the test suite.  The launches are
// replaced by stand-ins that count their calls, so every path runs without a GPU:
//   - rejected calls reach no launch, accepted ones exactly one, empty ones none;
//   - over sizes from 0 to the limits the plans are whole: a tile height the kernels have,
//     shares that cover every step and are none of them empty, workspaces that hold the
//     shares' sums and the copies, and queries that give 0 beyond the limits.
// Prints "ok" and exits 0, or the first failure and exits 1.
#include <hip/hip_runtime.h>

#include <cstdint>
#include <cstdio>
#include <cstdlib>

#include "dense_host.hpp"

namespace qtcq {
namespace host {

static int g_launches = 0;
// a status no entry point returns, inside the enumeration's value range (0..7)
constexpr qtcq_status kLaunched = (qtcq_status)7;

static qtcq_status stand_in()
{
    ++g_launches;
    return kLaunched;
}

qtcq_status launch_quantize_rows(const void*, int, int64_t, int, int64_t, int8_t*, int64_t, float*, hipStream_t)
{ return stand_in(); }
qtcq_status launch_decode_matrix(int, const CodeSel&, bool, const uint32_t*, int, int, int, void*, int64_t, float*,
                                 hipStream_t)
{ return stand_in(); }
qtcq_status launch_matmul_int8(const int8_t*, int64_t, const float*, const int8_t*, int64_t, const float*, int, int, int,
                               int, void*, int64_t, void*, size_t, hipStream_t)
{ return stand_in(); }
qtcq_status launch_gated_forward(const GatedCall&, void*, size_t, hipStream_t) { return stand_in(); }
qtcq_status launch_gated_vjp(const GatedVjpCall&, void*, size_t, hipStream_t) { return stand_in(); }

}  // namespace host
}  // namespace qtcq

using namespace qtcq::host;

static void check(bool ok, const char* what, int a = 0, int b = 0, int c = 0)
{
    if (ok) return;
    std::printf("failed: %s (%d, %d, %d)\n", what, a, b, c);
    std::exit(1);
}

static void one(qtcq_status s, qtcq_status want, const char* what)
{
    const int n = g_launches;
    g_launches = 0;
    check(s == want && n == (want == kLaunched ? 1 : 0), what, s, n);
}

static void plans(int mode, int size, int m, int n, int k)
{
    for (int whole = 0; whole < 2; ++whole) {
        const ProductPlan p = plan_product(mode, size, m, n, k, whole != 0);
        if (p.skinny) {
            check((mode == kPlanInt8 || mode == kPlanGated) && m <= 64, "few rows", m, n, k);
            check(rows_product_bytes(mode, size, m, n, k, whole != 0) == (whole ? 0 : p.p_bytes + p.q_bytes),
                  "few rows take no scratch", m, n, k);
            continue;
        }
        check(p.fp == 2 || p.fp == 4 || p.fp == 8, "tile height", m, n, k);
        check(mode != kPlanGradW || (p.fp == 8 && p.shares == 1), "weight gradient", m, n, k);
        const int per = 128 / size, steps = (k + per - 1) / per * (mode == kPlanGradX ? 2 : 1);
        check(p.shares >= 1 && p.share_steps >= 1 && (int64_t)p.shares * p.share_steps >= steps, "shares cover k", m, n, k);
        check(p.shares == 1 || (int64_t)(p.shares - 1) * p.share_steps < steps, "no empty share", m, n, k);
        check(p.part_pitch % 4 == 0 && p.part_pitch >= n * (mode == kPlanGated ? 2 : 1), "pitch", m, n, k);
        check(p.shares == 1 ? p.part_bytes == 0 : p.part_bytes >= (size_t)p.shares * m * p.part_pitch * 4, "sums", m, n, k);
        if (mode == kPlanInt8 || mode == kPlanGated)
            check(p.p_bytes >= (size_t)m * k * size && p.q_bytes >= (size_t)n * k * size * (mode == kPlanGated ? 2 : 1) &&
                      p.p_bytes % 256 == 0 && p.q_bytes % 256 == 0,
                  "copies", m, n, k);
    }
}

int main()
{
    void* f = reinterpret_cast<void*>((uintptr_t)1 << 20);
    float* fl = static_cast<float*>(f);
    int8_t* b = static_cast<int8_t*>(f);
    uint32_t* u = static_cast<uint32_t*>(f);
    one(qtcq_quantize_rows(f, QTCQ_F16, 3, 5, 5, b, 5, fl, nullptr), kLaunched, "quantize");
    one(qtcq_quantize_rows(f, QTCQ_F16, 3, 0, 0, nullptr, 0, fl, nullptr), kLaunched, "quantize: empty rows have scales");
    one(qtcq_quantize_rows(f, QTCQ_F16, 0, 5, 5, b, 5, fl, nullptr), QTCQ_OK, "quantize: no rows");
    one(qtcq_quantize_rows(f, QTCQ_F16, 3, 5, 4, b, 5, fl, nullptr), QTCQ_ERR_INVALID_ARG, "quantize: stride");
    one(qtcq_decode_matrix(u, 32, 48, 16, 2, QTCQ_CODE_1MAD, 1, QTCQ_I8, f, 48, fl, nullptr), kLaunched, "decode");
    one(qtcq_decode_matrix(u, 32, 48, 16, 2, QTCQ_CODE_1MAD, 1, QTCQ_F32, f, 48, nullptr, nullptr), kLaunched, "decode f32");
    one(qtcq_decode_matrix(u, 32, 48, 16, 2, QTCQ_CODE_1MAD, 1, QTCQ_I8, f, 48, nullptr, nullptr), QTCQ_ERR_INVALID_ARG, "decode: scale");
    one(qtcq_decode_matrix(u, 32, 0, 16, 2, QTCQ_CODE_1MAD, 1, QTCQ_I8, nullptr, 0, fl, nullptr), kLaunched, "decode: empty rows have scales");
    one(qtcq_matmul_int8(b, 64, fl, b, 64, fl, 4, 8, 64, QTCQ_BF16, f, 8, nullptr, 0, nullptr), kLaunched, "product");
    one(qtcq_matmul_int8(b, 64, fl, b, 64, fl, 4, 8, 65, QTCQ_BF16, f, 8, nullptr, 0, nullptr), QTCQ_ERR_INVALID_ARG, "product: stride");
    one(qtcq_matmul_int8(nullptr, 0, fl, nullptr, 0, fl, 4, 8, 0, QTCQ_BF16, f, 8, nullptr, 0, nullptr), kLaunched, "product: empty sum");
    one(qtcq_gated_forward(f, 64, f, f, 64, QTCQ_F16, 4, 8, 64, QTCQ_ACT_RELU, f, 8, nullptr, nullptr, 0, nullptr, 0, nullptr), kLaunched, "gated");
    one(qtcq_gated_forward(f, 64, f, f, 64, QTCQ_F16, 4, 8, 64, QTCQ_ACT_RELU, f, 8, f, nullptr, 8, nullptr, 0, nullptr), QTCQ_ERR_INVALID_ARG, "gated: one of two");
    one(qtcq_gated_vjp(f, 64, f, f, 64, f, f, 8, f, 8, QTCQ_F16, 4, 8, 64, 0, f, 64, f, f, 64, f, 1 << 20, nullptr), kLaunched, "vjp");
    one(qtcq_gated_vjp(f, 64, f, f, 64, f, f, 8, f, 8, QTCQ_F16, 4, 8, 64, 0, nullptr, 0, nullptr, nullptr, 0, nullptr, 0, nullptr), QTCQ_OK, "vjp: nothing wanted");

    const int dims[] = {0, 1, 2, 4, 5, 16, 63, 64, 65, 128, 129, 333, 4096, 14336, 28672, 131071, (1 << 20) + 3, 1 << 21, 1 << 24};
    for (int m : dims)
        for (int n : dims)
            for (int k : dims) {
                const bool i8 = k <= kInt8MaxK && ((m + 127LL) / 128) * ((n + 63LL) / 64) <= kDenseMaxTiles;
                check(i8 || qtcq_matmul_int8_workspace_bytes(m, n, k, 0) == 0, "8-bit sizes", m, n, k);
                if (i8) plans(kPlanInt8, 1, m, n, k);
                const bool half = n <= kHalfMaxRow && k <= kHalfMaxRow && ((m + 127LL) / 128) * ((n + 63LL) / 64) <= kDenseMaxTiles;
                check(half || qtcq_gated_workspace_bytes(m, n, k, 0) == 0, "gated sizes", m, n, k);
                if (half) plans(kPlanGated, 2, m, n, k);
                const size_t a = qtcq_gated_vjp_workspace_bytes(m, n, k, 1), c = qtcq_gated_vjp_workspace_bytes(m, n, k, 0);
                if (half && m > 0 && n > 0 && a > 0) {
                    plans(kPlanGradX, 2, m, k, n);
                    plans(kPlanGradW, 2, n, k, m);
                    check(a >= (size_t)4 * m * n && c >= a + (size_t)2 * k * (2 * (size_t)n + m), "vjp scratch", m, n, k);
                }
            }
    std::printf("ok\n");
    return 0;
}
