// launch_distill.hip -- launches of the distillation loss and its gradient (distill.hpp).
#include "model_host.hpp"
#include "distill.hpp"

namespace qtcq {
namespace host {
namespace {

// Segments of a row: enough for two workgroups a compute unit, of at least 8192 elements.
void cut_row(DistillArgs& a)
{
    const int64_t want = a.rows > 0 ? (2 * kComputeUnits + a.rows - 1) / a.rows : 1;
    const int64_t most = ((int64_t)a.vocab + 8191) / 8192;
    const int64_t n = want < most ? want : most;
    a.segment = a.vocab;
    if (n >= 2) a.segment = (int)((a.vocab + n - 1) / n + 7) / 8 * 8;
    a.segments = n < 2 ? 1 : (a.vocab + a.segment - 1) / a.segment;
}

// The same for the loss, which pays a launch more for them: rows of up to 65536 elements, and
// 128 or more rows, stay whole (us with the gradient, whole rows against segments: 300x32000
// 18.6 / 22, 64x50000 16.4 / 20, 256x128000 33 / 46, 64x128000 26.8 / 20.1, 16x128000 24.9 / 18.3,
// 1x131072 24.3 / 18.2).
void cut_row_for_loss(DistillArgs& a)
{
    cut_row(a);
    if (a.vocab <= 65536 || a.rows >= 128) a.segments = 1, a.segment = a.vocab;
}

unsigned capped(int64_t n) { return (unsigned)(n < (1 << 20) ? n : 1 << 20); }

// f(threads a row, chunks a thread holds) for rows or segments of n elements, long ones (as the
// segments of a loss always are)
template <typename T, typename F>
void with_long_shape(int n, F&& f)
{
    const int chunks = n / (16 / (int)sizeof(T));
    if (chunks <= 2048)
        f(int_c<256>{}, int_c<8>{});
    else if (chunks <= 8192)
        f(int_c<512>{}, int_c<16>{});
    else
        f(int_c<1024>{}, int_c<16>{});
}

template <typename T, typename F>
void with_shape(int n, F&& f)
{
    if (n / (16 / (int)sizeof(T)) <= 256)
        f(int_c<64>{}, int_c<4>{});
    else
        with_long_shape<T>(n, f);
}

template <typename T>
qtcq_status grad_impl(const DistillArgs& a, hipStream_t st)
{
    with_shape<T>(a.segment, [&](auto nt, auto) {
        constexpr int NT = decltype(nt)::value;
        hipLaunchKernelGGL((distill_grad<T, NT>), dim3(capped(a.rows * a.segments)), dim3(NT), sizeof(Entry) * a.k, st, a);
    });
    return launch_status();
}

template <typename T>
qtcq_status distill_impl(const DistillArgs& a, hipStream_t st)
{
    const size_t entries = sizeof(Entry) * a.k;
    if (a.segments == 1) {
        with_shape<T>(a.vocab, [&](auto nt, auto hold) {
            constexpr int NT = decltype(nt)::value, HOLD = decltype(hold)::value;
            // as many workgroups as run at once (by their registers), each of which goes through its
            // rows; a training row's loads then overlap the stores of the one before
            constexpr int64_t at_once = (int64_t)kComputeUnits * (NT == 64 ? 32 : NT == 256 ? 5 : 1024 / NT);
            if (a.grad)
                hipLaunchKernelGGL((distill_train<T, NT, HOLD>), dim3((unsigned)(a.rows < at_once ? a.rows : at_once)),
                                   dim3(NT), entries, st, a);
            else
                hipLaunchKernelGGL((distill_rows<T, NT>), dim3(capped(a.rows)), dim3(NT), entries, st, a);
        });
        return launch_status();
    }
    with_long_shape<T>(a.segment, [&](auto nt, auto) {
        constexpr int NT = decltype(nt)::value;
        hipLaunchKernelGGL((distill_partial<T, NT>), dim3((unsigned)(a.rows * a.segments)), dim3(NT), 0, st, a);
    });
    hipLaunchKernelGGL((distill_join<T, 256>), dim3((unsigned)a.rows), dim3(256), entries, st, a);
    if (!a.grad) return launch_status();
    DistillArgs g = a;
    cut_row(g);
    return grad_impl<T>(g, st);
}

}  // namespace

size_t distill_workspace_bytes(int64_t rows, int vocab)
{
    DistillArgs a = {};
    a.rows = rows;
    a.vocab = vocab;
    cut_row_for_loss(a);
    return a.segments == 1 ? 0 : round256((size_t)rows * a.segments * 8) + round256((size_t)rows * kDistillStats * 4);
}

qtcq_status launch_distill(DistillArgs a, int dtype, void* ws, hipStream_t st)
{
    cut_row_for_loss(a);
    a.part = static_cast<float*>(ws);
    // the gradient's launch reads the statistics
    if (a.segments > 1 && !a.stats)
        a.stats = reinterpret_cast<float*>(static_cast<char*>(ws) + round256((size_t)a.rows * a.segments * 8));
    switch (dtype) {
    case QTCQ_BF16: return distill_impl<__bf16>(a, st);
    case QTCQ_F16: return distill_impl<_Float16>(a, st);
    default: return distill_impl<float>(a, st);
    }
}

qtcq_status launch_distill_grad(DistillArgs a, int dtype, hipStream_t st)
{
    cut_row(a);
    switch (dtype) {
    case QTCQ_BF16: return grad_impl<__bf16>(a, st);
    case QTCQ_F16: return grad_impl<_Float16>(a, st);
    default: return grad_impl<float>(a, st);
    }
}

}  // namespace host
}  // namespace qtcq
