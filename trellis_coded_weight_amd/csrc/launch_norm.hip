// launch_norm.hip -- launches of layer norm and of its gradients (norm.hpp).
#include "model_host.hpp"
#include "norm.hpp"

namespace qtcq {
namespace host {
namespace {

// f(RT, NCH) for rows of `chunks` 16-byte chunks: the fewest threads a row that hold it in
// up to `hold` registers' chunks each
template <typename F>
void with_row_shape(int chunks, F&& f)
{
    if (chunks <= 64)
        f(int_c<64>{}, int_c<1>{});
    else if (chunks <= 256)
        f(int_c<256>{}, int_c<1>{});
    else if (chunks <= 1024)
        f(int_c<1024>{}, int_c<1>{});
    else
        f(int_c<1024>{}, int_c<2>{});
}

// row groups of the weight gradients' sums
constexpr int kMostWorkgroups = 512;

template <typename T, typename W>
qtcq_status norm_impl(const NormArgs& a, hipStream_t st)
{
    constexpr int E = 16 / (int)sizeof(T);
    with_row_shape((a.cols + E - 1) / E, [&](auto rt, auto nch) {
        constexpr int RT = decltype(rt)::value, NCH = decltype(nch)::value, PER = norm_threads(RT) / RT;
        const int64_t most = 256 * (2048 / norm_threads(RT)), groups = (a.rows + PER - 1) / PER;
        hipLaunchKernelGGL((layer_norm_rows<T, W, RT, NCH>), dim3((unsigned)(groups < most ? groups : most)),
                           dim3(norm_threads(RT)), 0, st, a);
    });
    return launch_status();
}

int part_pitch(int cols) { return (cols + 7) / 8 * 8; }

template <typename T, typename W>
qtcq_status grad_impl(NormGradArgs a, W* grad_weight, W* grad_bias, float* part, hipStream_t st)
{
    constexpr int E = 16 / (int)sizeof(T);
    const int chunks = (a.cols + E - 1) / E;
    const bool want_w = grad_weight || grad_bias, held = chunks <= 2048;
    int groups = 0;
    a.part_pitch = part_pitch(a.cols);
    a.part = want_w && held ? part : nullptr;
    if (a.grad_x || (want_w && held))
        with_row_shape(chunks, [&](auto rt, auto nch) {
            constexpr int RT = decltype(rt)::value, NCH = decltype(nch)::value, PER = norm_threads(RT) / RT;
            const int64_t most = kMostWorkgroups, all = (a.rows + PER - 1) / PER;
            const unsigned grid = (unsigned)(all < most ? all : most);
            groups = grid * PER;
            if (grid == 0) return;
            hipLaunchKernelGGL((layer_norm_grad<T, W, RT, NCH>), dim3(grid), dim3(norm_threads(RT)), 0, st, a);
        });
    if (want_w) {
        if (!held) {
            const int64_t share = a.rows / 64 + 1;
            groups = (int)((a.rows + share - 1) / share);
            a.part = part;
            if (groups > 0)
                hipLaunchKernelGGL(norm_column_sums<T>, dim3((unsigned)(chunks + 31) / 32, groups), dim3(256), 0, st, a, share);
        }
        hipLaunchKernelGGL(join_norm_sums<W>, dim3((unsigned)(a.cols + 63) / 64, 2), dim3(256), 0, st, part, groups,
                           a.part_pitch, a.cols, grad_weight, grad_bias);
    }
    return launch_status();
}

template <typename F>
qtcq_status with_types(int dtype, int weight_dtype, F&& f)
{
    if (dtype == QTCQ_F32) return f(0.0f, 0.0f);
    if (dtype == QTCQ_BF16) return weight_dtype == QTCQ_F32 ? f((__bf16)0.0f, 0.0f) : f((__bf16)0.0f, (__bf16)0.0f);
    return weight_dtype == QTCQ_F32 ? f((_Float16)0.0f, 0.0f) : f((_Float16)0.0f, (_Float16)0.0f);
}

}  // namespace

size_t norm_grad_workspace_bytes(int64_t rows, int cols)
{
    const int64_t most = 4 * kMostWorkgroups;
    return (size_t)(rows < most ? (rows + 3) / 4 * 4 : most) * 2 * part_pitch(cols) * 4;
}

qtcq_status launch_layer_norm(const NormArgs& a, int dtype, int weight_dtype, hipStream_t st)
{
    return with_types(dtype, weight_dtype, [&](auto t, auto w) { return norm_impl<decltype(t), decltype(w)>(a, st); });
}

qtcq_status launch_layer_norm_vjp(const NormGradArgs& a, int dtype, int weight_dtype, void* grad_weight, void* grad_bias,
                                  void* ws, hipStream_t st)
{
    return with_types(dtype, weight_dtype, [&](auto t, auto w) {
        typedef decltype(w) W;
        return grad_impl<decltype(t), W>(a, static_cast<W*>(grad_weight), static_cast<W*>(grad_bias),
                                         static_cast<float*>(ws), st);
    });
}

}  // namespace host
}  // namespace qtcq
