// launch_norm.hip -- launches of layer norm and of its gradients (norm.hpp).
#include "model_host.hpp"
#include "norm.hpp"

namespace qtcq {
namespace host {
namespace {

// most workgroups of the gradient, each of which writes a part of the weights' gradients
constexpr int kMostWorkgroups = 256;

template <typename T, typename W>
qtcq_status norm_impl(const NormArgs& a, hipStream_t st)
{
    constexpr int E = 16 / (int)sizeof(T);
    auto go = [&](auto rt, auto nch, auto is_long) {
        constexpr int RT = decltype(rt)::value, NCH = decltype(nch)::value, NT = norm_threads(RT), PER = NT / RT;
        const int64_t most = kComputeUnits * (2048 / NT), groups = (a.rows + PER - 1) / PER;
        hipLaunchKernelGGL((layer_norm_rows<T, W, RT, NCH, decltype(is_long)::value>), dim3((unsigned)(groups < most ? groups : most)), dim3(NT), 0, st,
                           a);
        return launch_status();
    };
    const int chunks = (a.cols + E - 1) / E;
    if (chunks <= 64) return go(int_c<64>{}, int_c<1>{}, bool_c<false>{});
    if (chunks <= 128) return go(int_c<64>{}, int_c<2>{}, bool_c<false>{});
    if (chunks <= 256) return go(int_c<64>{}, int_c<4>{}, bool_c<false>{});
    if (chunks <= 512) return go(int_c<256>{}, int_c<2>{}, bool_c<false>{});
    if (chunks <= 1024) return go(int_c<256>{}, int_c<4>{}, bool_c<false>{});
    if (chunks <= 2048) return go(int_c<1024>{}, int_c<2>{}, bool_c<false>{});
    return go(int_c<1024>{}, int_c<2>{}, bool_c<true>{});
}

int part_pitch(int cols) { return (cols + 7) / 8 * 8; }

// Whether the gradients take one launch that reads the rows a second time for the weights', by
// the sizes and the bytes of an element: few rows, whose second reading comes from the caches, in up
// to three readings of 512 rows, each longer the more columns there are (us of whole calls, one
// launch against two; 16 bits: 512x8192 13.9 / 17.9, 768x4096 13.8 / 16.7, 1024x3000 15.9 / 17.4,
// 1280x2048 14.9 / 16.5, 1536x1000 15.2 / 16.3, 1536x2048 16.2 / 16.9, 1400x2200 19.3 / 17.4, 2048x1000
// 19.5 / 16.3, 1000x8192 22.5 / 20.3; float32: 333x2731 13.2 / 16.8, 512x8192 17.7 / 17.6, 768x4096 15.7 /
// 16.8, 640x4900 19.9 / 17.2, 1024x2048 14.9 / 16.7, 1024x2560 18.0 / 16.6, 1536x1024 15.3 / 16.5, 1280x1600
// 17.2 / 16.5, 1536x2048 19.1 / 16.4).
bool norm_few_rows(int64_t rows, int cols, size_t size)
{
    if (rows <= 512) return cols <= 8192;
    if (size == 2) return rows <= 1024 ? rows * cols <= 3 << 20 : rows <= 1536 && cols <= 2048;
    return rows <= 768 ? cols <= 4096 : rows <= 1024 ? cols <= 2048 : rows <= 1536 && cols <= 1024;
}

template <typename T, typename W>
qtcq_status grad_impl(NormGradArgs a, W* grad_weight, W* grad_bias, float* part, hipStream_t st)
{
    constexpr int E = 16 / (int)sizeof(T);
    const int chunks = (a.cols + E - 1) / E;
    if (norm_few_rows(a.rows, a.cols, sizeof(T))) {
        auto few = [&](auto rt, auto nch) {
            constexpr int RT = decltype(rt)::value, NCH = decltype(nch)::value, R = NCH == 1 ? 2 : 1;
            constexpr int PER = kNormGradThreads / RT * R;
            const int nx = a.grad_x ? (int)((a.rows + PER - 1) / PER) : 0;
            const int ny = grad_weight || grad_bias ? (chunks + kNormFewChunks - 1) / kNormFewChunks : 0;
            hipLaunchKernelGGL((layer_norm_grad_few<T, W, RT, NCH, R>), dim3(nx + ny), dim3(kNormGradThreads), 0, st, a, grad_weight,
                               grad_bias, nx);
            return launch_status();
        };
        if (chunks <= 64) return few(int_c<64>{}, int_c<1>{});
        if (chunks <= 128) return few(int_c<128>{}, int_c<1>{});
        if (chunks <= 256) return few(int_c<256>{}, int_c<1>{});
        if (chunks <= 512) return few(int_c<512>{}, int_c<1>{});
        if (chunks <= 1024) return few(int_c<1024>{}, int_c<1>{});
        if constexpr (E == 4) return few(int_c<1024>{}, int_c<2>{});
    }
    const bool want_w = grad_weight || grad_bias, held = chunks <= 2048;
    int groups = 0;
    a.part_pitch = part_pitch(a.cols);
    a.part = want_w && held ? part : nullptr;
    auto go = [&](auto rt, auto nch, auto rows, auto is_long) {
        constexpr int RT = decltype(rt)::value, NCH = decltype(nch)::value, R = decltype(rows)::value;
        constexpr int PER = kNormGradThreads / RT * R;
        const int64_t all = (a.rows + PER - 1) / PER;
        groups = (int)(all < kMostWorkgroups ? all : kMostWorkgroups);
        if (groups > 0)
            hipLaunchKernelGGL((layer_norm_grad<T, W, RT, NCH, R, decltype(is_long)::value>), dim3(groups), dim3(kNormGradThreads), 0, st, a);
    };
    if (a.grad_x || (want_w && held)) {
        if (chunks <= 64)
            go(int_c<64>{}, int_c<1>{}, int_c<2>{}, bool_c<false>{});
        else if (chunks <= 128)
            go(int_c<128>{}, int_c<1>{}, int_c<2>{}, bool_c<false>{});
        else if (chunks <= 256)
            go(int_c<256>{}, int_c<1>{}, int_c<2>{}, bool_c<false>{});
        else if (chunks <= 512)
            go(int_c<512>{}, int_c<1>{}, int_c<2>{}, bool_c<false>{});
        else if (chunks <= 1024)
            go(int_c<1024>{}, int_c<1>{}, int_c<2>{}, bool_c<false>{});
        else if (held)
            go(int_c<1024>{}, int_c<2>{}, int_c<1>{}, bool_c<false>{});
        else
            go(int_c<1024>{}, int_c<1>{}, int_c<1>{}, bool_c<true>{});
    }
    if (want_w) {
        if (!held) {
            const int64_t share = a.rows / 64 + 1;
            groups = (int)((a.rows + share - 1) / share);
            a.part = part;
            if (groups > 0)
                hipLaunchKernelGGL(norm_column_sums<T>, dim3((unsigned)(chunks + 31) / 32, groups), dim3(256), 0, st, a, share);
        }
        hipLaunchKernelGGL(join_norm_sums<W>, dim3((unsigned)(a.cols + 31) / 32, 2), dim3(256), 0, st, part, groups,
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

size_t norm_grad_workspace_bytes(int64_t rows, int cols, size_t size)
{
    if (norm_few_rows(rows, cols, size)) return 0;
    return (size_t)(rows < kMostWorkgroups ? rows : kMostWorkgroups) * 2 * part_pitch(cols) * 4;
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
