// Host-side record of the model operators' launches, built host-only by the test suite with
// qtcq_model.hip and the launch units: hipLaunchKernel is replaced by a stand-in that keeps
// the kernel's name and its grid, so entry points run with made-up pointers and without a
// GPU.  Calls come from the standard input, one a line:
//   blocks DTYPE ROWS COLS BLOCK_ROWS
//   fp8 DTYPE M N K ALIGNED
//   norm DTYPE WEIGHT_DTYPE ROWS COLS
//   norm_vjp DTYPE WEIGHT_DTYPE ROWS COLS WANT    (1: grad_x, 2: weights' gradients, 3: both)
//   distill DTYPE ROWS VOCAB K GRAD
//   distill_vjp DTYPE ROWS VOCAB K
//   plan M N K WHOLE PRECISE    (the e4m3 product's choices, in the form of a launch)
//   kernels        (the names of all kernels, in the form of launches with no grid)
// (ALIGNED 0: operands one byte off 16.)  Workspaces are of the sizes queried.  Each answers with its status and, a line each, its
// launches: mangled name, grid.x, grid.y, block.x.
#include <hip/hip_runtime.h>

#include <cstdint>
#include <cstdio>
#include <iostream>
#include <map>
#include <string>

#include "model_host.hpp"
#include "qtcq.h"

static dim3 g_grid, g_block;

static std::map<const void*, std::string>& kernels()
{
    static std::map<const void*, std::string> names;
    return names;
}

extern "C" {

hipError_t __hipPushCallConfiguration(dim3 grid, dim3 block, size_t, hipStream_t)
{
    g_grid = grid;
    g_block = block;
    return hipSuccess;
}

hipError_t __hipPopCallConfiguration(dim3* grid, dim3* block, size_t* shared, hipStream_t* stream)
{
    *grid = g_grid;
    *block = g_block;
    *shared = 0;
    *stream = nullptr;
    return hipSuccess;
}

hipError_t hipLaunchKernel(const void* f, dim3 grid, dim3 block, void**, size_t, hipStream_t)
{
    const char* name = kernels().at(f).c_str();
    std::printf("%s %u %u %u\n", name, grid.x, grid.y, block.x);
    return hipSuccess;
}

hipError_t hipGetLastError() { return hipSuccess; }
void** __hipRegisterFatBinary(const void*) { static void* h; return &h; }
void __hipUnregisterFatBinary(void**) {}
void __hipRegisterFunction(void**, const void* f, char*, const char* name, unsigned, void*, void*, void*, void*, int*)
{
    kernels()[f] = name;
}
void __hipRegisterVar(void**, void*, char*, const char*, int, size_t, int, int) {}

}  // extern "C"

int main()
{
    std::string op;
    const auto at = [](unsigned long long tb, int off = 0) { return reinterpret_cast<void*>((tb << 40) + off); };
    const auto f = [&](unsigned long long tb) { return static_cast<float*>(at(tb)); };
    const auto b = [&](unsigned long long tb, int off = 0) { return static_cast<uint8_t*>(at(tb, off)); };
    while (std::cin >> op) {
        long long d = 0, wd = 0, m = 0, n = 0, k = 0, o = 0;
        int s = -1;
        if (op == "kernels") {
            for (const auto& it : kernels()) std::printf("%s 0 0 0\n", it.second.c_str());
            s = 0;
        } else if (op == "blocks") {
            std::cin >> d >> m >> n >> o;
            s = qtcq_quantize_blocks(at(1), (int)d, m, (int)n, n, (int)o, b(2), n, f(3), n + 1, 1, nullptr);
        } else if (op == "fp8") {
            std::cin >> d >> m >> n >> k >> o;
            s = qtcq_matmul_fp8(b(1, !o), k, f(2), 1, m, b(3, !o), k, f(4), 1, n, (int)m, (int)n, (int)k, (int)d, at(5), n, at(6),
                                qtcq_matmul_fp8_workspace_bytes((int)m, (int)n, (int)k, (int)o), nullptr);
        } else if (op == "plan") {
            std::cin >> m >> n >> k >> o >> d;
            const qtcq::host::Fp8Plan p = qtcq::host::plan_fp8((int)m, (int)n, (int)k, o != 0, d != 0);
            std::printf("%d %d %d %d %d %d %zu %zu %zu\n", p.skinny, p.fp, p.qg, p.shares, p.share_steps, p.part_pitch,
                        p.part_bytes, p.a_bytes, p.w_bytes);
            s = 0;
        } else if (op == "norm") {
            std::cin >> d >> wd >> m >> n;
            s = qtcq_layer_norm(at(1), (int)d, m, (int)n, n, at(2), at(3), (int)wd, 1e-5f, at(4), n, f(5), f(6), nullptr);
        } else if (op == "norm_vjp") {
            std::cin >> d >> wd >> m >> n >> o;
            s = qtcq_layer_norm_vjp(at(1), (int)d, m, (int)n, n, at(2), (int)wd, f(3), f(4), at(5), n, o & 1 ? at(6) : nullptr, n,
                                    o & 2 ? at(7) : nullptr, o & 2 ? at(8) : nullptr, at(9),
                                    qtcq_layer_norm_vjp_workspace_bytes(m, (int)n), nullptr);
        } else if (op == "distill") {
            std::cin >> d >> m >> n >> k >> o;
            s = qtcq_distill_topk(at(1), (int)d, m, (int)n, n, at(2), 8, k, at(3), QTCQ_F32, k, (int)k, 1.0f, nullptr, f(4),
                                  nullptr, f(5), o ? at(6) : nullptr, n, at(7),
                                  qtcq_distill_topk_workspace_bytes(m, (int)n), nullptr);
        } else if (op == "distill_vjp") {
            std::cin >> d >> m >> n >> k;
            s = qtcq_distill_topk_vjp(at(1), (int)d, m, (int)n, n, at(2), 8, k, at(3), QTCQ_F32, k, (int)k, 1.0f, f(4), f(5),
                                      at(6), n, nullptr);
        }
        std::printf("= %d\n", s);
    }
    return 0;
}
