// Host-side record of the dense operators' launches, built host-only by the test suite with
// qtcq_dense.hip and the launch units: hipLaunchKernel is replaced by a stand-in that keeps
// the kernel's name and its grid, so entry points run with made-up pointers and without a
// GPU.  Calls come from the standard input, one a line:
//   quantize DTYPE ROWS COLS
//   decode DTYPE M N TAILBITING
//   int8 DTYPE M N K ALIGNED
//   gated DTYPE M F K ALIGNED ACT
//   vjp DTYPE M F K ALIGNED ACT
//   kernels        (the names of all kernels, in the form of launches with no grid)
// (ALIGNED 0: operands one element off 16 bytes.)  Each answers with its status and, a
// line each, its launches: mangled name, grid.x, block.x, and for quantize_rows the rows and
// the three pointers it was given.
#include <hip/hip_runtime.h>

#include <cstdint>
#include <cstdio>
#include <cstring>
#include <iostream>
#include <map>
#include <string>

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

hipError_t hipLaunchKernel(const void* f, dim3 grid, dim3 block, void** args, size_t, hipStream_t)
{
    const char* name = kernels().at(f).c_str();
    std::printf("%s %u %u", name, grid.x, block.x);
    // quantize_rows(x, rows, cols, ldx, q, ldq, scale)
    if (std::strstr(name, "13quantize_rows"))
        std::printf(" %lld %llu %llu %llu", (long long)*static_cast<int64_t*>(args[1]),
                    (unsigned long long)*static_cast<uintptr_t*>(args[0]), (unsigned long long)*static_cast<uintptr_t*>(args[4]),
                    (unsigned long long)*static_cast<uintptr_t*>(args[6]));
    std::printf("\n");
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
    const auto at = [](unsigned long long where, int aligned, int size) {
        return reinterpret_cast<void*>(where + (aligned ? 0 : size));
    };
    while (std::cin >> op) {
        long long d = 0, m = 0, n = 0, k = 0, al = 1, act = 0;
        int s = -1;
        if (op == "kernels") {
            for (const auto& it : kernels()) std::printf("%s 0 0\n", it.second.c_str());
            s = 0;
        } else if (op == "quantize") {
            std::cin >> d >> m >> n;
            s = qtcq_quantize_rows(at(1ull << 40, 1, 0), (int)d, m, (int)n, n, (int8_t*)at(2ull << 40, 1, 0), n,
                                   (float*)at(3ull << 40, 1, 0), nullptr);
        } else if (op == "decode") {
            std::cin >> d >> m >> n >> al;
            s = qtcq_decode_matrix((const uint32_t*)at(1ull << 40, 1, 0), (int)m, (int)n, 16, 2, QTCQ_CODE_1MAD, (int)al, (int)d,
                                   at(2ull << 40, 1, 0), n, (float*)at(3ull << 40, 1, 0), nullptr);
        } else if (op == "int8") {
            std::cin >> d >> m >> n >> k >> al;
            s = qtcq_matmul_int8((const int8_t*)at(1ull << 40, (int)al, 1), k, (const float*)at(5ull << 40, 1, 0),
                                 (const int8_t*)at(2ull << 40, (int)al, 1), k, (const float*)at(6ull << 40, 1, 0), (int)m, (int)n,
                                 (int)k, (int)d, at(3ull << 40, 1, 0), n, at(4ull << 40, 1, 0), ~(size_t)0, nullptr);
        } else if (op == "gated") {
            std::cin >> d >> m >> n >> k >> al >> act;
            s = qtcq_gated_forward(at(1ull << 40, (int)al, 2), k, at(2ull << 40, (int)al, 2), at(3ull << 40, (int)al, 2), k, (int)d,
                                   (int)m, (int)n, (int)k, (int)act, at(5ull << 40, 1, 0), n, nullptr, nullptr, 0,
                                   at(4ull << 40, 1, 0), ~(size_t)0, nullptr);
        } else if (op == "vjp") {
            std::cin >> d >> m >> n >> k >> al >> act;
            s = qtcq_gated_vjp(at(1ull << 40, (int)al, 2), k, at(2ull << 40, (int)al, 2), at(3ull << 40, (int)al, 2), k,
                               at(5ull << 40, 1, 0), at(6ull << 40, 1, 0), n, at(7ull << 40, 1, 0), n, (int)d, (int)m, (int)n, (int)k,
                               (int)act, at(8ull << 40, 1, 0), k, at(9ull << 40, 1, 0), at(10ull << 40, 1, 0), k,
                               at(4ull << 40, 1, 0), ~(size_t)0, nullptr);
        }
        std::printf("= %d\n", s);
    }
    return 0;
}
