// norm.hpp -- layer norm over the columns of a row, and its gradients, gfx950.
//
//   mean = sum x / n,  rstd = 1 / sqrt(sum (x - mean)^2 / n + eps),  xh = (x - mean) rstd,
//   y = xh w + b;
//   with gw = g w:  dx = rstd (gw - sum gw / n - xh sum(gw xh) / n),
//   dw = sum over rows of g xh,  db = sum over rows of g.
//
// All in binary32, each result rounded once.  The variance is the mean of the squared
// differences, never a difference of squares: a row is held in registers between its passes.
//
// Both directions are bound by memory (x, g read once, y or dx written once).  RT threads a
// row (64: a wave, no barrier; 256 and 1024: a workgroup), NCH 16-byte chunks a thread; a
// workgroup goes through rows blockIdx, + gridDim, ... and keeps the weights of its columns,
// which all rows share, in registers.  So do the sums of dw and db: each row group (the RT
// threads) adds its rows in order and writes its sums to part, which join_norm_sums adds in
// order.  No atomics: the same bits on every run.
#pragma once

#include "model_args.hpp"
#include "reduce.hpp"
#include "rows.hpp"

namespace qtcq {

constexpr int norm_threads(int rt) { return rt < 256 ? 256 : rt; }

// Sums over the RT threads of a row of N values at once; red: [2][N][16] in LDS, the two
// halves in turn, so that one barrier a call is enough.
template <int RT, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float (*red)[N][16], int& turn)
{
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
    if constexpr (RT > 64) {
        const int wave = threadIdx.x >> 6;
        if ((threadIdx.x & 63) == 0)
#pragma unroll
            for (int i = 0; i < N; ++i) red[turn][i][wave] = v[i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            v[i] = 0.0f;
#pragma unroll
            for (int w = 0; w < RT / 64; ++w) v[i] += red[turn][i][w];
        }
        turn ^= 1;
    }
}

// grid.x: any number of workgroups up to ceil(rows / row groups a workgroup)
template <typename T, typename W, int RT, int NCH>
__global__ void __launch_bounds__(norm_threads(RT))
layer_norm_rows(NormArgs a)
{
    constexpr int E = 16 / (int)sizeof(T), PER = norm_threads(RT) / RT;
    __shared__ float red[2][1][16];
    const int t = threadIdx.x % RT, n = a.cols, nch = (n + E - 1) / E;
    const T* x = static_cast<const T*>(a.x);
    T* y = static_cast<T*>(a.y);
    const W* weight = static_cast<const W*>(a.weight);
    const W* bias = static_cast<const W*>(a.bias);
    Elems<W, E> hw[NCH], hb[NCH];
    auto weights = [&](int c) { return load_elems<W, E>(weight, c * E, weight ? n : 0, (W)1.0f); };
    auto biases = [&](int c) { return load_elems<W, E>(bias, c * E, bias ? n : 0, (W)0.0f); };
#pragma unroll
    for (int i = 0; i < NCH; ++i)
        if (t + i * RT < nch) hw[i] = weights(t + i * RT), hb[i] = biases(t + i * RT);
    int turn = 0;
    for (int64_t row = (int64_t)blockIdx.x * PER + threadIdx.x / RT; row < a.rows; row += (int64_t)gridDim.x * PER) {
        const T* xr = x + row * a.ldx;
        Elems<T, E> held[NCH];
        auto load = [&](int c) { return load_elems<T, E>(xr, c * E, n, (T)0.0f); };
        float s[1] = {0.0f};
        auto add = [&](const Elems<T, E>& o) {
#pragma unroll
            for (int e = 0; e < E; ++e) s[0] += to_f32(o.e[e]);
        };
#pragma unroll
        for (int i = 0; i < NCH; ++i)
            if (t + i * RT < nch) held[i] = load(t + i * RT);
#pragma unroll
        for (int i = 0; i < NCH; ++i)
            if (t + i * RT < nch) add(held[i]);
        for (int c = t + NCH * RT; c < nch; c += RT) add(load(c));
        row_sums<RT>(s, red, turn);
        const float mean = s[0] / (float)n;
        s[0] = 0.0f;
        auto square = [&](int c, const Elems<T, E>& o) {
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float d = c * E + e < n ? to_f32(o.e[e]) - mean : 0.0f;
                s[0] = __builtin_fmaf(d, d, s[0]);
            }
        };
#pragma unroll
        for (int i = 0; i < NCH; ++i)
            if (t + i * RT < nch) square(t + i * RT, held[i]);
        for (int c = t + NCH * RT; c < nch; c += RT) square(c, load(c));
        row_sums<RT>(s, red, turn);
        const float rstd = 1.0f / __builtin_sqrtf(s[0] / (float)n + a.eps);
        if (a.mean && t == 0) a.mean[row] = mean, a.rstd[row] = rstd;
        auto put = [&](int c, const Elems<T, E>& o, const Elems<W, E>& w, const Elems<W, E>& b) {
            float v[E];
#pragma unroll
            for (int e = 0; e < E; ++e)
                v[e] = __builtin_fmaf((to_f32(o.e[e]) - mean) * rstd, to_f32(w.e[e]), to_f32(b.e[e]));
            store_chunk<T>(y + row * a.ldy, c * E, n, pack<T>(v));
        };
#pragma unroll
        for (int i = 0; i < NCH; ++i)
            if (t + i * RT < nch) put(t + i * RT, held[i], hw[i], hb[i]);
        for (int c = t + NCH * RT; c < nch; c += RT) put(c, load(c), weights(c), biases(c));
    }
}

// grad_x, and the sums of dw and db where a.part is there (then every chunk of a row is held:
// nch <= NCH RT).
//   grid.x: any number of workgroups up to ceil(rows / row groups a workgroup); row group
//   blockIdx.x * (row groups a workgroup) + threadIdx.x / RT writes its part, of zeros where
//   it had no row
template <typename T, typename W, int RT, int NCH>
__global__ void __launch_bounds__(norm_threads(RT))
layer_norm_grad(NormGradArgs a)
{
    constexpr int E = 16 / (int)sizeof(T), PER = norm_threads(RT) / RT;
    __shared__ float red[2][2][16];
    const int t = threadIdx.x % RT, n = a.cols, nch = (n + E - 1) / E;
    const T* x = static_cast<const T*>(a.x);
    const T* gy = static_cast<const T*>(a.grad_y);
    T* gx = static_cast<T*>(a.grad_x);
    const W* weight = static_cast<const W*>(a.weight);
    const bool want_w = a.part != nullptr;
    Elems<W, E> hw[NCH];
    auto weights = [&](int c) { return load_elems<W, E>(weight, c * E, weight ? n : 0, (W)1.0f); };
    float dw[NCH][E] = {}, db[NCH][E] = {};
#pragma unroll
    for (int i = 0; i < NCH; ++i)
        if (t + i * RT < nch) hw[i] = weights(t + i * RT);
    int turn = 0;
    for (int64_t row = (int64_t)blockIdx.x * PER + threadIdx.x / RT; row < a.rows; row += (int64_t)gridDim.x * PER) {
        const T* xr = x + row * a.ldx;
        const T* gr = gy + row * a.ldgy;
        const float mean = a.mean[row], rstd = a.rstd[row];
        Elems<T, E> hx[NCH], hg[NCH];
        auto load_x = [&](int c) { return load_elems<T, E>(xr, c * E, n, (T)0.0f); };
        auto load_g = [&](int c) { return load_elems<T, E>(gr, c * E, n, (T)0.0f); };
#pragma unroll
        for (int i = 0; i < NCH; ++i)
            if (t + i * RT < nch) hx[i] = load_x(t + i * RT), hg[i] = load_g(t + i * RT);
        float s[2] = {0.0f, 0.0f};
        // an element past the row's end has g = 0, and x = 0 as any finite x
        auto add = [&](const Elems<T, E>& ox, const Elems<T, E>& og, const Elems<W, E>& w) {
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float xh = (to_f32(ox.e[e]) - mean) * rstd, gw = to_f32(og.e[e]) * to_f32(w.e[e]);
                s[0] += gw;
                s[1] = __builtin_fmaf(gw, xh, s[1]);
            }
        };
#pragma unroll
        for (int i = 0; i < NCH; ++i)
            if (t + i * RT < nch) {
                add(hx[i], hg[i], hw[i]);
                if (want_w)
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        const float g = to_f32(hg[i].e[e]);
                        dw[i][e] = __builtin_fmaf(g, (to_f32(hx[i].e[e]) - mean) * rstd, dw[i][e]);
                        db[i][e] += g;
                    }
            }
        if (!gx) continue;
        for (int c = t + NCH * RT; c < nch; c += RT) add(load_x(c), load_g(c), weights(c));
        row_sums<RT>(s, red, turn);
        const float m1 = s[0] / (float)n, m2 = s[1] / (float)n;
        auto put = [&](int c, const Elems<T, E>& ox, const Elems<T, E>& og, const Elems<W, E>& w) {
            float v[E];
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float xh = (to_f32(ox.e[e]) - mean) * rstd, gw = to_f32(og.e[e]) * to_f32(w.e[e]);
                v[e] = rstd * (gw - __builtin_fmaf(xh, m2, m1));
            }
            store_chunk<T>(gx + row * a.ldgx, c * E, n, pack<T>(v));
        };
#pragma unroll
        for (int i = 0; i < NCH; ++i)
            if (t + i * RT < nch) put(t + i * RT, hx[i], hg[i], hw[i]);
        for (int c = t + NCH * RT; c < nch; c += RT) put(c, load_x(c), load_g(c), weights(c));
    }
    if (!want_w) return;
    float* p = a.part + ((int64_t)blockIdx.x * PER + threadIdx.x / RT) * 2 * a.part_pitch;
#pragma unroll
    for (int i = 0; i < NCH; ++i)
        if (t + i * RT < nch) {
            const int at = (t + i * RT) * E;              // part rows hold whole chunks
#pragma unroll
            for (int e = 0; e < E; e += 4) {
                *reinterpret_cast<f32x4*>(p + at + e) = f32x4{dw[i][e], dw[i][e + 1], dw[i][e + 2], dw[i][e + 3]};
                *reinterpret_cast<f32x4*>(p + a.part_pitch + at + e) = f32x4{db[i][e], db[i][e + 1], db[i][e + 2], db[i][e + 3]};
            }
        }
}

// Sums of dw and db over the rows of one share, for rows too long to be held: a workgroup
// takes 32 chunks of columns, its 8 groups of 32 threads the rows r, r + 8, ... of the share.
//   grid = (ceil(chunks / 32), shares), block = 256
template <typename T>
__global__ void __launch_bounds__(256)
norm_column_sums(NormGradArgs a, int64_t share_rows)
{
    constexpr int E = 16 / (int)sizeof(T);
    __shared__ float red[8][32][2 * E + 1];
    const int r = threadIdx.x >> 5, t = threadIdx.x & 31;
    const int c = blockIdx.x * 32 + t, n = a.cols;
    const int64_t first = blockIdx.y * share_rows;
    const int64_t last = first + share_rows < a.rows ? first + share_rows : a.rows;
    float s[2 * E] = {};
    if (c * E < n)
        for (int64_t row = first + r; row < last; row += 8) {
            const Elems<T, E> ox = load_elems<T, E>(static_cast<const T*>(a.x) + row * a.ldx, c * E, n, (T)0.0f);
            const Elems<T, E> og = load_elems<T, E>(static_cast<const T*>(a.grad_y) + row * a.ldgy, c * E, n, (T)0.0f);
            const float mean = a.mean[row], rstd = a.rstd[row];
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float g = to_f32(og.e[e]);
                s[e] = __builtin_fmaf(g, (to_f32(ox.e[e]) - mean) * rstd, s[e]);
                s[E + e] += g;
            }
        }
#pragma unroll
    for (int e = 0; e < 2 * E; ++e) red[r][t][e] = s[e];
    __syncthreads();
    // thread (r, t): of the 2 E sums of chunk t the ones r, r + 8
#pragma unroll
    for (int e = r; e < 2 * E; e += 8) {
        float v = 0.0f;
#pragma unroll
        for (int k = 0; k < 8; ++k) v += red[k][t][e];
        if (c * E < n) a.part[((int64_t)blockIdx.y * 2 + e / E) * a.part_pitch + c * E + e % E] = v;
    }
}

// The row groups' sums added in order: four columns of dw (blockIdx.y = 0) or db (1) a
// thread, in 16 runs of the groups side by side.
//   part [groups][2][part_pitch]; grid = (ceil(cols / 64), 2), block = 256
template <typename W>
__global__ void __launch_bounds__(256)
join_norm_sums(const float* __restrict__ part, int groups, int part_pitch, int cols, W* __restrict__ dw, W* __restrict__ db)
{
    __shared__ f32x4 red[16][16];
    const int run = threadIdx.x >> 4, t = threadIdx.x & 15, col = (blockIdx.x * 16 + t) * 4;
    W* out = blockIdx.y ? db : dw;
    if (!out) return;
    f32x4 s = {0.0f, 0.0f, 0.0f, 0.0f};
    const int per = (groups + 15) / 16, first = run * per, last = first + per < groups ? first + per : groups;
    if (col < cols)
        for (int g = first; g < last; ++g)
            s += *reinterpret_cast<const f32x4*>(part + ((int64_t)g * 2 + blockIdx.y) * part_pitch + col);
    red[run][t] = s;
    __syncthreads();
    if (run != 0 || col >= cols) return;
#pragma unroll
    for (int k = 1; k < 16; ++k) s += red[k][t];
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (col + e < cols) out[col + e] = from_f32<W>(s[e]);
}

}  // namespace qtcq
