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
// Both directions are bound by memory (x, g read once, y or dx written once), so a row's loads
// are issued before the work on the rows ahead of it.  RT threads a row, NCH 16-byte chunks
// a thread; a workgroup goes through its rows and keeps the weights of its columns, which all
// rows share, in registers.  So do the sums of dw and db: each group of RT threads adds
// its rows in order, a workgroup its groups, and join_norm_sums the workgroups.  No atomics:
// the same bits on every run.
//
// 8192x8192 bf16, calls in a row: forward 54 us (5.0 TB/s), gradients 83, of which 78 (5.2 TB/s) and
// 5 for the 256 workgroups' sums; 333x2731 float32 gradients in one launch 7.2 in the kernel.
// Without the next rows' loads ahead of the work the forward took 78, the gradients 128.
#pragma once

#include "model_args.hpp"
#include "reduce.hpp"
#include "rows.hpp"

namespace qtcq {

// Sums over the RT threads of a row of N values at once (a row group's threads lie together);
// red: [2][N][waves of the workgroup] in LDS, the two halves in turn, so that one barrier a
// call is enough.
template <int NT, int RT, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float (*red)[N][NT / 64], int& turn)
{
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
    if constexpr (RT > 64) {
        const int wave = threadIdx.x >> 6, first = wave & ~(RT / 64 - 1);
        if ((threadIdx.x & 63) == 0)
#pragma unroll
            for (int i = 0; i < N; ++i) red[turn][i][wave] = v[i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            v[i] = red[turn][i][first + (threadIdx.x & (RT / 64 - 1))];
#pragma unroll
            for (int o = RT / 128; o > 0; o >>= 1) v[i] += __shfl_xor(v[i], o, 64);
        }
        turn ^= 1;
    }
}

constexpr int norm_threads(int rt) { return rt < 256 ? 256 : rt; }

// One row a row group at a time, the next one on its way.  LONG: chunks beyond NCH RT are read
// anew by each pass.
//   grid.x: any number of workgroups up to ceil(rows / row groups a workgroup)
template <typename T, typename W, int RT, int NCH, bool LONG>
__global__ void __launch_bounds__(norm_threads(RT))
layer_norm_rows(NormArgs a)
{
    constexpr int E = 16 / (int)sizeof(T), NT = norm_threads(RT), PER = NT / RT;
    __shared__ float red[2][1][NT / 64];
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
    Place place[NCH];
#pragma unroll
    for (int i = 0; i < NCH; ++i) place[i] = place_of<T>(t + i * RT, n);
    const bool uneven = n % E != 0;
    const int64_t step = (int64_t)gridDim.x * PER;
    int64_t row = (int64_t)blockIdx.x * PER + threadIdx.x / RT;
    u32x4 next[NCH];
    auto load = [&](int64_t r, int c) { return load_zero<T>(x + r * a.ldx, c, n); };
    auto fetch = [&](int64_t r) {
        const T* xr = x + (r < a.rows ? r : a.rows - 1) * a.ldx;
        if (n < E) {
            next[0] = load_short(xr, n);
        } else {
#pragma unroll
            for (int i = 0; i < NCH; ++i) next[i] = load_loose(xr + place[i].at);
        }
    };
    fetch(row);
    int turn = 0;
    // row groups of a workgroup stay together, for the barriers
    for (; row - threadIdx.x / RT < a.rows; row += step) {
        const bool there = row < a.rows;
        u32x4 held[NCH];
#pragma unroll
        for (int i = 0; i < NCH; ++i) held[i] = uneven && n > E ? behind(next[i], place[i].bits) : next[i];
        if (row + step - threadIdx.x / RT < a.rows) fetch(row + step);
        float s[1] = {0.0f};
        auto add = [&](u32x4 o) {
            float v[E];
            unpack<T>(o, v);
#pragma unroll
            for (int e = 0; e < E; ++e) s[0] += v[e];
        };
#pragma unroll
        for (int i = 0; i < NCH; ++i)
            if (t + i * RT < nch) add(held[i]);
        if (LONG && there)
            for (int c = t + NCH * RT; c < nch; c += RT) add(load(row, c));
        row_sums<NT, RT>(s, red, turn);
        const float mean = s[0] / (float)n;
        s[0] = 0.0f;
        auto square = [&](int c, u32x4 o) {
            float v[E];
            unpack<T>(o, v);
            if ((c + 1) * E <= n) {
#pragma unroll
                for (int e = 0; e < E; ++e) s[0] = __builtin_fmaf(v[e] - mean, v[e] - mean, s[0]);
            } else {
#pragma unroll
                for (int e = 0; e < E; ++e)
                    if (c * E + e < n) s[0] = __builtin_fmaf(v[e] - mean, v[e] - mean, s[0]);
            }
        };
#pragma unroll
        for (int i = 0; i < NCH; ++i)
            if (t + i * RT < nch) square(t + i * RT, held[i]);
        if (LONG && there)
            for (int c = t + NCH * RT; c < nch; c += RT) square(c, load(row, c));
        row_sums<NT, RT>(s, red, turn);
        if (!there) continue;
        const float rstd = 1.0f / __builtin_sqrtf(s[0] / (float)n + a.eps);
        if (a.mean && t == 0) a.mean[row] = mean, a.rstd[row] = rstd;
        auto put = [&](int c, u32x4 o, const Elems<W, E>& w, const Elems<W, E>& b) {
            float v[E];
            unpack<T>(o, v);
#pragma unroll
            for (int e = 0; e < E; ++e) v[e] = __builtin_fmaf((v[e] - mean) * rstd, to_f32(w.e[e]), to_f32(b.e[e]));
            store_chunk<T>(y + row * a.ldy, c * E, n, pack<T>(v));
        };
#pragma unroll
        for (int i = 0; i < NCH; ++i)
            if (t + i * RT < nch) put(t + i * RT, held[i], hw[i], hb[i]);
        for (int c = t + NCH * RT; LONG && c < nch; c += RT) put(c, load(row, c), weights(c), biases(c));
    }
}

constexpr int kNormGradThreads = 1024;

// LDS of the gradient: of the sums over a row, and of those over row groups or rows
template <int R>
struct NormGradShared {
    float red[2][2 * R][kNormGradThreads / 64];
    float sums[16 * kNormGradThreads];
};

// grad_x, and the sums of dw and db where a.part is there (then every chunk of a row is held:
// nch <= NCH RT): R rows a row group at a time, the next ones on their way.  LONG: chunks
// beyond NCH RT are read anew by each pass.
//   workgroup `block` of `blocks`, of 1024 threads; each writes its part, of zeros where it had
//   no row
template <typename T, typename W, int RT, int NCH, int R, bool LONG>
__device__ __forceinline__ void norm_grad_rows(const NormGradArgs& a, unsigned block, unsigned blocks, NormGradShared<R>& sh)
{
    constexpr int E = 16 / (int)sizeof(T), NT = kNormGradThreads, PER = NT / RT;
    static_assert(PER == 1 || NCH == 1, "row groups are joined with one chunk a thread");
    const int t = threadIdx.x % RT, group = threadIdx.x / RT, n = a.cols, nch = (n + E - 1) / E;
    const T* x = static_cast<const T*>(a.x);
    const T* gy = static_cast<const T*>(a.grad_y);
    T* gx = static_cast<T*>(a.grad_x);
    const W* weight = static_cast<const W*>(a.weight);
    const bool want_w = a.part != nullptr;
    auto weights = [&](int c) { return load_elems<W, E>(weight, c * E, weight ? n : 0, (W)1.0f); };
    Elems<W, E> hw[NCH];
    float dw[NCH][E] = {}, db[NCH][E] = {};
#pragma unroll
    for (int i = 0; i < NCH; ++i)
        if (t + i * RT < nch) hw[i] = weights(t + i * RT);
    auto load_x = [&](int64_t r, int c) { return load_zero<T>(x + r * a.ldx, c, n); };
    auto load_g = [&](int64_t r, int c) { return load_zero<T>(gy + r * a.ldgy, c, n); };
    struct Rows { u32x4 x[R][NCH], g[R][NCH]; float mean[R], rstd[R]; };
    Place place[NCH];
#pragma unroll
    for (int i = 0; i < NCH; ++i) place[i] = place_of<T>(t + i * RT, n);
    const bool uneven = n % E != 0;
    // rows past the last are read as the last one
    auto fetch = [&](int64_t row, Rows& o) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int64_t at = row + r < a.rows ? row + r : a.rows - 1;
            o.mean[r] = a.mean[at];
            o.rstd[r] = a.rstd[at];
            if (n < E) {
                o.x[r][0] = load_short(x + at * a.ldx, n);
                o.g[r][0] = load_short(gy + at * a.ldgy, n);
                continue;
            }
#pragma unroll
            for (int i = 0; i < NCH; ++i) {
                o.x[r][i] = load_loose(x + at * a.ldx + place[i].at);
                o.g[r][i] = load_loose(gy + at * a.ldgy + place[i].at);
            }
        }
    };
    const int64_t step = (int64_t)blocks * PER * R;
    int64_t row = ((int64_t)block * PER + group) * R;
    Rows cur, next;
    fetch(row, next);
    int turn = 0;
    for (int64_t first = (int64_t)block * PER * R; first < a.rows; first += step, row += step) {
        cur = next;
        if (first + step < a.rows) fetch(row + step, next);
        // into place, and rows past the last to zeros
        if ((uneven && n > E) || first + PER * R > a.rows) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const bool there = row + r < a.rows;
                if (!there) cur.mean[r] = cur.rstd[r] = 0.0f;
#pragma unroll
                for (int i = 0; i < NCH; ++i) {
                    const int bits = !there ? 128 : (n > E ? place[i].bits : 0);
                    cur.x[r][i] = behind(cur.x[r][i], bits);
                    cur.g[r][i] = behind(cur.g[r][i], bits);
                }
            }
        }
        float s[2 * R] = {};
        // an element past the row's end has g = 0, and x = 0 as any finite x
        auto add = [&](int r, u32x4 ox, u32x4 og, const Elems<W, E>& w) {
            float xv[E], gv[E];
            unpack<T>(ox, xv);
            unpack<T>(og, gv);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float gw = gv[e] * to_f32(w.e[e]);
                s[2 * r] += gw;
                s[2 * r + 1] = __builtin_fmaf(gw, (xv[e] - cur.mean[r]) * cur.rstd[r], s[2 * r + 1]);
            }
        };
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int i = 0; i < NCH; ++i) {
                if (t + i * RT >= nch) continue;
                add(r, cur.x[r][i], cur.g[r][i], hw[i]);
                if (want_w) {
                    float xv[E], gv[E];
                    unpack<T>(cur.x[r][i], xv);
                    unpack<T>(cur.g[r][i], gv);
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        dw[i][e] = __builtin_fmaf(gv[e], (xv[e] - cur.mean[r]) * cur.rstd[r], dw[i][e]);
                        db[i][e] += gv[e];
                    }
                }
            }
        if (!gx) continue;
#pragma unroll
        for (int r = 0; r < R; ++r)
            if (LONG && row + r < a.rows)
                for (int c = t + NCH * RT; c < nch; c += RT) add(r, load_x(row + r, c), load_g(row + r, c), weights(c));
        row_sums<NT, RT>(s, sh.red, turn);
        // (the elements are taken from their chunks again: kept in binary32 over the sums, they
        // would not fit the registers)
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int i = 0; i < NCH; ++i) asm volatile("" : "+v"(cur.x[r][i]), "+v"(cur.g[r][i]));
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (row + r >= a.rows) continue;
            const float m1 = s[2 * r] / (float)n, m2 = s[2 * r + 1] / (float)n;
            auto put = [&](int c, u32x4 ox, u32x4 og, const Elems<W, E>& w) {
                float xv[E], gv[E];
                unpack<T>(ox, xv);
                unpack<T>(og, gv);
#pragma unroll
                for (int e = 0; e < E; ++e)
                    xv[e] = cur.rstd[r] * (gv[e] * to_f32(w.e[e]) - __builtin_fmaf((xv[e] - cur.mean[r]) * cur.rstd[r], m2, m1));
                store_chunk<T>(gx + (row + r) * a.ldgx, c * E, n, pack<T>(xv));
            };
#pragma unroll
            for (int i = 0; i < NCH; ++i)
                if (t + i * RT < nch) put(t + i * RT, cur.x[r][i], cur.g[r][i], hw[i]);
            for (int c = t + NCH * RT; LONG && c < nch; c += RT) put(c, load_x(row + r, c), load_g(row + r, c), weights(c));
        }
    }
    if (!want_w) return;
    float* p = a.part + (int64_t)block * 2 * a.part_pitch;
    if constexpr (PER == 1) {
#pragma unroll
        for (int i = 0; i < NCH; ++i)
            if (t + i * RT < nch) {
                const int at = (t + i * RT) * E;          // part rows hold whole chunks
#pragma unroll
                for (int e = 0; e < E; e += 4) {
                    *reinterpret_cast<f32x4*>(p + at + e) = f32x4{dw[i][e], dw[i][e + 1], dw[i][e + 2], dw[i][e + 3]};
                    *reinterpret_cast<f32x4*>(p + a.part_pitch + at + e) =
                        f32x4{db[i][e], db[i][e + 1], db[i][e + 2], db[i][e + 3]};
                }
            }
    } else {
        // the row groups' sums in order: group g adds up sums g, g + PER, ... of its chunk
#pragma unroll
        for (int e = 0; e < E; ++e) {
            sh.sums[e * NT + threadIdx.x] = dw[0][e];
            sh.sums[(E + e) * NT + threadIdx.x] = db[0][e];
        }
        __syncthreads();
        for (int e = group; e < 2 * E; e += PER) {
            float v = 0.0f;
#pragma unroll
            for (int k = 0; k < PER; ++k) v += sh.sums[e * NT + k * RT + t];
            if (t < nch) p[(e < E ? 0 : a.part_pitch) + t * E + e % E] = v;
        }
    }
}

// grid.x: any number of workgroups
template <typename T, typename W, int RT, int NCH, int R, bool LONG>
__global__ void __launch_bounds__(kNormGradThreads)
layer_norm_grad(NormGradArgs a)
{
    __shared__ NormGradShared<R> sh;
    norm_grad_rows<T, W, RT, NCH, R, LONG>(a, blockIdx.x, gridDim.x, sh);
}

// Few rows, in one launch: workgroups 0 .. nx - 1 write grad_x, and each of the others takes 8
// chunks of columns over all rows, which it reads again, 512 rows at a time, and writes their
// weights' gradients.
//   grid.x = nx + ceil(chunks / 8) (nx alone where no weight's gradient is wanted)
constexpr int kNormFewChunks = 8;
template <typename T, typename W, int RT, int NCH, int R>
__global__ void __launch_bounds__(kNormGradThreads)
layer_norm_grad_few(NormGradArgs a, W* __restrict__ dw, W* __restrict__ db, int nx)
{
    __shared__ NormGradShared<R> sh;
    if ((int)blockIdx.x < nx) {
        norm_grad_rows<T, W, RT, NCH, R, false>(a, blockIdx.x, nx, sh);
        return;
    }
    constexpr int E = 16 / (int)sizeof(T), U = 4, CW = kNormFewChunks, ROWS = kNormGradThreads / CW;
    const int r = threadIdx.x / CW, t = threadIdx.x % CW, n = a.cols;
    const int c = ((int)blockIdx.x - nx) * CW + t;
    const T* x = static_cast<const T*>(a.x);
    const T* gy = static_cast<const T*>(a.grad_y);
    float s[2 * E] = {};
    if (c * E < n)
        for (int64_t row = r; row < a.rows; row += U * ROWS) {
            u32x4 xv[U], gv[U];
            float mean[U], rstd[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                // (rows past the last are read as it, and left out below)
                const int64_t at = row + u * ROWS < a.rows ? row + u * ROWS : a.rows - 1;
                xv[u] = load_zero<T>(x + at * a.ldx, c, n);
                gv[u] = load_zero<T>(gy + at * a.ldgy, c, n);
                mean[u] = a.mean[at];
                rstd[u] = a.rstd[at];
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (row + u * ROWS >= a.rows) continue;
                float xf[E], gf[E];
                unpack<T>(xv[u], xf);
                unpack<T>(gv[u], gf);
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    s[e] = __builtin_fmaf(gf[e], (xf[e] - mean[u]) * rstd[u], s[e]);
                    s[E + e] += gf[e];
                }
            }
        }
#pragma unroll
    for (int e = 0; e < 2 * E; ++e) sh.sums[e * kNormGradThreads + threadIdx.x] = s[e];
    __syncthreads();
    // sum e of chunk q over the rows' threads: LANES lanes, four runs each, and then by twos (float32
    // 333x2731 within 0.9e-7 of the norm; in four runs of 32 it was 1.3e-7)
    constexpr int LANES = kNormGradThreads / (2 * E * CW);
    const int lane = threadIdx.x % LANES, e = threadIdx.x / LANES / CW, q = threadIdx.x / LANES % CW;
    f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < ROWS; k += 4 * LANES)
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] += sh.sums[e * kNormGradThreads + (k + i * LANES + lane) * CW + q];
    float sum = (v.x + v.y) + (v.z + v.w);
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) sum += __shfl_xor(sum, o, 64);
    const int at = (((int)blockIdx.x - nx) * CW + q) * E + e % E;
    W* out = e < E ? dw : db;
    if (lane == 0 && at < n && out) out[at] = from_f32<W>(sum);
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
            float xv[E], gv[E];
            unpack<T>(load_zero<T>(static_cast<const T*>(a.x) + row * a.ldx, c, n), xv);
            unpack<T>(load_zero<T>(static_cast<const T*>(a.grad_y) + row * a.ldgy, c, n), gv);
            const float mean = a.mean[row], rstd = a.rstd[row];
#pragma unroll
            for (int e = 0; e < E; ++e) {
                s[e] = __builtin_fmaf(gv[e], (xv[e] - mean) * rstd, s[e]);
                s[E + e] += gv[e];
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
// thread, in 32 runs of the groups side by side, 8 loads of each on their way at once (256
// groups of 8192 columns 4.9 us, 7.5 in 16 runs with one load at a time).
//   part [groups][2][part_pitch]; grid = (ceil(cols / 32), 2), block = 256
template <typename W>
__global__ void __launch_bounds__(256)
join_norm_sums(const float* __restrict__ part, int groups, int part_pitch, int cols, W* __restrict__ dw, W* __restrict__ db)
{
    constexpr int RUNS = 32, T = 256 / RUNS, U = 8;
    __shared__ f32x4 red[RUNS][T];
    const int run = threadIdx.x / T, t = threadIdx.x % T, col = (blockIdx.x * T + t) * 4;
    W* out = blockIdx.y ? db : dw;
    if (!out) return;
    const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
    f32x4 s = zero;
    const int per = (groups + RUNS - 1) / RUNS, first = run * per, last = first + per < groups ? first + per : groups;
    if (col < cols)
        for (int g = first; g < last; g += U) {
            f32x4 v[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                v[u] = g + u < last ? *reinterpret_cast<const f32x4*>(part + ((int64_t)(g + u) * 2 + blockIdx.y) * part_pitch + col) : zero;
#pragma unroll
            for (int u = 0; u < U; ++u) s += v[u];
        }
    red[run][t] = s;
    __syncthreads();
    if (run != 0 || col >= cols) return;
#pragma unroll
    for (int k = 1; k < RUNS; ++k) s += red[k][t];
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (col + e < cols) out[col + e] = from_f32<W>(s[e]);
}

}  // namespace qtcq
