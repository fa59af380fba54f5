// distill.hpp -- divergence of a model's distribution over the vocabulary from a teacher's,
// given by its top logits, and its gradient with respect to the model's logits, gfx950.
//
// For a token with logits z [V], the teacher's logits t_j of the vocabulary entries i_j,
// j = 1 .. k, and the temperature tau:
//   q = softmax(z / tau),  p_j = exp(t_j / tau) / (the sum of them, or a sum the caller gives),
//   loss = sum_j p_j (log p_j - log q[i_j]),
//   dloss/dz = ((sum_j p_j) q - sum_j p_j e[i_j]) / tau.
// Entries with an index outside 0 .. V - 1 are padding.  An entry with p_j = 0 adds nothing,
// whatever q is there; a token without entries has loss 0 and gradient 0, whatever its logits
// are.  The same index twice: both entries count.
//
// The work is reading the logits (V a token, some 10^5) and writing their gradient, so a
// thread keeps a running maximum m and the sum s of exp((z - m) / tau), and the row is read
// once for the loss.  (z - m) is formed first: neither a row of very low values (a masked
// vocabulary) nor a large maximum costs digits.  A workgroup takes a row, and with the
// gradient wanted in the same call reads it again at once, while the caches still hold it;
// with few rows several workgroups share one (distill_partial, distill_join, distill_grad).
// The k entries' own arithmetic is in binary64.
//
// stats [rows][kDistillStats]: m, log s, the same two of the teacher, and sum p.
#pragma once

#include "dense.hpp"
#include "norm.hpp"
#include "reduce.hpp"

namespace qtcq {

constexpr int kDistillMaxK = 1024;
constexpr int kDistillStats = 5;

struct DistillArgs {
    const void* logits;
    int64_t rows, ldl;
    int vocab;
    const void* index;       // [rows][k] int32, or int64 where wide
    int64_t ldi;
    bool wide;
    const void* teacher;     // [rows][k]
    int64_t ldt;
    int teacher_type;        // qtcq_dtype: float32, bfloat16, float16
    int k;
    float tau;
    const float* teacher_log_z;  // [rows], or NULL: the sum over the entries
    float* loss;             // [rows]
    float* stats;            // [rows][kDistillStats], or NULL
    const float* grad_loss;  // [rows]
    void* grad;              // [rows][vocab], or NULL
    int64_t ldg;
    float* part;             // [rows][segments][2]: m and s of each segment
    int segments, segment;   // a row's segments and their length
};

struct RowStats { float m, ls, tm, tls, mass; };

constexpr float kLog2e = 1.4426950408889634f;

// where a maximum of -infinity is subtracted (a row without anything finite): 0
__device__ __forceinline__ float finite_ref(float m) { return m == -__builtin_inff() ? 0.0f : m; }

// LDS of a workgroup that finishes rows
struct DistillShared {
    float red[2][16];
    double sum[16];
    int index[kDistillMaxK];
    float p[kDistillMaxK];
};

__device__ __forceinline__ double wave_sum(double v)
{
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
    return v;
}

__device__ __forceinline__ float wave_max_f32(float v)
{
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v = __builtin_fmaxf(v, __shfl_xor(v, o, 64));
    return v;
}

// over the workgroup's NT threads, the same in all of them; LDS is free again on return
template <int NT>
__device__ __forceinline__ float block_max(float v, float (&red)[16])
{
    v = wave_max_f32(v);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < NT / 64; ++w) v = __builtin_fmaxf(v, red[w]);
    __syncthreads();
    return v;
}
template <int NT, typename F>
__device__ __forceinline__ F block_sum(F v, F* red)
{
    v = wave_sum(v);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0;
#pragma unroll
    for (int w = 0; w < NT / 64; ++w) v += red[w];
    __syncthreads();
    return v;
}

// The running maximum m and sum s of elements lo .. hi - 1 of a row, of the whole workgroup.
template <typename T, int NT>
__device__ __forceinline__ void softmax_sums(const T* row, int lo, int hi, float k2, DistillShared& sh, float& m, float& s)
{
    constexpr int E = 16 / (int)sizeof(T), U = 4;
    m = -__builtin_inff();
    s = 0.0f;
    for (int at = lo + (int)threadIdx.x * E; at < hi; at += U * NT * E) {
        Elems<T, E> v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = at + u * NT * E;
            v[u] = load_elems<T, E>(row, c < hi ? c : hi, hi, (T)-__builtin_inff());
        }
        float top = m;
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int e = 0; e < E; ++e) top = __builtin_fmaxf(top, to_f32(v[u].e[e]));
        const float ref = finite_ref(top);
        s *= __builtin_amdgcn_exp2f((m - ref) * k2);
        m = top;
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int e = 0; e < E; ++e) s += __builtin_amdgcn_exp2f((to_f32(v[u].e[e]) - ref) * k2);
    }
    const float all = block_max<NT>(m, sh.red[0]);
    s = block_sum<NT>(s * __builtin_amdgcn_exp2f((m - finite_ref(all)) * k2), sh.red[1]);
    m = all;
}

__device__ __forceinline__ float teacher_at(const DistillArgs& a, int64_t row, int j)
{
    const int64_t at = row * a.ldt + j;
    if (a.teacher_type == 1) return to_f32(static_cast<const __bf16*>(a.teacher)[at]);
    if (a.teacher_type == 2) return to_f32(static_cast<const _Float16*>(a.teacher)[at]);
    return static_cast<const float*>(a.teacher)[at];
}

// an entry's index, -1 where it is padding
__device__ __forceinline__ int index_at(const DistillArgs& a, int64_t row, int j)
{
    const int64_t at = row * a.ldi + j;
    const int64_t v = a.wide ? static_cast<const int64_t*>(a.index)[at] : static_cast<const int32_t*>(a.index)[at];
    return v >= 0 && v < a.vocab ? (int)v : -1;
}

// From a row's maximum and sum: its loss, and its statistics.
template <typename T, int NT>
__device__ __forceinline__ RowStats finish_row(const DistillArgs& a, int64_t row, float m, float s, DistillShared& sh)
{
    const T* z = static_cast<const T*>(a.logits) + row * a.ldl;
    const double inv = 1.0 / (double)a.tau;
    const double ls = log((double)s);
    const double ref = (double)finite_ref(m);
    // the teacher's maximum and sum, or those that the given sum stands for
    float tm = 0.0f;
    double tls = 0.0;
    if (a.teacher_log_z) {
        tls = (double)a.teacher_log_z[row];
    } else {
        tm = -__builtin_inff();
        for (int j = threadIdx.x; j < a.k; j += NT)
            if (index_at(a, row, j) >= 0) tm = __builtin_fmaxf(tm, teacher_at(a, row, j));
        tm = finite_ref(block_max<NT>(tm, sh.red[0]));
        double e = 0.0;
        for (int j = threadIdx.x; j < a.k; j += NT)
            if (index_at(a, row, j) >= 0) e += exp(((double)teacher_at(a, row, j) - (double)tm) * inv);
        tls = log(block_sum<NT>(e, sh.sum));
    }
    double loss = 0.0, mass = 0.0;
    for (int j = threadIdx.x; j < a.k; j += NT) {
        const int i = index_at(a, row, j);
        if (i < 0) continue;
        const double t = ((double)teacher_at(a, row, j) - (double)tm) * inv;
        // log p; nothing has a share where the sum is 0
        const double lp = t - tls, p = t == -__builtin_inf() ? 0.0 : exp(lp);
        mass += p;
        if (p != 0.0) loss += p * (lp - (((double)to_f32(z[i]) - ref) * inv - ls));
    }
    loss = block_sum<NT>(loss, sh.sum);
    mass = block_sum<NT>(mass, sh.sum);
    if (!a.teacher_log_z && mass > 0.0) mass = 1.0;
    const RowStats r = {m, (float)ls, tm, (float)tls, (float)mass};
    if (threadIdx.x == 0) {
        a.loss[row] = (float)loss;
        if (a.stats) {
            float* o = a.stats + row * kDistillStats;
            o[0] = r.m, o[1] = r.ls, o[2] = r.tm, o[3] = r.tls, o[4] = r.mass;
        }
    }
    return r;
}

// The gradient of elements lo .. hi - 1 of a row: first as if no entry were there, then the
// entries' elements again.  An index that comes up more than once is written by its first
// entry, with all of their p in order.
template <typename T, int NT>
__device__ __forceinline__ void gradient(const DistillArgs& a, int64_t row, int lo, int hi, const RowStats& r,
                                         DistillShared& sh)
{
    constexpr int E = 16 / (int)sizeof(T), U = 2;
    const T* z = static_cast<const T*>(a.logits) + row * a.ldl;
    T* g = static_cast<T*>(a.grad) + row * a.ldg;
    const float k2 = kLog2e / a.tau, ref = finite_ref(r.m), ls2 = r.ls * kLog2e;
    const float scale = a.grad_loss[row] / a.tau, coef = scale * r.mass;
    const bool none = r.mass == 0.0f;
    for (int j = threadIdx.x; j < a.k; j += NT) {
        const int i = index_at(a, row, j);
        sh.index[j] = i;
        sh.p[j] = i >= 0 ? __builtin_amdgcn_exp2f((teacher_at(a, row, j) - r.tm) * k2 - r.tls * kLog2e) : 0.0f;
    }
    auto q = [&](float x) { return none ? 0.0f : coef * __builtin_amdgcn_exp2f(__builtin_fmaf(x - ref, k2, -ls2)); };
    for (int at = lo + (int)threadIdx.x * E; at < hi; at += U * NT * E) {
        Elems<T, E> v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = at + u * NT * E;
            v[u] = load_elems<T, E>(z, c < hi ? c : hi, hi, (T)0.0f);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = at + u * NT * E;
            float o[E];
#pragma unroll
            for (int e = 0; e < E; ++e) o[e] = q(to_f32(v[u].e[e]));
            if (c < hi) store_elems<T, E>(g, c, hi, o);
        }
    }
    // the stores above are done before the entries' are issued, in every wave
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (!none)
        for (int j = threadIdx.x; j < a.k; j += NT) {
            const int i = sh.index[j];
            if (i < lo || i >= hi) continue;
            float p = 0.0f;
            bool first = true;
            for (int l = 0; l < a.k; ++l)
                if (sh.index[l] == i) {
                    first = first && l >= j;
                    p += sh.p[l];
                }
            if (first) g[i] = from_f32<T>(q(to_f32(z[i])) - scale * p);
        }
    __syncthreads();                                  // LDS is free for the next row
}

// A workgroup a row.  grid.x: any number of workgroups up to the rows
template <typename T, int NT, bool GRAD>
__global__ void __launch_bounds__(NT)
distill_rows(DistillArgs a)
{
    __shared__ DistillShared sh;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        float m, s;
        softmax_sums<T, NT>(static_cast<const T*>(a.logits) + row * a.ldl, 0, a.vocab, kLog2e / a.tau, sh, m, s);
        const RowStats r = finish_row<T, NT>(a, row, m, s, sh);
        if constexpr (GRAD) gradient<T, NT>(a, row, 0, a.vocab, r, sh);
    }
}

// A workgroup a segment of a row: its maximum and sum.  grid.x = rows * segments
template <typename T, int NT>
__global__ void __launch_bounds__(NT)
distill_partial(DistillArgs a)
{
    __shared__ DistillShared sh;
    const int64_t row = blockIdx.x / a.segments;
    const int lo = (int)(blockIdx.x - row * a.segments) * a.segment;
    const int hi = lo + a.segment < a.vocab ? lo + a.segment : a.vocab;
    float m, s;
    softmax_sums<T, NT>(static_cast<const T*>(a.logits) + row * a.ldl, lo, hi, kLog2e / a.tau, sh, m, s);
    if (threadIdx.x == 0) {
        a.part[blockIdx.x * 2] = m;
        a.part[blockIdx.x * 2 + 1] = s;
    }
}

// The segments of a row joined in order, and its loss.  grid.x = rows
template <typename T, int NT>
__global__ void __launch_bounds__(NT)
distill_join(DistillArgs a)
{
    __shared__ DistillShared sh;
    const int64_t row = blockIdx.x;
    const float* p = a.part + row * a.segments * 2;
    const float k2 = kLog2e / a.tau;
    float m = -__builtin_inff(), s = 0.0f;
    for (int i = 0; i < a.segments; ++i) m = __builtin_fmaxf(m, p[2 * i]);
    for (int i = 0; i < a.segments; ++i) s += p[2 * i + 1] * __builtin_amdgcn_exp2f((p[2 * i] - finite_ref(m)) * k2);
    finish_row<T, NT>(a, row, m, s, sh);
}

// A workgroup a segment of a row: its gradient.  Segment i of rows * segments, in turn
template <typename T, int NT>
__global__ void __launch_bounds__(NT)
distill_grad(DistillArgs a)
{
    __shared__ DistillShared sh;
    for (int64_t b = blockIdx.x; b < a.rows * a.segments; b += gridDim.x) {
        const int64_t row = b / a.segments;
        const int lo = (int)(b - row * a.segments) * a.segment;
        const int hi = lo + a.segment < a.vocab ? lo + a.segment : a.vocab;
        const float* s = a.stats + row * kDistillStats;
        gradient<T, NT>(a, row, lo, hi, RowStats{s[0], s[1], s[2], s[3], s[4]}, sh);
    }
}

}  // namespace qtcq
