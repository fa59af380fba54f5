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
// The k entries' own sums are in binary64.
//
// stats [rows][kDistillStats]: m, log2 s, the same two of the teacher, and sum p.
#pragma once

#include "model_args.hpp"
#include "reduce.hpp"
#include "rows.hpp"

namespace qtcq {

struct RowStats { float m, ls, tm, tls, mass; };

constexpr float kLog2e = 1.4426950408889634f;

// where a maximum of -infinity is subtracted (a row without anything finite): 0
__device__ __forceinline__ float finite_ref(float m) { return m == -__builtin_inff() ? 0.0f : m; }

// LDS of a workgroup: reductions, and the row's entries (dynamic, 16 bytes each)
struct DistillShared {
    float red[2][16];
    double sum[2][16];
};
struct Entry { int index; float t, z, p; };     // p: for the gradient
extern __shared__ __align__(16) char distill_entries[];

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
    if constexpr (NT > 64) {
        if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
        __syncthreads();
        v = red[threadIdx.x & (NT / 64 - 1)];
#pragma unroll
        for (int o = NT / 128; o > 0; o >>= 1) v = __builtin_fmaxf(v, __shfl_xor(v, o, 64));
        __syncthreads();
    }
    return v;
}
template <int NT, typename F>
__device__ __forceinline__ F block_sum(F v, F* red)
{
    v = wave_sum(v);
    if constexpr (NT > 64) {
        if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
        __syncthreads();
        v = red[threadIdx.x & (NT / 64 - 1)];
#pragma unroll
        for (int o = NT / 128; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
        __syncthreads();
    }
    return v;
}

// The chunks of 16 bytes of a row's elements lo .. hi - 1, two at a time: f(v, c, whole) for
// chunks c and c + NT of the thread, of which those below `whole` are there (`fill` elsewhere),
// with the next two on their way.  The elements behind the last whole chunk are the last
// thread's, which takes them last: f(v, whole, 0) with them in v[0].
template <typename T, int NT, typename F>
__device__ __forceinline__ void each_pair(const T* row, int lo, int hi, T fill, F&& f)
{
    constexpr int E = 16 / (int)sizeof(T);
    const T* z = row + lo;
    const int whole = (hi - lo) / E, t = threadIdx.x;
    const u32x4 none = __builtin_bit_cast(u32x4, load_filled<T>(row, 0, 0, fill));
    u32x4 v[2];
    int c = t, left = whole;                           // whole chunks from the workgroup's first on
    if (left >= 2 * NT) {
        v[0] = load_loose(z + c * E);
        v[1] = load_loose(z + (c + NT) * E);
        for (; left >= 4 * NT; left -= 2 * NT, c += 2 * NT) {
            const u32x4 next[2] = {load_loose(z + (c + 2 * NT) * E), load_loose(z + (c + 3 * NT) * E)};
            f(v, c, whole);
            v[0] = next[0];
            v[1] = next[1];
        }
        f(v, c, whole);
        left -= 2 * NT, c += 2 * NT;
    }
    if (left > 0) {
        v[0] = c < whole ? load_loose(z + c * E) : none;
        v[1] = c + NT < whole ? load_loose(z + (c + NT) * E) : none;
        f(v, c, whole);
    }
    if (t == NT - 1 && whole * E < hi - lo) {
        v[0] = load_filled<T>(z, whole * E, hi - lo, fill);
        v[1] = none;
        f(v, whole, 0);
    }
}

// Two chunks into the running maximum m and sum s of a thread.  One of -infinities changes
// no bit of them.
template <typename T>
__device__ __forceinline__ void take_pair(const u32x4* v, float k2, float& m, float& s)
{
    constexpr int E = 16 / (int)sizeof(T);
    float x[2][E], top = m;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        unpack<T>(v[u], x[u]);
#pragma unroll
        for (int e = 0; e < E; ++e) top = __builtin_fmaxf(top, x[u][e]);
    }
    const float ref = finite_ref(top);
    float sum[2] = {s * __builtin_amdgcn_exp2f((m - ref) * k2), 0.0f};
    m = top;
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int e = 0; e < E; ++e) sum[e & 1] += __builtin_amdgcn_exp2f((x[u][e] - ref) * k2);
    s = sum[0] + sum[1];
}

// The threads' maxima and sums joined, the same in all of the workgroup.
template <int NT>
__device__ __forceinline__ void join_threads(float k2, DistillShared& sh, float& m, float& s)
{
    const float all = block_max<NT>(m, sh.red[0]);
    s = block_sum<NT>(s * __builtin_amdgcn_exp2f((m - finite_ref(all)) * k2), sh.red[1]);
    m = all;
}

// The running maximum m and sum s of elements lo .. hi - 1 of a row, of the whole workgroup.
template <typename T, int NT>
__device__ __forceinline__ void softmax_sums(const T* row, int lo, int hi, float k2, DistillShared& sh, float& m, float& s)
{
    m = -__builtin_inff();
    s = 0.0f;
    each_pair<T, NT>(row, lo, hi, (T)-__builtin_inff(), [&](const u32x4* v, int, int) { take_pair<T>(v, k2, m, s); });
    join_threads<NT>(k2, sh, m, s);
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

// A row's entries to LDS, with the logits at them; thread t has the entries t, t + NT, ... from
// here to their last use but for the search for repeated indices.
template <typename T, int NT>
__device__ __forceinline__ void load_entries(const DistillArgs& a, int64_t row)
{
    Entry* en = reinterpret_cast<Entry*>(distill_entries);
    for (int j = threadIdx.x; j < a.k; j += NT) {
        const int i = index_at(a, row, j);
        const float t = teacher_at(a, row, j);
        en[j] = Entry{i, t, i >= 0 ? to_f32(static_cast<const T*>(a.logits)[row * a.ldl + i]) : 0.0f, 0.0f};
    }
}

// log2 of a sum that is 1 or more (or 0, infinite or NaN): the exponent, and the logarithm of
// the mantissa, whose error is then 2^-24 and not that of a number above 16.
__device__ __forceinline__ double log2_of(float s)
{
    if (!(s >= 1.0f && s < __builtin_inff())) return (double)__builtin_amdgcn_logf(s);
    const uint32_t b = __builtin_bit_cast(uint32_t, s);
    return (double)((int)(b >> 23) - 127) + (double)__builtin_amdgcn_logf(__builtin_bit_cast(float, (b & 0x7FFFFFu) | 0x3F800000u));
}

// 2^v: the hardware's exp2 takes the part behind the point
__device__ __forceinline__ float exp2_of(double v)
{
    if (!(v > -160.0)) return v == v ? 0.0f : (float)v;
    const double n = rint(v);
    return __builtin_ldexpf(__builtin_amdgcn_exp2f((float)(v - n)), (int)n);
}

// From a row's maximum and sum: its loss, and its statistics.
template <int NT>
__device__ __forceinline__ RowStats finish_row(const DistillArgs& a, int64_t row, float m, float s, DistillShared& sh)
{
    const Entry* en = reinterpret_cast<const Entry*>(distill_entries);
    const double k2 = 1.4426950408889634 / (double)a.tau;
    const double ls = log2_of(s);
    const double ref = (double)finite_ref(m);
    // the teacher's maximum and sum, or those that the given sum stands for
    float tm = 0.0f;
    double tls = 0.0;
    if (a.teacher_log_z) {
        tls = (double)a.teacher_log_z[row] * 1.4426950408889634;
    } else {
        tm = -__builtin_inff();
        for (int j = threadIdx.x; j < a.k; j += NT)
            if (en[j].index >= 0) tm = __builtin_fmaxf(tm, en[j].t);
        tm = finite_ref(block_max<NT>(tm, sh.red[0]));
        double e = 0.0;
        for (int j = threadIdx.x; j < a.k; j += NT)
            if (en[j].index >= 0) e += (double)exp2_of(((double)en[j].t - (double)tm) * k2);
        tls = log2_of((float)block_sum<NT>(e, sh.sum[0]));
    }
    double loss = 0.0, mass = 0.0;
    for (int j = threadIdx.x; j < a.k; j += NT) {
        if (en[j].index < 0) continue;
        const double t = ((double)en[j].t - (double)tm) * k2;
        // log p; nothing has a share where the sum is 0
        const double lp = t - tls, p = t == -__builtin_inf() ? 0.0 : (double)exp2_of(lp);
        mass += p;
        if (p != 0.0) loss += p * (lp - (((double)en[j].z - ref) * k2 - ls));
    }
    loss = block_sum<NT>(loss, sh.sum[0]) * 0.6931471805599453;
    mass = block_sum<NT>(mass, sh.sum[1]);
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

// The gradient of a row's elements as if no entry were there (q), and the entries' elements.
template <typename T>
struct RowGradient {
    static constexpr int E = 16 / (int)sizeof(T);
    T* g;
    float k2, ref, ls, scale, coef;
    bool none;

    __device__ __forceinline__ RowGradient(const DistillArgs& a, int64_t row, const RowStats& r)
        : g(static_cast<T*>(a.grad) + row * a.ldg), k2(kLog2e / a.tau), ref(finite_ref(r.m)), ls(r.ls),
          scale(a.grad_loss[row] / a.tau), coef(scale * r.mass), none(r.mass == 0.0f) {}
    __device__ __forceinline__ float q(float x) const
    {
        return coef * __builtin_amdgcn_exp2f(__builtin_fmaf(x - ref, k2, -ls));
    }
    __device__ __forceinline__ u32x4 chunk(u32x4 v) const
    {
        float x[E];
        unpack<T>(v, x);
#pragma unroll
        for (int e = 0; e < E; ++e) x[e] = q(x[e]);
        return none ? u32x4{0u, 0u, 0u, 0u} : pack<T>(x);
    }
    // The elements lo .. hi - 1 that entries are at, once all others are written.  An index that
    // comes up more than once is written by its first entry, with all of their p in order.
    template <int NT>
    __device__ __forceinline__ void entries(int k, int lo, int hi) const
    {
        // the chunks' stores are done before the entries' are issued, in every wave
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
        const Entry* en = reinterpret_cast<const Entry*>(distill_entries);
        if (!none)
            for (int j = threadIdx.x; j < k; j += NT) {
                const int i = en[j].index;
                if (i < lo || i >= hi) continue;
                float p = 0.0f;
                bool first = true;
                for (int l = 0; l < k; ++l)
                    if (en[l].index == i) {
                        first = first && l >= j;
                        p += en[l].p;
                    }
                if (first) g[i] = from_f32<T>(q(en[j].z) - scale * p);
            }
        __syncthreads();                              // LDS is free for the next row
    }
};

// p of a row's entries, as their gradients take it
template <int NT>
__device__ __forceinline__ void entry_shares(const DistillArgs& a, const RowStats& r)
{
    Entry* en = reinterpret_cast<Entry*>(distill_entries);
    for (int j = threadIdx.x; j < a.k; j += NT)
        en[j].p = en[j].index >= 0 ? __builtin_amdgcn_exp2f((en[j].t - r.tm) * (kLog2e / a.tau) - r.tls) : 0.0f;
}

// A workgroup a row, for the loss.  grid.x: any number of workgroups up to the rows
// (eight waves a SIMD: 64 registers, so that two rows of 1024 threads run on a compute unit)
template <typename T, int NT>
__global__ void __launch_bounds__(NT, 8)
distill_rows(DistillArgs a)
{
    __shared__ DistillShared sh;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        float m, s;
        load_entries<T, NT>(a, row);
        softmax_sums<T, NT>(static_cast<const T*>(a.logits) + row * a.ldl, 0, a.vocab, kLog2e / a.tau, sh, m, s);
        finish_row<NT>(a, row, m, s, sh);
        __syncthreads();                              // LDS is free for the next row
    }
}

// A workgroup a row, for the loss and the gradient: HOLD chunks a thread of the row stay in
// registers from the one to the other; what a longer row has beyond them is read again.  The
// chunks are taken in the order of each_pair, so that the loss is that of distill_rows.
//   grid.x: any number of workgroups up to the rows
template <typename T, int NT, int HOLD>
__global__ void __launch_bounds__(NT)
distill_train(DistillArgs a)
{
    constexpr int E = 16 / (int)sizeof(T);
    static_assert(HOLD % 2 == 0, "chunks are taken in pairs");
    __shared__ DistillShared sh;
    const float k2 = kLog2e / a.tau;
    const int whole = a.vocab / E, t = threadIdx.x;   // whole chunks; the last thread has the rest
    const bool last = t == NT - 1 && whole * E < a.vocab;
    const T low = (T)-__builtin_inff();
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const T* z = static_cast<const T*>(a.logits) + row * a.ldl;
        const u32x4 none = __builtin_bit_cast(u32x4, load_filled<T>(z, 0, 0, low));
        u32x4 held[HOLD];
#pragma unroll
        for (int i = 0; i < HOLD; ++i) held[i] = t + i * NT < whole ? load_loose(z + (t + i * NT) * E) : none;
        load_entries<T, NT>(a, row);
        float m = -__builtin_inff(), s = 0.0f;
#pragma unroll
        for (int i = 0; i < HOLD; i += 2)
            if (i * NT < whole) take_pair<T>(held + i, k2, m, s);
        for (int c = t + HOLD * NT; c < whole; c += 2 * NT) {
            const u32x4 v[2] = {load_loose(z + c * E), c + NT < whole ? load_loose(z + (c + NT) * E) : none};
            take_pair<T>(v, k2, m, s);
        }
        if (last) {
            const u32x4 v[2] = {load_filled<T>(z, whole * E, a.vocab, low), none};
            take_pair<T>(v, k2, m, s);
        }
        join_threads<NT>(k2, sh, m, s);
        const RowStats r = finish_row<NT>(a, row, m, s, sh);
        const RowGradient<T> grad(a, row, r);
        entry_shares<NT>(a, r);
        // (the places of the chunks are formed again: kept, they would take HOLD registers)
        int c0 = t;
        asm volatile("" : "+v"(c0));
#pragma unroll
        for (int i = 0; i < HOLD; ++i)
            if (c0 + i * NT < whole) store_loose(grad.g + (c0 + i * NT) * E, grad.chunk(held[i]));
        for (int c = c0 + HOLD * NT; c < whole; c += NT) store_loose(grad.g + c * E, grad.chunk(load_loose(z + c * E)));
        if (last) store_chunk(grad.g, whole * E, a.vocab, grad.chunk(load_filled<T>(z, whole * E, a.vocab, low)));
        grad.template entries<NT>(a.k, 0, a.vocab);
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
    load_entries<T, NT>(a, row);
    for (int i = 0; i < a.segments; ++i) m = __builtin_fmaxf(m, p[2 * i]);
    for (int i = 0; i < a.segments; ++i) s += p[2 * i + 1] * __builtin_amdgcn_exp2f((p[2 * i] - finite_ref(m)) * k2);
    finish_row<NT>(a, row, m, s, sh);
}

// A workgroup a segment of a row: its gradient.  Segment i of rows * segments, in turn
template <typename T, int NT>
__global__ void __launch_bounds__(NT)
distill_grad(DistillArgs a)
{
    for (int64_t b = blockIdx.x; b < a.rows * a.segments; b += gridDim.x) {
        const int64_t row = b / a.segments;
        const int lo = (int)(b - row * a.segments) * a.segment;
        const int hi = lo + a.segment < a.vocab ? lo + a.segment : a.vocab;
        const float* s = a.stats + row * kDistillStats;
        const RowStats r = {s[0], s[1], s[2], s[3], s[4]};
        load_entries<T, NT>(a, row);
        entry_shares<NT>(a, r);
        const RowGradient<T> grad(a, row, r);
        constexpr int E = 16 / (int)sizeof(T);
        T* g = grad.g + lo;
        each_pair<T, NT>(static_cast<const T*>(a.logits) + row * a.ldl, lo, hi, (T)0.0f, [&](const u32x4* v, int c, int whole) {
            if (whole == 0) {
                store_chunk(g, c * E, hi - lo, grad.chunk(v[0]));
            } else {
                if (c < whole) store_loose(g + c * E, grad.chunk(v[0]));
                if (c + NT < whole) store_loose(g + (c + NT) * E, grad.chunk(v[1]));
            }
        });
        grad.template entries<NT>(a.k, lo, hi);
    }
}

}  // namespace qtcq
