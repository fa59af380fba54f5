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
// gradient wanted in the same call holds it in registers until the sum is known; with few rows
// several workgroups share one (distill_partial, distill_join, distill_grad).  The k entries'
// own sums are in binary64.
//
// Bound by memory: 4096x128000 bf16 486 us with the gradient (4.3 TB/s; 717 when the row was read
// again), 181 for the loss alone (5.8 TB/s), 395 for the gradient alone; 1001x50021 fp16 58 us, in
// two rows a workgroup, of which the first's loads and the last's stores overlap nothing.
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
// z: the logit at the index, and then, for the gradient, the number of the next entry of its
// list (1 and up; 0 ends it).  t: the teacher's logit, and then what its element's gradient has
// to give up: the p of all entries at the index for the first of them, 0 for the others.
struct Entry { int index; union { float z; uint32_t next; }; float t, p; };
// lists of entries by the chunk that they are in, and how many there are
constexpr int kLists(int nt) { return nt < 512 ? nt * 8 : 4096; }
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
// thread's, whose wave takes them last: f(v, whole, whole + 1) with them in that thread's v[0],
// and c past that in the other threads.
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
    if (t >= NT - 64 && whole * E < hi - lo) {
        const bool mine = t == NT - 1;
        v[0] = mine ? load_filled<T>(z, whole * E, hi - lo, fill) : none;
        v[1] = none;
        f(v, mine ? whole : whole + 1, whole + 1);
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
        en[j].index = i;
        en[j].z = i >= 0 ? to_f32(static_cast<const T*>(a.logits)[row * a.ldl + i]) : 0.0f;
        en[j].t = t;
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
    // the teacher's maximum, and the sum about it or the one that the given sum stands for: both
    // of p's parts stay small, so that the gradient's binary32 p is that of the loss
    float tm = -__builtin_inff();
    for (int j = threadIdx.x; j < a.k; j += NT)
        if (en[j].index >= 0) tm = __builtin_fmaxf(tm, en[j].t);
    tm = block_max<NT>(tm, sh.red[0]);
    double tls;
    if (a.teacher_log_z) {
        tm = __builtin_fabsf(tm) < __builtin_inff() ? tm : 0.0f;
        tls = (double)a.teacher_log_z[row] * 1.4426950408889634 - (double)tm * k2;
    } else {
        tm = finite_ref(tm);
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

// The gradient of a row's elements lo .. hi - 1, a chunk at a time.  A chunk's list holds the
// entries that are in it (and in others of the same list), each taken off its element before
// the store.
template <typename T, int NT>
struct RowGradient {
    static constexpr int E = 16 / (int)sizeof(T);
    T* g;                                             // from lo on
    int lo, n;
    float k2, ref, ls, scale, coef;
    bool none;
    const uint32_t* lists;

    __device__ __forceinline__ RowGradient(const DistillArgs& a, int64_t row, int from, int to, const RowStats& r,
                                           const uint32_t* heads)
        : g(static_cast<T*>(a.grad) + row * a.ldg + from), lo(from), n(to - from), k2(kLog2e / a.tau), ref(finite_ref(r.m)),
          ls(r.ls), scale(a.grad_loss[row] / a.tau), coef(scale * r.mass), none(r.mass == 0.0f), lists(heads) {}

    // chunk c (from lo on) with the logits v, if it is `there`
    __device__ __forceinline__ void put(bool there, int c, u32x4 v) const
    {
        float x[E];
        unpack<T>(v, x);
#pragma unroll
        for (int e = 0; e < E; ++e) x[e] = coef * __builtin_amdgcn_exp2f(__builtin_fmaf(x[e] - ref, k2, -ls));
        uint32_t at = there ? lists[c & (kLists(NT) - 1)] : 0u;
        if (__builtin_expect(at != 0u, 0)) {
            const Entry* en = reinterpret_cast<const Entry*>(distill_entries);
            do {
                const Entry o = en[at - 1];
                const int e0 = o.index - lo - c * E;
                if (o.t != 0.0f && e0 >= 0 && e0 < E) {
                    const float p = scale * o.t;
#pragma unroll
                    for (int e = 0; e < E; ++e) x[e] = e == e0 ? x[e] - p : x[e];
                }
                at = o.next;
            } while (at != 0u);
        }
        if (there) store_chunk(g, c * E, n, none ? u32x4{0u, 0u, 0u, 0u} : pack<T>(x));
    }
};

// The lists of a row's entries in the elements lo .. hi - 1.  Their order within a list is that
// of arrival, on which no result depends: an index's first entry alone has a share to give
// up, the sum of p over the entries at that index in their own order.
template <typename T, int NT>
__device__ __forceinline__ void list_entries(const DistillArgs& a, int lo, int hi, const RowStats& r, uint32_t* lists)
{
    constexpr int E = 16 / (int)sizeof(T);
    Entry* en = reinterpret_cast<Entry*>(distill_entries);
    for (int i = threadIdx.x; i < kLists(NT); i += NT) lists[i] = 0;
    __syncthreads();
    const bool any = r.mass != 0.0f;
    auto inside = [&](int j) { return any && en[j].index >= lo && en[j].index < hi; };
    for (int j = threadIdx.x; j < a.k; j += NT)
        if (inside(j)) {
            en[j].p = __builtin_amdgcn_exp2f((en[j].t - r.tm) * (kLog2e / a.tau) - r.tls);
            en[j].next = atomicExch(&lists[(en[j].index - lo) / E & (kLists(NT) - 1)], (uint32_t)j + 1u);
        }
    __syncthreads();
    for (int j = threadIdx.x; j < a.k; j += NT)
        if (inside(j)) {
            const int i = en[j].index;
            bool first = true, alone = true;
            for (uint32_t l = lists[(i - lo) / E & (kLists(NT) - 1)]; l != 0u; l = en[l - 1].next)
                if (en[l - 1].index == i && (int)l - 1 != j) {
                    alone = false;
                    first = first && (int)l - 1 > j;
                }
            double p = first ? (double)en[j].p : 0.0;
            if (first && !alone)
                for (int l = j + 1; l < a.k; ++l)
                    if (en[l].index == i) p += (double)en[l].p;
            en[j].t = (float)p;
        }
    __syncthreads();
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
// registers from the one to the other; what a longer row has beyond them is read again.  As
// a chunk's gradient is stored, the same chunk of the workgroup's next row is loaded in its
// place.  The chunks are taken in the order of each_pair, so that the loss is that of
// distill_rows.
//   grid.x: any number of workgroups up to the rows
template <typename T, int NT, int HOLD>
__global__ void __launch_bounds__(NT)
distill_train(DistillArgs a)
{
    constexpr int E = 16 / (int)sizeof(T);
    static_assert(HOLD % 2 == 0, "chunks are taken in pairs");
    __shared__ DistillShared sh;
    __shared__ uint32_t lists[kLists(NT)];
    const float k2 = kLog2e / a.tau;
    const int whole = a.vocab / E, t = threadIdx.x;   // whole chunks; the last thread has the rest
    const bool rest = t >= NT - 64 && whole * E < a.vocab, last = t == NT - 1;
    const T low = (T)-__builtin_inff();
    const T* z = static_cast<const T*>(a.logits) + blockIdx.x * a.ldl;
    const u32x4 none = __builtin_bit_cast(u32x4, load_filled<T>(z, 0, 0, low));
    u32x4 held[HOLD];
#pragma unroll
    for (int i = 0; i < HOLD; ++i) held[i] = t + i * NT < whole ? load_loose(z + (t + i * NT) * E) : none;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        load_entries<T, NT>(a, row);
        float m = -__builtin_inff(), s = 0.0f;
#pragma unroll
        for (int i = 0; i < HOLD; i += 2)
            if (i * NT < whole) take_pair<T>(held + i, k2, m, s);
        for (int c = t + HOLD * NT; c < whole; c += 2 * NT) {
            const u32x4 v[2] = {load_loose(z + c * E), c + NT < whole ? load_loose(z + (c + NT) * E) : none};
            take_pair<T>(v, k2, m, s);
        }
        if (rest) {
            const u32x4 v[2] = {last ? load_filled<T>(z, whole * E, a.vocab, low) : none, none};
            take_pair<T>(v, k2, m, s);
        }
        join_threads<NT>(k2, sh, m, s);
        const RowStats r = finish_row<NT>(a, row, m, s, sh);
        list_entries<T, NT>(a, 0, a.vocab, r, lists);
        const RowGradient<T, NT> grad(a, row, 0, a.vocab, r, lists);
        // (the places of the chunks and their binary32 elements are formed again: kept from the
        // loss on, they would take more registers than the chunks)
        int c0 = t;
        asm volatile("" : "+v"(c0));
#pragma unroll
        for (int i = 0; i < HOLD; ++i) asm volatile("" : "+v"(held[i]));
        for (int c = HOLD * NT; c < whole; c += NT) {
            const bool there = c + c0 < whole;
            grad.put(there, c + c0, there ? load_loose(z + (c + c0) * E) : none);
        }
        if (rest) grad.put(last, whole, last ? load_filled<T>(z, whole * E, a.vocab, low) : none);
        const bool more = row + gridDim.x < a.rows;
        z += gridDim.x * a.ldl;
#pragma unroll
        for (int i = 0; i < HOLD; ++i)
            if (i * NT < whole) {
                const bool there = c0 + i * NT < whole;
                grad.put(there, c0 + i * NT, held[i]);
                held[i] = there && more ? load_loose(z + (c0 + i * NT) * E) : none;
            }
        __syncthreads();                              // LDS is free for the next row
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

// The segments of a row joined, and its loss.  grid.x = rows
template <typename T, int NT>
__global__ void __launch_bounds__(NT)
distill_join(DistillArgs a)
{
    __shared__ DistillShared sh;
    const int64_t row = blockIdx.x;
    const float* p = a.part + row * a.segments * 2;
    const float k2 = kLog2e / a.tau;
    // (a thread's first segment is read beside the entries)
    const bool any = (int)threadIdx.x < a.segments;
    float m = any ? p[2 * threadIdx.x] : -__builtin_inff(), s = any ? p[2 * threadIdx.x + 1] : 0.0f;
    load_entries<T, NT>(a, row);
    for (int i = threadIdx.x + NT; i < a.segments; i += NT) {
        const float top = __builtin_fmaxf(m, p[2 * i]), ref = finite_ref(top);
        s = s * __builtin_amdgcn_exp2f((m - ref) * k2) + p[2 * i + 1] * __builtin_amdgcn_exp2f((p[2 * i] - ref) * k2);
        m = top;
    }
    join_threads<NT>(k2, sh, m, s);
    finish_row<NT>(a, row, m, s, sh);
}

// A workgroup a segment of a row: its gradient.  Segment i of rows * segments, in turn
template <typename T, int NT>
__global__ void __launch_bounds__(NT)
distill_grad(DistillArgs a)
{
    __shared__ uint32_t lists[kLists(NT)];
    for (int64_t b = blockIdx.x; b < a.rows * a.segments; b += gridDim.x) {
        const int64_t row = b / a.segments;
        const int lo = (int)(b - row * a.segments) * a.segment;
        const int hi = lo + a.segment < a.vocab ? lo + a.segment : a.vocab;
        const float* s = a.stats + row * kDistillStats;
        const RowStats r = {s[0], s[1], s[2], s[3], s[4]};
        load_entries<T, NT>(a, row);
        list_entries<T, NT>(a, lo, hi, r, lists);
        const RowGradient<T, NT> grad(a, row, lo, hi, r, lists);
        each_pair<T, NT>(static_cast<const T*>(a.logits) + row * a.ldl, lo, hi, (T)0.0f, [&](const u32x4* v, int c, int whole) {
            grad.put(c < whole, c, v[0]);
            grad.put(c + NT < whole, c + NT, v[1]);
        });
        __syncthreads();                              // LDS is free for the next row
    }
}

}  // namespace qtcq
