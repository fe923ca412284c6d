// Router: every token's k largest logits, their gates, each choice's row among
// the rows sorted by expert, and the balance loss
//
//     loss = experts * sum_e (counts_e / all rows) (sum_t p(t,e) / tokens with a choice),   p = softmax(logits)
//
// and the gradient of gates and loss in the logits.
//
// A token's logits lie in the registers of 16 lanes (64 above 256 experts), V
// consecutive experts to a lane, four tokens at once in a wave. They are compared
// as doubles that hold the logit and, in bits that fp32 leaves free, the
// expert's number: these order like the logits, of equal ones the lower expert
// first, and all differ, so that a maximum and a minimum are a comparator. Each
// lane sorts its K largest (k rounded up to a power of two), and four exchanges
// between lanes merge them: the larger of the first list's i-th and the second's
// last-but-i-th are the K largest of both, and log2 K rounds of comparators sort
// them. Lane j then holds choice j.
//
// The order of the rows needs every earlier token's choices. A workgroup takes 64
// tokens at a time and marks each choice as a token's bit in its expert's 64-bit
// word in LDS: the expert's count is the bits set, a choice's place among
// them the bits below its own. Each workgroup's counts go to the workspace,
// and a second launch adds up those of the workgroups before it (which each does
// for itself: the table is small) and the offsets. Up to kAlone tokens one
// workgroup does it all in one launch. No sum depends on the order of
// execution.
//
// Neither memory nor the vector unit bounds it, but the way through both: 16384
// tokens x 128 experts, 8 choices 8.5 us (4 of them vector instructions) and 6.9
// for 10 MB, 16 x 32, 2 choices 4.5, the gradient of 8191 x 64 3.8.

#include "layer.hpp"

namespace dg {
namespace {

constexpr float kInf = __builtin_inff();
constexpr float kLog2e = 1.44269504f;
// Of choose: two turns for 64 tokens of 16 lanes. With 1024 threads the waves' share
// of setting up and adding up counts twice (16384 x 128, 8 choices 9.8 us against
// 8.7, x 256 14.3 against 11.5).
constexpr int kThreads = 512;
constexpr int kChunk = 64;          // tokens at a time

// One workgroup up to here: 64 tokens at a time take as long as two launches at two
// turns (128 tokens x 128 experts, 8 choices 12.2 us against 7.7 + 4.6 and a
// second call; 256 x 64, 4 choices 12.6 against 5.2 + 5.4).
constexpr int kAlone = 128;

typedef float f32x2_a4 __attribute__((ext_vector_type(2), aligned(4)));
typedef uint32_t u32_a2 __attribute__((aligned(2)));
typedef uint32_t u32x2_a2 __attribute__((ext_vector_type(2), aligned(2)));

template <int APART>
__device__ __forceinline__ float max_lanes(float v) {
    uint32_t x, y;
    both_lanes<APART>(__builtin_bit_cast(uint32_t, v), x, y);
    return fmaxf(__builtin_bit_cast(float, x), __builtin_bit_cast(float, y));
}

template <int CTRL>
__device__ __forceinline__ float max_dpp(float v) {
    return fmaxf(v, __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true)));
}

// Largest and sum over the L lanes of a row, in all of them.
template <int L>
__device__ __forceinline__ float row_max(float v) {
    v = max_dpp<0x140>(max_dpp<0x141>(max_dpp<0x4E>(max_dpp<0xB1>(v))));
    if constexpr (L == 64) {
        v = max_lanes<32>(max_lanes<16>(v));
    }
    return v;
}
template <int L>
__device__ __forceinline__ float row_sum(float v) {
    if constexpr (L == 64) return wave_sum(v);
    else return sum_of_16(v);
}

// V logits of a row from expert e0 on: -infinity past the last. `whole`: the
// experts are a multiple of V, and lanes lie inside or outside as a whole.
template <int V>
__device__ __forceinline__ void load_logits(const float* p, int e0, int experts, bool whole, float* l) {
    if (whole) {
        p += e0 < experts ? e0 : 0;
        if constexpr (V >= 4) {
#pragma unroll
            for (int q = 0; q < V / 4; ++q) {
                const f32x4 w = *reinterpret_cast<const f32x4_a4*>(p + 4 * q);
#pragma unroll
                for (int i = 0; i < 4; ++i) l[4 * q + i] = w[i];
            }
        } else if constexpr (V == 2) {
            const f32x2_a4 w = *reinterpret_cast<const f32x2_a4*>(p);
            l[0] = w[0];
            l[1] = w[1];
        } else {
            l[0] = *p;
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) l[i] = p[e0 + i < experts ? e0 + i : experts - 1];
    }
#pragma unroll
    for (int i = 0; i < V; ++i) l[i] = e0 + i < experts ? l[i] : -kInf;
}
template <int V>
__device__ __forceinline__ void load_logits(const uint16_t* p, int e0, int experts, bool whole, float* l) {
    constexpr int kWords = (V + 1) / 2;
    uint32_t raw[kWords];
    if (whole) {
        p += e0 < experts ? e0 : 0;
        if constexpr (V >= 8) {
#pragma unroll
            for (int q = 0; q < V / 8; ++q) {
                const u32x4 w = *reinterpret_cast<const u32x4_a2*>(p + 8 * q);
#pragma unroll
                for (int i = 0; i < 4; ++i) raw[4 * q + i] = w[i];
            }
        } else if constexpr (V == 4) {
            const u32x2_a2 w = *reinterpret_cast<const u32x2_a2*>(p);
            raw[0] = w[0];
            raw[1] = w[1];
        } else if constexpr (V == 2) {
            raw[0] = *reinterpret_cast<const u32_a2*>(p);
        } else {
            raw[0] = *p;
        }
    } else {
        uint16_t one[2 * kWords] = {};
#pragma unroll
        for (int i = 0; i < V; ++i) one[i] = p[e0 + i < experts ? e0 + i : experts - 1];
#pragma unroll
        for (int q = 0; q < kWords; ++q) raw[q] = one[2 * q] | (uint32_t)one[2 * q + 1] << 16;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const uint32_t w = raw[i / 2];
        l[i] = e0 + i < experts ? __builtin_bit_cast(float, (i & 1) ? w & 0xffff0000u : w << 16) : -kInf;
    }
}

// Softmax of a row: ex = exp(l - m) (0 for a row of -infinities), and 1 / their sum: 0 for
// such a row, NaN for one that holds a NaN or +infinity (whose difference from
// itself is NaN).
template <int L, int V>
__device__ __forceinline__ float softmax(const float* l, float* ex, float& m) {
    float top = l[0], s = 0.f;
#pragma unroll
    for (int i = 1; i < V; ++i) top = fmaxf(top, l[i]);
    top = row_max<L>(top);
    m = top == -kInf ? 0.f : top;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        ex[i] = __builtin_amdgcn_exp2f((l[i] - m) * kLog2e);
        s += ex[i];
    }
    s = row_sum<L>(s);
    return s == 0.f ? 0.f : 1.f / s;
}

// A logit and its expert as a double: the logit's 24 bits stay, and the lowest
// ones take the expert so that the lower one is larger. -infinity becomes kNone, below
// every other; a -0 counts as 0.
constexpr double kNone = -0x1p1000;
__device__ __forceinline__ double keyed(float l, int e) {
    l += 0.f;
    const uint64_t bits = __builtin_bit_cast(uint64_t, (double)l);
    const uint32_t low = (uint32_t)(e ^ (kMaxExperts - 1)) ^ (uint32_t)((__builtin_bit_cast(int, l) >> 31) & (kMaxExperts - 1));
    return l == -kInf ? kNone : __builtin_bit_cast(double, bits | low);
}
__device__ __forceinline__ int expert_of(double key) {
    const u32x2 w = __builtin_bit_cast(u32x2, key);
    return (int)((w[0] ^ (uint32_t)((int)~w[1] >> 31)) & (kMaxExperts - 1));
}

__device__ __forceinline__ void larger_first(double& a, double& b) {
    const double big = __builtin_fmax(a, b);
    b = __builtin_fmin(a, b);
    a = big;
}
// v falls, or rises and falls: sorted, the largest first.
template <int N>
__device__ __forceinline__ void sort_bitonic(double* v) {
#pragma unroll
    for (int h = N / 2; h > 0; h /= 2)
#pragma unroll
        for (int i = 0; i < N; ++i)
            if ((i & h) == 0) larger_first(v[i], v[i + h]);
}
template <int N>
__device__ __forceinline__ void sort(double* v) {
    if constexpr (N > 1) {
        sort<N / 2>(v);
        sort<N / 2>(v + N / 2);
#pragma unroll
        for (int i = 0; i < N / 2; ++i) larger_first(v[i], v[N - 1 - i]);
        sort_bitonic<N / 2>(v);
        sort_bitonic<N / 2>(v + N / 2);
    }
}
// The K largest of V keys, sorted.
template <int V, int K>
__device__ __forceinline__ void largest(double* v, double* out) {
    if constexpr (V <= K) {
        sort<V>(v);
#pragma unroll
        for (int i = 0; i < K; ++i) out[i] = i < V ? v[i < V ? i : 0] : kNone;
    } else {
        double other[K];
        largest<V / 2, K>(v, out);
        largest<V / 2, K>(v + V / 2, other);
#pragma unroll
        for (int i = 0; i < K; ++i) out[i] = __builtin_fmax(out[i], other[K - 1 - i]);
        sort_bitonic<K>(out);
    }
}
template <int K, int CTRL>
__device__ __forceinline__ void merge_dpp(double* v) {
    double o[K];
#pragma unroll
    for (int i = 0; i < K; ++i) {
        const u32x2 w = __builtin_bit_cast(u32x2, v[i]);
        o[i] = __builtin_bit_cast(double, u32x2{(uint32_t)__builtin_amdgcn_mov_dpp((int)w[0], CTRL, 0xf, 0xf, true),
                                                (uint32_t)__builtin_amdgcn_mov_dpp((int)w[1], CTRL, 0xf, 0xf, true)});
    }
#pragma unroll
    for (int i = 0; i < K; ++i) v[i] = __builtin_fmax(v[i], o[K - 1 - i]);
    sort_bitonic<K>(v);
}
template <int K, int APART>
__device__ __forceinline__ void merge_lanes(double* v) {
    double a[K], b[K];
#pragma unroll
    for (int i = 0; i < K; ++i) {
        const u32x2 w = __builtin_bit_cast(u32x2, v[i]);
        uint32_t alo, blo, ahi, bhi;
        both_lanes<APART>(w[0], alo, blo);
        both_lanes<APART>(w[1], ahi, bhi);
        a[i] = __builtin_bit_cast(double, u32x2{alo, ahi});
        b[i] = __builtin_bit_cast(double, u32x2{blo, bhi});
    }
#pragma unroll
    for (int i = 0; i < K; ++i) v[i] = __builtin_fmax(a[i], b[K - 1 - i]);
    sort_bitonic<K>(v);
}
// Over the L lanes of a row: all of them end with the same K keys.
template <int L, int K>
__device__ __forceinline__ void merge_row(double* v) {
    merge_dpp<K, 0xB1>(v);
    merge_dpp<K, 0x4E>(v);
    merge_dpp<K, 0x141>(v);
    merge_dpp<K, 0x140>(v);
    if constexpr (L == 64) {
        merge_lanes<K, 16>(v);
        merge_lanes<K, 32>(v);
    }
}

// What choose leaves for place, for each workgroup: its counts, its sums of p and
// its tokens with a choice.
struct Table {
    uint16_t* counts;       // workgroups x stride
    float* sums;            // workgroups x stride
    int32_t* some;          // workgroups
    int stride;             // experts rounded up to 4
};
inline int table_stride(int experts) { return (experts + 3) & ~3; }

// Exclusive sums of counts[0 .. experts - 1] into first[0 .. experts], by one wave.
__device__ __forceinline__ void scan_counts(const int* counts, int* first, int experts, int lane) {
    const int per = (experts + 63) / 64, lo = lane * per, hi = lo + per < experts ? lo + per : experts;
    int mine = 0;
    for (int e = lo; e < hi; ++e) mine += counts[e];
    const int upto = wave_scan(mine, lane);
    int at = upto - mine;
    for (int e = lo; e < hi; ++e) {
        first[e] = at;
        at += counts[e];
    }
    if (lane == 63) first[experts] = upto;
}

// Offsets, counts and loss from the counts and sums of p over all tokens, by one
// workgroup; `red` has a float for each of its waves.
template <int THREADS, typename T>
__device__ __forceinline__ void finish(const RouteArgs<T>& a, const int* counts, const int* first, int tokens,
                                       const float* sums, float* red) {
    const int t = threadIdx.x;
    for (int e = t; e <= a.experts; e += THREADS) {
        a.offsets[e] = first[e];
        a.counts[e] = e < a.experts ? counts[e] : tokens;
    }
    if (a.loss == nullptr) return;
    float s = 0.f;
    for (int e = t; e < a.experts; e += THREADS) s += (float)counts[e] * sums[e];
    s = wave_sum(s);
    if ((t & 63) == 0) red[t >> 6] = s;
    __syncthreads();
    if (t != 0) return;
    s = 0.f;
    for (int w = 0; w < THREADS / 64; ++w) s += red[w];
    const int all = first[a.experts];
    *a.loss = (float)a.experts * (s / (float)(all > 1 ? all : 1)) / (float)(tokens > 1 ? tokens : 1);
}

// Choices, gates and, into slots, each choice's place among its expert's rows of
// this workgroup, whose tokens are `rows` from blockIdx.x * rows on (a multiple of
// kChunk). alone: the only workgroup, which finishes too.
template <typename T, int L, int V, int K>
__global__ __launch_bounds__(kThreads) void choose(RouteArgs<T> a, Table table, int rows, bool alone) {
    constexpr int kAtOnce = kThreads / L, kMost = L * V, kWaves = kThreads / 64;
    __shared__ unsigned long long bits[kMost];
    __shared__ int chosen[kChunk * K];
    __shared__ int total[kMost + 1], first[kMost + 1];
    __shared__ float sums[kWaves][kMost], red[kWaves];
    const int t = threadIdx.x, lane64 = t & 63, lane = t % L, group = t / L;
    const int e0 = lane * V;
    const bool whole = a.experts % V == 0;
    const int64_t lo = (int64_t)blockIdx.x * rows;
    const int64_t hi = lo + rows < a.tokens ? lo + rows : a.tokens;
    float psum[V] = {};
    for (int e = t; e <= a.experts; e += kThreads) total[e] = 0;
    int some = 0;                                   // the wave's tokens with a choice
    for (int64_t base = lo; base < hi; base += kChunk) {
        for (int e = t; e < a.experts; e += kThreads) bits[e] = 0;
        __syncthreads();
#pragma unroll 1
        for (int at = 0; at < kChunk; at += kAtOnce) {
            const int local = at + group;
            const int64_t token = base + local;
            const bool on = token < hi;
            float l[V], ex[V], m;
            double key[V], top[K];
            load_logits<V>(a.logits + (on ? token : hi - 1) * a.ldl, e0, a.experts, whole, l);
            const float inv = softmax<L, V>(l, ex, m);
#pragma unroll
            for (int i = 0; i < V; ++i) psum[i] += ex[i] * (on ? inv : 0.f);
#pragma unroll
            for (int i = 0; i < V; ++i) key[i] = keyed(l[i], e0 + i);
            largest<V, K>(key, top);
            merge_row<L, K>(top);
            double mine = top[0];
#pragma unroll
            for (int j = 1; j < K; ++j) mine = lane == j ? top[j] : mine;
            const bool bad = !(inv == inv);
            const bool go = on && !bad && lane < a.k && mine > kNone;
            const int e = go ? expert_of(mine) : -1;
            const float p = go ? __builtin_amdgcn_exp2f(((float)mine - m) * kLog2e) : 0.f;
            const float sum = row_sum<L>(p);
            if (lane < a.k) {
                chosen[local * a.k + lane] = e;
                if (go) atomicOr(&bits[e], 1ull << local);
                if (on) {
                    a.choice[token * a.k + lane] = e;
                    a.gates[token * a.k + lane] = bad ? inv : (go ? (a.renormalize ? p / sum : p * inv) : 0.f);
                }
            }
            some += __builtin_popcountll(__ballot(go && lane == 0));
        }
        __syncthreads();
        const int have = (int)(hi - base < kChunk ? hi - base : kChunk) * a.k;
        for (int i = t; i < have; i += kThreads) {
            const int e = chosen[i], local = i / a.k;
            a.slots[base * a.k + i] = e < 0 ? -1 : total[e] + __builtin_popcountll(bits[e] & ((1ull << local) - 1));
        }
        __syncthreads();
        for (int e = t; e < a.experts; e += kThreads) total[e] += __builtin_popcountll(bits[e]);
    }
    __syncthreads();
    if (lane64 == 0) atomicAdd(&total[a.experts], some);
    if (a.loss != nullptr) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if constexpr (L == 16) psum[i] = add_lanes<32>(add_lanes<16>(psum[i]));
            if (lane64 < L) sums[t >> 6][e0 + i] = psum[i];
        }
    }
    __syncthreads();
    if (a.loss != nullptr)
        for (int e = t; e < a.experts; e += kThreads) {
            float s = sums[0][e];
#pragma unroll
            for (int w = 1; w < kWaves; ++w) s += sums[w][e];
            if (alone) sums[0][e] = s;
            else table.sums[(int64_t)blockIdx.x * table.stride + e] = s;
        }
    if (!alone) {
        for (int e = t; e < table.stride; e += kThreads)
            table.counts[(int64_t)blockIdx.x * table.stride + e] = e < a.experts ? (uint16_t)total[e] : 0;
        if (t == 0) table.some[blockIdx.x] = total[a.experts];
        return;
    }
    if (t < 64) scan_counts(total, first, a.experts, t);
    __syncthreads();
    for (int64_t i = t; i < (int64_t)a.tokens * a.k; i += kThreads) {
        const int e = a.choice[i];
        if (e >= 0) a.slots[i] += first[e];
    }
    finish<kThreads>(a, total, first, total[a.experts], sums[0], red);
}

// Slots, from each workgroup's counts: those of the workgroups before this one
// and all of them. One workgroup more, the last, writes offsets, counts and loss.
// The tables are read by up to kSets sets of threads, 4 columns to a thread; a
// column's sets are added by one thread. N threads: 512, or 1024 above 128 experts
// (16384 tokens x 128 experts 7.0 us with 512, 7.5 with 1024; x 256 12.7 and 10.3).
// LDS additions to one address cost 8 ns each, so what many threads add up goes
// through lanes or sets first.
constexpr int kSets = 32;
template <typename T, int N>
__global__ __launch_bounds__(N) void place(RouteArgs<T> a, Table table, int rows, int blocks) {
    __shared__ int before[kMaxExperts], total[kMaxExperts], first[kMaxExperts + 1], tokens;
    __shared__ float sums[kMaxExperts], red[N / 64];
    __shared__ u32x4 part[2][N];
    const int t = threadIdx.x, words = table.stride / 4, sets = N / words < kSets ? N / words : kSets;
    const bool last = (int)blockIdx.x == blocks;
    const int64_t lo = (int64_t)blockIdx.x * rows * a.k, most = (int64_t)a.tokens * a.k;
    const int64_t hi = last ? 0 : (lo + (int64_t)rows * a.k < most ? lo + (int64_t)rows * a.k : most);
    // The first of this thread's choices, on its way while the counts are added.
    int e0 = -1, s0 = 0;
    if (lo + t < hi) {
        e0 = a.choice[lo + t];
        s0 = a.slots[lo + t];
    }
    int some = 0;                       // by the last wave, which has the fewest columns
    if (last && t >= N - 64) {
#pragma unroll 4
        for (int b = t - (N - 64); b < blocks; b += 64) some += table.some[b];
    }
    // Two 16-bit counts to an addition, for as many rows as cannot overflow them: the
    // vector unit, not memory, is what every workgroup's sum of the whole table
    // costs.
    if (t < words * sets) {
        const int w = t % words, at_once = 65535 / rows * sets;
        u32x4 all = {0, 0, 0, 0}, mine = {0, 0, 0, 0};
        for (int b0 = t / words; b0 < blocks; b0 += at_once) {
            const int end = blocks - b0 < at_once ? blocks : b0 + at_once;
            u32x2 va = {0, 0}, vm = {0, 0};
#pragma unroll 8
            for (int b = b0; b < end; b += sets) {
                const u32x2 v = *reinterpret_cast<const u32x2*>(table.counts + (int64_t)b * table.stride + 4 * w);
                const bool earlier = b < (int)blockIdx.x;
                va += v;
                vm += u32x2{earlier ? v[0] : 0u, earlier ? v[1] : 0u};
            }
            all += u32x4{va[0] & 0xffffu, va[0] >> 16, va[1] & 0xffffu, va[1] >> 16};
            mine += u32x4{vm[0] & 0xffffu, vm[0] >> 16, vm[1] & 0xffffu, vm[1] >> 16};
        }
        part[0][t] = all;
        part[1][t] = mine;
    }
    f32x4 psum = {0.f, 0.f, 0.f, 0.f};
    if (last && a.loss != nullptr && t < words * sets) {
#pragma unroll 8
        for (int b = t / words; b < blocks; b += sets)
            psum += *reinterpret_cast<const f32x4*>(table.sums + (int64_t)b * table.stride + 4 * (t % words));
    }
    __syncthreads();
    if (last && t >= N - 64) {
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) some += __shfl_xor(some, d, 64);
        tokens = some;
    }
    for (int e = t; e < table.stride; e += N) {
        const uint32_t* p = reinterpret_cast<const uint32_t*>(part) + e;
        int all = 0, mine = 0;
        for (int q = 0; q < sets; ++q) {
            all += (int)p[q * table.stride];
            mine += (int)p[4 * N + q * table.stride];
        }
        total[e] = all;
        before[e] = mine;
    }
    __syncthreads();
    if (t < 64) scan_counts(total, first, a.experts, t);
    if (last && t < words * sets) part[0][t] = __builtin_bit_cast(u32x4, psum);
    __syncthreads();
    if (!last) {
        if (e0 >= 0) a.slots[lo + t] = s0 + first[e0] + before[e0];
        for (int64_t i = lo + t + N; i < hi; i += N) {
            const int e = a.choice[i];
            if (e >= 0) a.slots[i] += first[e] + before[e];
        }
        return;
    }
    for (int e = t; e < a.experts; e += N) {
        const float* p = reinterpret_cast<const float*>(part[0]) + e;
        float v = p[0];
        for (int q = 1; q < sets; ++q) v += p[q * table.stride];
        sums[e] = v;
    }
    __syncthreads();
    finish<N>(a, total, first, tokens, sums, red);
}

// The gradient, L lanes to a token, whose softmax is taken again from its logits. The
// choices' gradients reach the lanes that hold their experts through LDS.
template <typename T, int L, int V>
__global__ __launch_bounds__(256) void route_grad(RouteGradArgs<T> a) {
    struct Chosen {
        float d;
        int in;
    };
    __shared__ Chosen lds[256 * V];
    const int t = threadIdx.x, lane = t % L, e0 = lane * V;
    Chosen* row = lds + t / L * (L * V);
    const bool whole = a.experts % V == 0;
    float bal[V], all = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        bal[i] = e0 + i < a.experts ? (float)a.counts[e0 + i] : 0.f;
        all += bal[i];
    }
    all = row_sum<L>(all);
    const float f =
        a.dloss != nullptr && all > 0.f ? *a.dloss * (float)a.experts / (all * (float)a.counts[a.experts]) : 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) bal[i] *= f;
    for (int64_t base = (int64_t)blockIdx.x * (256 / L); base < a.tokens; base += (int64_t)gridDim.x * (256 / L)) {
        const int64_t token = base + t / L;
        const bool on = token < a.tokens;
        const int64_t from = on ? token : a.tokens - 1;
        float l[V], p[V], g[V], m;
        load_logits<V>(a.logits + from * a.ldl, e0, a.experts, whole, l);
        int e = -1;
        float d = 0.f;
        if (a.dgates != nullptr && lane < a.k) {
            e = a.choice[from * a.k + lane];
            d = a.dgates[from * a.k + lane];
        }
#pragma unroll
        for (int i = 0; i < V; ++i) row[e0 + i] = Chosen{0.f, 0};
        __syncthreads();
        if (e >= 0 && e < a.experts) row[e] = Chosen{d, 1};
        __syncthreads();
        const float inv = softmax<L, V>(l, p, m);
        float s = 0.f, sd = 0.f, sum = 0.f;
        Chosen c[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            c[i] = row[e0 + i];
            p[i] *= inv;
            g[i] = bal[i];
            if (a.renormalize) {
                sum += c[i].in ? p[i] : 0.f;
                sd += c[i].in ? c[i].d * p[i] : 0.f;
            } else {
                g[i] += c[i].d;
            }
            s = __builtin_fmaf(g[i], p[i], s);
        }
        s = row_sum<L>(s);
        float scale = 0.f;
        if (a.renormalize) {
            sum = row_sum<L>(sum);
            scale = sum > 0.f ? 1.f / sum : 0.f;
            sd = row_sum<L>(sd) * scale;
        }
        T out[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float o = p[i] * (g[i] - s);
            if (a.renormalize) o += c[i].in ? p[i] * scale * (c[i].d - sd) : 0.f;
            if constexpr (sizeof(T) == 4) out[i] = o;
            else out[i] = f32_to_bf16(o);
        }
        T* to = a.dlogits + from * a.lddl + e0;
        if (on && whole) {
            if (e0 < a.experts) __builtin_memcpy(to, out, sizeof(out));
        } else if (on) {
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (e0 + i < a.experts) to[i] = out[i];
        }
    }
}

// Tokens to a workgroup: 64, or as many more that the workgroups stay at most
// 256, one to a compute unit (each adds up all their counts), within 16 bits
// for a count.
int rows_each(int tokens) {
    constexpr int64_t kBlocks = 256, kMostRows = 65472;
    const int64_t chunks = ((int64_t)tokens + kChunk * kBlocks - 1) / (kChunk * kBlocks);
    const int64_t rows = (chunks < 1 ? 1 : chunks) * kChunk;
    return (int)(rows < kMostRows ? rows : kMostRows);
}
int64_t blocks_of(int tokens) { return ((int64_t)tokens + rows_each(tokens) - 1) / rows_each(tokens); }

// The tables one after another, each from a multiple of 256 bytes on.
struct Layout {
    size_t sums, some, bytes;
};
Layout layout_of(int64_t blocks, int experts) {
    const auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
    const size_t each = (size_t)blocks * table_stride(experts);
    Layout l;
    l.sums = up(each * 2);
    l.some = l.sums + up(each * 4);
    l.bytes = l.some + up((size_t)blocks * 4) + 256;
    return l;
}

template <typename T, int L, int V, int K>
hipError_t launch_choose(const RouteArgs<T>& a, const Table& table, hipStream_t s) {
    if (a.tokens <= kAlone)
        return launch_kernel(&choose<T, L, V, K>, dim3(1), dim3(kThreads), s, a, table,
                             (a.tokens + kChunk - 1) / kChunk * kChunk, true);
    const int rows = rows_each(a.tokens);
    const unsigned blocks = (unsigned)blocks_of(a.tokens);
    const hipError_t e = launch_kernel(&choose<T, L, V, K>, dim3(blocks), dim3(kThreads), s, a, table, rows, false);
    if (e != hipSuccess) return e;
    if (a.experts > 128)
        return launch_kernel(&place<T, 1024>, dim3(blocks + 1), dim3(1024), s, a, table, rows, (int)blocks);
    return launch_kernel(&place<T, 512>, dim3(blocks + 1), dim3(512), s, a, table, rows, (int)blocks);
}
template <typename T, int L, int V>
hipError_t launch_choose(const RouteArgs<T>& a, const Table& table, hipStream_t s) {
    if (a.k <= 2) return launch_choose<T, L, V, 2>(a, table, s);
    if (a.k <= 4) return launch_choose<T, L, V, 4>(a, table, s);
    if (a.k <= 8) return launch_choose<T, L, V, 8>(a, table, s);
    return launch_choose<T, L, V, 16>(a, table, s);
}

template <typename T>
hipError_t launch(const RouteArgs<T>& a, hipStream_t s) {
    Table table;
    table.stride = table_stride(a.experts);
    table.counts = static_cast<uint16_t*>(a.ws);
    const Layout l = layout_of(blocks_of(a.tokens), a.experts);
    table.sums = reinterpret_cast<float*>(static_cast<char*>(a.ws) + l.sums);
    table.some = reinterpret_cast<int32_t*>(static_cast<char*>(a.ws) + l.some);
    if (a.experts <= 16) return launch_choose<T, 16, 1>(a, table, s);
    if (a.experts <= 32) return launch_choose<T, 16, 2>(a, table, s);
    if (a.experts <= 64) return launch_choose<T, 16, 4>(a, table, s);
    if (a.experts <= 128) return launch_choose<T, 16, 8>(a, table, s);
    if (a.experts <= 256) return launch_choose<T, 16, 16>(a, table, s);
    if (a.experts <= 512) return launch_choose<T, 64, 8>(a, table, s);
    return launch_choose<T, 64, 16>(a, table, s);
}

template <typename T>
hipError_t launch_grad(const RouteGradArgs<T>& a, hipStream_t s) {
    const int at_once = a.experts <= 256 ? 16 : 4;
    const dim3 grid(grid_for(((int64_t)a.tokens + at_once - 1) / at_once)), block(256);
    if (a.experts <= 16) return launch_kernel(&route_grad<T, 16, 1>, grid, block, s, a);
    if (a.experts <= 32) return launch_kernel(&route_grad<T, 16, 2>, grid, block, s, a);
    if (a.experts <= 64) return launch_kernel(&route_grad<T, 16, 4>, grid, block, s, a);
    if (a.experts <= 128) return launch_kernel(&route_grad<T, 16, 8>, grid, block, s, a);
    if (a.experts <= 256) return launch_kernel(&route_grad<T, 16, 16>, grid, block, s, a);
    if (a.experts <= 512) return launch_kernel(&route_grad<T, 64, 8>, grid, block, s, a);
    return launch_kernel(&route_grad<T, 64, 16>, grid, block, s, a);
}

}  // namespace

size_t route_workspace(int64_t tokens, int64_t experts, int) {
    return layout_of(blocks_of((int)tokens), (int)experts).bytes;
}

hipError_t launch_route(const RouteArgs<uint16_t>& a, hipStream_t s) { return launch(a, s); }
hipError_t launch_route(const RouteArgs<float>& a, hipStream_t s) { return launch(a, s); }
hipError_t launch_route_grad(const RouteGradArgs<uint16_t>& a, hipStream_t s) { return launch_grad(a, s); }
hipError_t launch_route_grad(const RouteGradArgs<float>& a, hipStream_t s) { return launch_grad(a, s); }

}  // namespace dg
