// Router: every token's k largest logits, their gates, each choice's row among
// the rows sorted by expert, and the balance loss
//
//     loss = experts * sum_e (counts_e / all rows) (sum_t p(t,e) / tokens with a choice),   p = softmax(logits)
//
// and the gradient of gates and loss in the logits.
//
// A token's logits lie in the registers of 16 lanes (64 above 256 experts), V
// consecutive experts to a lane, so that a maximum is V - 1 operations and four
// lane exchanges of the vector unit, for four tokens at once in a wave. The k
// choices are k such searches; of equal logits the lowest lane's first takes it.
//
// The order of the rows needs every earlier token's choices. A workgroup takes 64
// tokens at a time and marks each choice as a token's bit in its expert's 64-bit
// word in LDS: the expert's count is the bits set, a choice's place among
// them the bits below its own. Each workgroup's counts go to the workspace,
// and a second launch adds up those of the workgroups before it (which each does
// for itself: the table is small) and the offsets. Up to kAlone tokens one
// workgroup does it all in one launch. No sum depends on the order of
// execution.

#include "layer.hpp"

namespace dg {
namespace {

constexpr float kInf = __builtin_inff();
constexpr float kLog2e = 1.44269504f;
constexpr int kThreads = 1024;      // of choose and place
constexpr int kChunk = 64;          // tokens at a time

// One workgroup up to here.
constexpr int kAlone = 256;

__device__ __forceinline__ float max_of_16(float v) {
    auto step = [](float a, auto ctrl) {
        return fmaxf(a, __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, a), ctrl(), 0xf, 0xf, true)));
    };
    v = step(v, [] { return 0xB1; });
    v = step(v, [] { return 0x4E; });
    v = step(v, [] { return 0x141; });
    return step(v, [] { return 0x140; });
}

// Largest and sum over the L lanes of a row, in all of them.
template <int L>
__device__ __forceinline__ float row_max(float v) {
    v = max_of_16(v);
    if constexpr (L == 64) {
        v = fmaxf(v, __shfl_xor(v, 16, 64));
        v = fmaxf(v, __shfl_xor(v, 32, 64));
    }
    return v;
}
template <int L>
__device__ __forceinline__ float row_sum(float v) {
    if constexpr (L == 64) return wave_sum(v);
    else return sum_of_16(v);
}
// The L lanes' bits of a ballot, lane 0's lowest.
template <int L>
__device__ __forceinline__ uint64_t row_ballot(bool b, int lane64) {
    const uint64_t all = __ballot(b);
    if constexpr (L == 64) return all;
    else return (all >> (lane64 & 48)) & 0xffff;
}

// V logits of a row from expert e0 on: -infinity past the last. `whole`: the
// experts are a multiple of V, and lanes lie inside or outside as a whole.
template <typename T, int V>
__device__ __forceinline__ void load_logits(const T* p, int e0, int experts, bool whole, float* l) {
    T raw[V];
    if (whole) {
        __builtin_memcpy(raw, p + (e0 < experts ? e0 : 0), sizeof(raw));
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) raw[i] = p[e0 + i < experts ? e0 + i : experts - 1];
    }
#pragma unroll
    for (int i = 0; i < V; ++i) l[i] = e0 + i < experts ? elem_f32(raw[i]) : -kInf;
}

// Softmax of a row: ex = exp(l - m) (0 for a row of -infinities), and 1 / their sum: 0 for
// such a row, NaN for one that holds a NaN or +infinity.
template <int L, int V>
__device__ __forceinline__ float softmax(const float* l, float* ex, float& m, int lane64) {
    bool bad = false;
    float top = -kInf, s = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        bad |= !(l[i] < kInf);
        top = fmaxf(top, l[i]);
    }
    bad = row_ballot<L>(bad, lane64) != 0;
    top = row_max<L>(top);
    m = top == -kInf ? 0.f : top;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        ex[i] = __builtin_amdgcn_exp2f((l[i] - m) * kLog2e);
        s += ex[i];
    }
    s = row_sum<L>(s);
    return bad ? __builtin_nanf("") : (s > 0.f ? 1.f / s : 0.f);
}

// What choose leaves for place, for each workgroup: its counts (and its tokens
// with a choice at [experts]) and its sums of p.
struct Table {
    uint16_t* counts;       // workgroups x stride
    float* sums;            // workgroups x experts
    int stride;
};
inline __host__ __device__ int table_stride(int experts) { return (experts + 1 + 3) & ~3; }

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
template <typename T>
__device__ __forceinline__ void finish(const RouteArgs<T>& a, const int* counts, const int* first, const float* sums,
                                       float* red) {
    const int t = threadIdx.x;
    for (int e = t; e <= a.experts; e += kThreads) {
        a.offsets[e] = first[e];
        a.counts[e] = counts[e];
    }
    if (a.loss == nullptr) return;
    float s = 0.f;
    for (int e = t; e < a.experts; e += kThreads) s += (float)counts[e] * sums[e];
    s = wave_sum(s);
    if ((t & 63) == 0) red[t >> 6] = s;
    __syncthreads();
    if (t != 0) return;
    s = 0.f;
    for (int w = 0; w < kThreads / 64; ++w) s += red[w];
    const int all = first[a.experts], tokens = counts[a.experts];
    *a.loss = (float)a.experts * (s / (float)(all > 1 ? all : 1)) / (float)(tokens > 1 ? tokens : 1);
}

// Choices, gates and, into slots, each choice's place among its expert's rows of
// this workgroup, whose tokens are `rows` from blockIdx.x * rows on (a multiple of
// kChunk). ALONE: the only workgroup, which finishes too.
template <typename T, int L, int V, bool ALONE>
__global__ __launch_bounds__(kThreads) void choose(RouteArgs<T> a, Table table, int rows) {
    constexpr int kAtOnce = kThreads / L, kMost = L * V, kWaves = kThreads / 64;
    __shared__ unsigned long long bits[kMost];
    __shared__ int chosen[kChunk * kMaxChoices];
    __shared__ int total[kMost + 1];
    __shared__ float sums[kWaves][kMost];
    __shared__ int first[ALONE ? kMost + 1 : 1];
    __shared__ float red[ALONE ? kWaves : 1];
    const int t = threadIdx.x, lane64 = t & 63, lane = t % L, group = t / L;
    const int e0 = lane * V;
    const bool whole = a.experts % V == 0;
    const int64_t lo = (int64_t)blockIdx.x * rows;
    const int64_t hi = lo + rows < a.tokens ? lo + rows : a.tokens;
    float psum[V] = {};
    for (int e = t; e <= a.experts; e += kThreads) total[e] = 0;
    int some = 0;                                   // tokens with a choice, in a row's first lane
    for (int64_t base = lo; base < hi; base += kChunk) {
        for (int e = t; e < a.experts; e += kThreads) bits[e] = 0;
        __syncthreads();
#pragma unroll
        for (int at = 0; at < kChunk; at += kAtOnce) {
            const int local = at + group;
            const int64_t token = base + local;
            const bool on = token < hi;
            float l[V], ex[V], m;
            load_logits<T, V>(a.logits + (on ? token : hi - 1) * a.ldl, e0, a.experts, whole, l);
            const float inv = softmax<L, V>(l, ex, m, lane64);
            const bool bad = !(inv == inv);
            if (on) {
#pragma unroll
                for (int i = 0; i < V; ++i) psum[i] += bad ? inv : ex[i] * inv;
            }
            float gate = bad ? inv : 0.f, sum = 0.f;
            for (int j = 0; j < a.k; ++j) {
                float mine = l[0];
#pragma unroll
                for (int i = 1; i < V; ++i) mine = fmaxf(mine, l[i]);
                const float top = row_max<L>(mine);
                const bool go = top > -kInf && !bad && on;
                const int winner = __builtin_ctzll(row_ballot<L>(mine == top, lane64) | (1ull << 63));
                const float p = __builtin_amdgcn_exp2f((top - m) * kLog2e);
                if (go) {
                    sum += p;
                    if (lane == j) gate = p;
                    if (lane == winner) {
                        int e = -1;
#pragma unroll
                        for (int i = V - 1; i >= 0; --i) e = l[i] == top ? i : e;
#pragma unroll
                        for (int i = 0; i < V; ++i) l[i] = i == e ? -kInf : l[i];
                        chosen[local * a.k + j] = e0 + e;
                        atomicOr(&bits[e0 + e], 1ull << local);
                    }
                } else if (lane == 0) {
                    chosen[local * a.k + j] = -1;
                }
                if (j == 0 && go) some += 1;
            }
            if (on && lane < a.k) {
                if (!bad && sum > 0.f) gate = a.renormalize ? gate / sum : gate * inv;
                a.gates[token * a.k + lane] = gate;
            }
        }
        __syncthreads();
        const int have = (int)(hi - base < kChunk ? hi - base : kChunk) * a.k;
        for (int i = t; i < have; i += kThreads) {
            const int e = chosen[i], local = i / a.k;
            a.choice[base * a.k + i] = e;
            a.slots[base * a.k + i] =
                e < 0 ? -1 : total[e] + __builtin_popcountll(bits[e] & ((1ull << local) - 1));
        }
        __syncthreads();
        for (int e = t; e < a.experts; e += kThreads) total[e] += __builtin_popcountll(bits[e]);
    }
    __syncthreads();
    if (lane == 0 && some != 0) atomicAdd(&total[a.experts], some);
    if (a.loss != nullptr) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if constexpr (L == 16) {
                psum[i] += __shfl_xor(psum[i], 16, 64);
                psum[i] += __shfl_xor(psum[i], 32, 64);
            }
            if (lane64 < L) sums[t >> 6][e0 + i] = psum[i];
        }
    }
    __syncthreads();
    if (a.loss != nullptr)
        for (int e = t; e < a.experts; e += kThreads) {
            float s = sums[0][e];
#pragma unroll
            for (int w = 1; w < kWaves; ++w) s += sums[w][e];
            if constexpr (ALONE) sums[0][e] = s;
            else table.sums[(int64_t)blockIdx.x * a.experts + e] = s;
        }
    if constexpr (!ALONE) {
        for (int e = t; e < table.stride; e += kThreads)
            table.counts[(int64_t)blockIdx.x * table.stride + e] = e <= a.experts ? (uint16_t)total[e] : 0;
    } else {
        if (t < 64) scan_counts(total, first, a.experts, t);
        __syncthreads();
        // The places were written by this workgroup; total is complete.
        for (int64_t i = t; i < (int64_t)a.tokens * a.k; i += kThreads) {
            const int e = a.choice[i];
            if (e >= 0) a.slots[i] += first[e];
        }
        finish(a, total, first, sums[0], red);
    }
}

// Slots, from each workgroup's counts: those of the workgroups before this one
// and all of them. The first one writes offsets, counts and loss too.
template <typename T>
__global__ __launch_bounds__(kThreads) void place(RouteArgs<T> a, Table table, int rows, int blocks) {
    __shared__ int before[kMaxExperts + 4], total[kMaxExperts + 4], first[kMaxExperts + 1];
    __shared__ float sums[kMaxExperts], red[kThreads / 64];
    const int t = threadIdx.x, words = table.stride / 4, sets = kThreads / words;
    for (int e = t; e < table.stride; e += kThreads) before[e] = total[e] = 0;
    __syncthreads();
    if (t < words * sets) {
        const int w = t % words;
        int all[4] = {}, mine[4] = {};
#pragma unroll 4
        for (int b = t / words; b < blocks; b += sets) {
            const u32x2 v = *reinterpret_cast<const u32x2*>(table.counts + (int64_t)b * table.stride + 4 * w);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int n = (int)((i & 1) ? v[i >> 1] >> 16 : v[i >> 1] & 0xffffu);
                all[i] += n;
                mine[i] += b < (int)blockIdx.x ? n : 0;
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            atomicAdd(&total[4 * w + i], all[i]);
            atomicAdd(&before[4 * w + i], mine[i]);
        }
    }
    __syncthreads();
    if (t < 64) scan_counts(total, first, a.experts, t);
    __syncthreads();
    const int64_t lo = (int64_t)blockIdx.x * rows * a.k, most = (int64_t)a.tokens * a.k;
    const int64_t hi = lo + (int64_t)rows * a.k < most ? lo + (int64_t)rows * a.k : most;
    for (int64_t i = lo + t; i < hi; i += kThreads) {
        const int e = a.choice[i];
        if (e >= 0) a.slots[i] += first[e] + before[e];
    }
    if (blockIdx.x != 0) return;
    if (a.loss != nullptr) {
        // A column of sums to each thread, 1024 / experts threads to a column: in a fixed order.
        float* part = reinterpret_cast<float*>(before);
        const int share = kThreads / a.experts, e = t % a.experts, s = t / a.experts;
        float v = 0.f;
        if (s < share)
#pragma unroll 8
            for (int b = s; b < blocks; b += share) v += table.sums[(int64_t)b * a.experts + e];
        __syncthreads();
        if (s < share) part[s * a.experts + e] = v;
        __syncthreads();
        for (int c = t; c < a.experts; c += kThreads) {
            v = part[c];
            for (int q = 1; q < share; ++q) v += part[q * a.experts + c];
            sums[c] = v;
        }
        __syncthreads();
    }
    finish(a, total, first, sums, red);
}

// The gradient, L lanes to a token. The choices' gradients reach the lanes that
// hold their experts through LDS.
template <typename T, int L, int V>
__global__ __launch_bounds__(256) void route_grad(RouteGradArgs<T> a) {
    struct Chosen {
        float d;
        int in;
    };
    __shared__ Chosen lds[256 * V];
    const int t = threadIdx.x, lane64 = t & 63, lane = t % L, e0 = lane * V;
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
        load_logits<T, V>(a.logits + from * a.ldl, e0, a.experts, whole, l);
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
        const float inv = softmax<L, V>(l, p, m, lane64);
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
// 1024 (each adds up all their counts), within 16 bits for a count.
int rows_each(int tokens) {
    constexpr int64_t kBlocks = 1024, kMostRows = 65472;
    const int64_t chunks = ((int64_t)tokens + kChunk * kBlocks - 1) / (kChunk * kBlocks);
    const int64_t rows = (chunks < 1 ? 1 : chunks) * kChunk;
    return (int)(rows < kMostRows ? rows : kMostRows);
}
int64_t blocks_of(int tokens) { return ((int64_t)tokens + rows_each(tokens) - 1) / rows_each(tokens); }
size_t sums_at(int64_t blocks, int experts) { return ((size_t)blocks * table_stride(experts) * 2 + 255) & ~(size_t)255; }

template <typename T, int L, int V>
hipError_t launch_choose(const RouteArgs<T>& a, const Table& table, hipStream_t s) {
    if (a.tokens <= kAlone)
        return launch_kernel(&choose<T, L, V, true>, dim3(1), dim3(kThreads), s, a, table,
                             (a.tokens + kChunk - 1) / kChunk * kChunk);
    const int rows = rows_each(a.tokens);
    const unsigned blocks = (unsigned)blocks_of(a.tokens);
    const hipError_t e = launch_kernel(&choose<T, L, V, false>, dim3(blocks), dim3(kThreads), s, a, table, rows);
    if (e != hipSuccess) return e;
    return launch_kernel(&place<T>, dim3(blocks), dim3(kThreads), s, a, table, rows, (int)blocks);
}

template <typename T>
hipError_t launch(const RouteArgs<T>& a, hipStream_t s) {
    Table table;
    table.stride = table_stride(a.experts);
    table.counts = static_cast<uint16_t*>(a.ws);
    table.sums = reinterpret_cast<float*>(static_cast<char*>(a.ws) + sums_at(blocks_of(a.tokens), a.experts));
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
    const int64_t blocks = blocks_of((int)tokens);
    return sums_at(blocks, (int)experts) + (size_t)blocks * experts * sizeof(float) + 256;
}

hipError_t launch_route(const RouteArgs<uint16_t>& a, hipStream_t s) { return launch(a, s); }
hipError_t launch_route(const RouteArgs<float>& a, hipStream_t s) { return launch(a, s); }
hipError_t launch_route_grad(const RouteGradArgs<uint16_t>& a, hipStream_t s) { return launch_grad(a, s); }
hipError_t launch_route_grad(const RouteGradArgs<float>& a, hipStream_t s) { return launch_grad(a, s); }

}  // namespace dg
