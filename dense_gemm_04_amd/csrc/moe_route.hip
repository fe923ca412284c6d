// Router: every token's k largest logits, their gates, each choice's row among
// the rows sorted by expert, and the balance loss
//
//     loss = experts * sum_e (counts_e / all rows) (sum_t p(t,e) / tokens with a choice),   p = softmax(logits)
//
// and the gradient of gates and loss in the logits.

#include "layer.hpp"

namespace dg {
namespace {

constexpr float kInf = __builtin_inff();
constexpr int kLanes = 64;
constexpr int kPer = kMaxExperts / kLanes;       // logits of a row in one lane

// A row's logits in a wave: expert e in lane e % 64, place e / 64; -infinity past
// the last. m: the largest; sum: of exp(l - m), 0 for a row of -infinities, NaN for
// one that holds a NaN or +infinity.
struct Row {
    float l[kPer];
    float m, sum;
};

template <typename T>
__device__ __forceinline__ Row load_row(const T* p, int experts, int lane) {
    Row r;
    bool bad = false;
    r.m = -kInf;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int e = lane + i * kLanes;
        r.l[i] = e < experts ? elem_f32(p[e]) : -kInf;
        bad |= !(r.l[i] < kInf);
        r.m = fmaxf(r.m, r.l[i]);
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) r.m = fmaxf(r.m, __shfl_xor(r.m, d, 64));
    bad = __ballot(bad) != 0;
    r.sum = 0.f;
    if (r.m == -kInf) r.m = 0.f;                 // exp(-infinity - 0) = 0
#pragma unroll
    for (int i = 0; i < kPer; ++i) r.sum += expf(r.l[i] - r.m);
    r.sum = bad ? __builtin_nanf("") : wave_sum(r.sum);
    return r;
}

// Choices and gates of each token, a wave to a token. stats: m and 1 / sum (0
// without a choice).
template <typename T>
__global__ __launch_bounds__(256) void choose(RouteArgs<T> a, float* stats) {
    const int lane = threadIdx.x & 63;
    for (int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); t < a.tokens; t += (int64_t)gridDim.x * 4) {
        Row r = load_row(a.logits + t * a.ldl, a.experts, lane);
        const bool bad = !(r.sum == r.sum);
        const float inv = r.sum > 0.f ? 1.f / r.sum : r.sum;
        if (lane == 0) {
            stats[2 * t] = r.m;
            stats[2 * t + 1] = inv;
        }
        float gate = bad ? __builtin_nanf("") : 0.f, chosen = 0.f;
        int mine = -1;
        for (int j = 0; j < a.k && !bad; ++j) {
            float top = -kInf;
            int at = a.experts;
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                if (r.l[i] > top) {
                    top = r.l[i];
                    at = lane + i * kLanes;
                }
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const float o = __shfl_xor(top, d, 64);
                const int w = __shfl_xor(at, d, 64);
                if (o > top || (o == top && w < at)) {
                    top = o;
                    at = w;
                }
            }
            if (top == -kInf) break;
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                if (at == lane + i * kLanes) r.l[i] = -kInf;
            const float p = expf(top - r.m);
            chosen += p;
            if (lane == j) {
                mine = at;
                gate = p;
            }
        }
        if (mine >= 0) gate = a.renormalize ? gate / chosen : gate * inv;
        if (lane < a.k) {
            a.choice[t * a.k + lane] = mine;
            a.gates[t * a.k + lane] = gate;
        }
    }
}

// A workgroup to an expert: the number of earlier tokens that chose it (into
// slots), its count, and the sum of its probabilities. The last one counts the
// tokens with a choice.
template <typename T>
__global__ __launch_bounds__(256) void count(RouteArgs<T> a, const float* stats, float* psum) {
    __shared__ int part[4];
    __shared__ float sums[4];
    const int e = blockIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int total = 0;
    float s = 0.f;
    for (int64_t t0 = 0; t0 < a.tokens; t0 += 256) {
        const int64_t t = t0 + threadIdx.x;
        int at = -1;
        if (t < a.tokens) {
            if (e == a.experts) {
                at = a.choice[t * a.k] >= 0 ? 0 : -1;
            } else {
                for (int j = 0; j < a.k; ++j)
                    if (a.choice[t * a.k + j] == e) at = j;
                s += expf(elem_f32(a.logits[t * a.ldl + e]) - stats[2 * t]) * stats[2 * t + 1];
            }
        }
        const unsigned long long hit = __ballot(at >= 0);
        __syncthreads();
        if (lane == 0) part[wave] = __builtin_popcountll(hit);
        __syncthreads();
        int before = total + __builtin_popcountll(hit & ((1ull << lane) - 1));
        for (int w = 0; w < wave; ++w) before += part[w];
        if (at >= 0 && e < a.experts) a.slots[t * a.k + at] = before;
        total += part[0] + part[1] + part[2] + part[3];
    }
    s = wave_sum(s);
    if (lane == 0) sums[wave] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        a.counts[e] = total;
        if (e < a.experts) psum[e] = (sums[0] + sums[1]) + (sums[2] + sums[3]);
    }
}

// Offsets and loss: one thread (the experts are few).
template <typename T>
__global__ __launch_bounds__(64) void offsets(RouteArgs<T> a, const float* psum) {
    if (threadIdx.x != 0) return;
    int all = 0;
    float s = 0.f;
    for (int e = 0; e < a.experts; ++e) {
        a.offsets[e] = all;
        all += a.counts[e];
        s += (float)a.counts[e] * psum[e];
    }
    a.offsets[a.experts] = all;
    if (a.loss != nullptr) {
        const float rows = (float)(all > 1 ? all : 1), tokens = (float)(a.counts[a.experts] > 1 ? a.counts[a.experts] : 1);
        *a.loss = (float)a.experts * (s / rows) / tokens;
    }
}

template <typename T>
__global__ __launch_bounds__(256) void place(RouteArgs<T> a) {
    const int64_t all = (int64_t)a.tokens * a.k;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < all; i += (int64_t)gridDim.x * 256) {
        const int e = a.choice[i];
        a.slots[i] = e < 0 ? -1 : a.offsets[e] + a.slots[i];
    }
}

// The gradient, a wave to a token.
template <typename T>
__global__ __launch_bounds__(256) void route_grad(RouteGradArgs<T> a) {
    const int lane = threadIdx.x & 63;
    float all = 0.f;
    for (int e = lane; e < a.experts; e += kLanes) all += (float)a.counts[e];
    all = wave_sum(all);
    const float tokens = (float)a.counts[a.experts];
    const float f = a.dloss != nullptr && all > 0.f ? *a.dloss * (float)a.experts / (all * tokens) : 0.f;
    for (int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); t < a.tokens; t += (int64_t)gridDim.x * 4) {
        const Row r = load_row(a.logits + t * a.ldl, a.experts, lane);
        const float inv = r.sum == 0.f ? 0.f : 1.f / r.sum;
        float p[kPer], g[kPer], d[kPer], chosen = 0.f;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int e = lane + i * kLanes;
            p[i] = expf(r.l[i] - r.m) * inv;
            g[i] = e < a.experts ? f * (float)a.counts[e] : 0.f;
            d[i] = 0.f;
        }
        bool in[kPer] = {};
        for (int j = 0; j < a.k && a.dgates != nullptr; ++j) {
            const int e = a.choice[t * a.k + j];
            const float dg = a.dgates[t * a.k + j];
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                if (e == lane + i * kLanes && e < a.experts) {
                    in[i] = true;
                    d[i] += dg;
                }
        }
        float s = 0.f, sd = 0.f;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            if (in[i] && a.renormalize) {
                chosen += p[i];
                sd += d[i] * p[i];
            } else if (in[i]) {
                g[i] += d[i];
            }
        }
        if (a.renormalize) {
            chosen = wave_sum(chosen);
            sd = wave_sum(sd);
        }
#pragma unroll
        for (int i = 0; i < kPer; ++i) s += g[i] * p[i];
        s = wave_sum(s);
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int e = lane + i * kLanes;
            float out = p[i] * (g[i] - s);
            if (in[i] && a.renormalize && chosen > 0.f) out += p[i] / chosen * (d[i] - sd / chosen);
            if (e < a.experts) {
                if constexpr (sizeof(T) == 4) a.dlogits[t * a.lddl + e] = out;
                else a.dlogits[t * a.lddl + e] = f32_to_bf16(out);
            }
        }
    }
}

template <typename T>
hipError_t launch(const RouteArgs<T>& a, hipStream_t s) {
    float* psum = static_cast<float*>(a.ws);
    float* stats = psum + kMaxExperts;
    const unsigned blocks = grid_for(((int64_t)a.tokens + 3) / 4);
    hipError_t e = launch_kernel(&choose<T>, dim3(blocks), dim3(256), s, a, stats);
    if (e == hipSuccess)
        e = launch_kernel(&count<T>, dim3(a.experts + 1), dim3(256), s, a, static_cast<const float*>(stats), psum);
    if (e == hipSuccess)
        e = launch_kernel(&offsets<T>, dim3(1), dim3(64), s, a, static_cast<const float*>(psum));
    if (e == hipSuccess && a.tokens > 0)
        e = launch_kernel(&place<T>, dim3(grid_for(((int64_t)a.tokens * a.k + 255) / 256)), dim3(256), s, a);
    return e;
}

template <typename T>
hipError_t launch_grad(const RouteGradArgs<T>& a, hipStream_t s) {
    return launch_kernel(&route_grad<T>, dim3(grid_for(((int64_t)a.tokens + 3) / 4)), dim3(256), s, a);
}

}  // namespace

size_t route_workspace(int64_t tokens, int64_t, int) { return (size_t)(kMaxExperts + 2 * tokens) * sizeof(float); }

hipError_t launch_route(const RouteArgs<uint16_t>& a, hipStream_t s) { return launch(a, s); }
hipError_t launch_route(const RouteArgs<float>& a, hipStream_t s) { return launch(a, s); }
hipError_t launch_route_grad(const RouteGradArgs<uint16_t>& a, hipStream_t s) { return launch_grad(a, s); }
hipError_t launch_route_grad(const RouteGradArgs<float>& a, hipStream_t s) { return launch_grad(a, s); }

}  // namespace dg
