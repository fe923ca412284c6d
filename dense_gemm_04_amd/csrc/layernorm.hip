// Layer norm of the rows of a matrix, and its gradients.
//
//     m = mean(x),  r = 1 / sqrt(mean((x - m)^2) + eps),  y = (x - m) r w + b
//     dx = R + r (g - mean(g) - h mean(g h)),  g = dy w,  h = (x - m) r
//     dw = beta dw + sum over rows of dy h,    db = beta db + sum over rows of dy
//
// Bound by memory: X is read once and Y written once, X, dY (and R) read and dX
// written once, with every value in registers between a row's sums and its
// result. The second pass over the registers sums the differences from the first
// one's mean beside their squares: what the mean lost in its sum and in rounding
// to fp32 goes into y and the variance, so that rows far from zero come out as
// exact as others (4096 columns around 4096, spread 1: y off by 5.6e-4 without it,
// 5.6e-7 with it). The gradients take the mean rounded to fp32. Rows whose columns
// are not whole vectors read their last n columns again, at whatever alignment,
// and count each once.
//
// One MI355X: the norm of 8192 x 4096 bf16 26 us (5.2 TB/s; a copy of as much
// 26.5), its gradients with a residual 52 us and 5 for the last sums (4.7 TB/s over
// all); 262144 x 128 bf16 28 and, with a residual, 52 us; 16 x 8192 bf16 3.6 us.

#include "layer.hpp"

namespace dg {
namespace {

// s / cols as rounded, from inv = 1 / cols: the rest of the first quotient is exact.
__device__ __forceinline__ float over_cols(float s, float cols, float inv) {
    const float q = s * inv;
    return __builtin_fmaf(__builtin_fmaf(-q, cols, s), inv, q);
}

// What is left of a row's mean after its first estimate m, and 1 / the deviation, from the
// means of x - m and of their squares.
struct Rest {
    float mean, rstd, least;
    __device__ __forceinline__ Rest(float rest, float squares, float eps) : mean(rest) {
        const float var = squares - mean * mean;
        rstd = 1.f / sqrtf((var < 0.f ? 0.f : var) + eps);          // a NaN stays
        least = var * 0x1p-40f;
    }
    // Up to 2^-20 of the deviation the rest may come from the roundings of the differences
    // and of their sum, and near zero the first sum is the more exact one (bf16 4096 columns around
    // 0: the mean off by 4e-8 of itself, 1.5e-6 with the rest on top).
    __device__ __forceinline__ float full_mean(float m) const { return mean * mean <= least ? m : m + mean; }
};

// Sum over a workgroup of 256 threads, in every thread. `part`: 4 values of LDS.
__device__ __forceinline__ float block_sum(float v, float* part) {
    v = wave_sum(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    return (part[0] + part[1]) + (part[2] + part[3]);
}

// Rows of any width: one workgroup to a row, which it reads three times (from the
// caches after the first). For rows shorter than a vector or longer than the
// kernel below takes.
template <typename T>
__global__ __launch_bounds__(256) void norm_rows(NormArgs<T> a) {
    constexpr int n = Vec<T>::n;
    __shared__ float part[4];
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const T* x = a.X + row * a.ldx;
        float s = 0.f;
        for (int64_t c = (int64_t)threadIdx.x * n; c < a.cols; c += 256 * n) {
            Vec<T> v;
            v.load(x + c, inside(a.cols, c, n));
#pragma unroll
            for (int e = 0; e < n; ++e) s += v.at(e);
        }
        const float m = block_sum(s, part) / (float)a.cols;
        double all = 0.;                     // of any number of vectors
        float sq = 0.f;
        for (int64_t c = (int64_t)threadIdx.x * n; c < a.cols; c += 256 * n) {
            Vec<T> v;
            const int valid = inside(a.cols, c, n);
            v.load(x + c, valid);
            float sd = 0.f;
#pragma unroll
            for (int e = 0; e < n; ++e) {
                const float d = v.at(e) - m;
                sd += e < valid ? d : 0.f;
                sq += e < valid ? d * d : 0.f;
            }
            all += (double)sd;
        }
        const float sd = block_sum((float)all, part) / (float)a.cols;
        const Rest rest(sd, block_sum(sq, part) / (float)a.cols, a.eps);
        const float r = rest.rstd, shift = -rest.mean * r;
        if (threadIdx.x == 0) {
            if (a.mean != nullptr) a.mean[row] = rest.full_mean(m);
            if (a.rstd != nullptr) a.rstd[row] = r;
        }
        for (int64_t c = (int64_t)threadIdx.x * n; c < a.cols; c += 256 * n) {
            Vec<T> v, w, b;
            const int valid = inside(a.cols, c, n);
            v.load(x + c, valid);
            if (a.weight != nullptr) w.load(a.weight + c, valid);
            if (a.bias != nullptr) b.load(a.bias + c, valid);
            float y[n];
#pragma unroll
            for (int e = 0; e < n; ++e) {
                const float h = __builtin_fmaf(v.at(e) - m, r, shift);
                y[e] = __builtin_fmaf(h, a.weight != nullptr ? w.at(e) : 1.f, a.bias != nullptr ? b.at(e) : 0.f);
            }
            v.set(y);
            v.store(a.Y + row * a.ldy + c, valid);
        }
    }
}

// L threads to a row (16, or whole waves), V vectors to a thread: one read of X, whose
// values stay in registers between the mean, the squares and Y. A wave to a row
// needs no barrier. inv: 1 / columns.
template <typename T, int L, int V>
__global__ __launch_bounds__(L < 256 ? 256 : L) void norm(NormArgs<T> a, float inv) {
    constexpr int n = Vec<T>::n, kThreads = L < 256 ? 256 : L, kGroups = kThreads / L, kWaves = L / 64;
    __shared__ float part[kThreads / 64];
    __shared__ float2 parts[kThreads / 64];
    const int t = threadIdx.x, lane = t % L, cols = (int)a.cols;
    const int64_t row0 = (int64_t)blockIdx.x * kGroups + t / L;
    const bool on = row0 < a.rows;                      // the others go along to the end
    const int64_t row = on ? row0 : a.rows - 1;
    int col[V];
#pragma unroll
    for (int i = 0; i < V; ++i) col[i] = (i * L + lane) * n;
    const LastVec last = last_vec(cols, col[V - 1], n);
    col[V - 1] = last.from;
    Vec<T> x[V], w[V], b[V];
#pragma unroll
    for (int i = 0; i < V; ++i) x[i].load(a.X + row * a.ldx + col[i], n);
    // Weight and bias are on their way beside X where the 128 registers of 1024
    // threads hold all three; where they would spill, they come after the sums
    // (1024 x 65536 bf16 98 us, 124 with spilled registers; 512 x 49160 30 and 40).
    constexpr bool kLate = kThreads == 1024 && sizeof(T) == 2 && V > 6;
    const auto load_columns = [&] {
        if (a.weight != nullptr) {
#pragma unroll
            for (int i = 0; i < V; ++i) w[i].load(a.weight + col[i], n);
        }
        if (a.bias != nullptr) {
#pragma unroll
            for (int i = 0; i < V; ++i) b[i].load(a.bias + col[i], n);
        }
    };
    if constexpr (!kLate) load_columns();
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int e = 0; e < n; ++e) s += i == V - 1 && e < last.skip ? 0.f : x[i].at(e);
    s = L == 16 ? sum_of_16(s) : wave_sum(s);
    if constexpr (kWaves > 1) {
        if ((t & 63) == 0) part[t >> 6] = s;
        lds_only_barrier();                      // weight and bias stay on their way
        s = 0.f;
#pragma unroll
        for (int q = 0; q < kWaves; ++q) s += part[t / L * kWaves + q];
    }
    const float m = over_cols(s, (float)cols, inv);
    float sd = 0.f, sq = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int e = 0; e < n; ++e) {
            const float d = x[i].at(e) - m;
            const bool skip = i == V - 1 && e < last.skip;
            sd += skip ? 0.f : d;
            sq = skip ? sq : __builtin_fmaf(d, d, sq);
        }
    if constexpr (L == 16) {
        sd = sum_of_16(sd);
        sq = sum_of_16(sq);
    } else {
        wave_sums(sd, sq);
    }
    if constexpr (kWaves > 1) {
        if ((t & 63) == 0) parts[t >> 6] = float2{sd, sq};
        lds_only_barrier();
        sd = sq = 0.f;
#pragma unroll
        for (int q = 0; q < kWaves; ++q) {
            sd += parts[t / L * kWaves + q].x;
            sq += parts[t / L * kWaves + q].y;
        }
    }
    const Rest rest(sd * inv, over_cols(sq, (float)cols, inv), a.eps);
    const float r = rest.rstd, shift = -rest.mean * r;
    if (!on) return;
    if (lane == 0) {
        if (a.mean != nullptr) a.mean[row] = rest.full_mean(m);
        if (a.rstd != nullptr) a.rstd[row] = r;
    }
    if constexpr (kLate) load_columns();
#pragma unroll
    for (int i = 0; i < V; ++i) {
        float y[n];
#pragma unroll
        for (int e = 0; e < n; ++e) {
            y[e] = __builtin_fmaf(x[i].at(e) - m, r, shift);
            if (a.weight != nullptr) y[e] *= w[i].at(e);
            if (a.bias != nullptr) y[e] += b[i].at(e);
        }
        x[i].set(y);
        T* p = a.Y + row * a.ldy + col[i];
        if (i < V - 1 || last.skip == 0) {
            x[i].store(p, n);
        } else {
#pragma unroll
            for (int e = 0; e < n; ++e)
                if (e >= last.skip) x[i].store1(p + e, e);
        }
    }
}

// The gradients of rows of any width, in two kernels. dX: one workgroup to a row,
// read twice.
template <typename T>
__global__ __launch_bounds__(256) void norm_grad_rows(NormGradArgs<T> a) {
    constexpr int n = Vec<T>::n;
    __shared__ float part[4];
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const float m = a.mean[row], r = a.rstd[row];
        float sg = 0.f, sgh = 0.f;
        for (int pass = 0; pass < 2; ++pass) {
            for (int64_t c = (int64_t)threadIdx.x * n; c < a.cols; c += 256 * n) {
                Vec<T> x, dy, w, res;
                const int valid = inside(a.cols, c, n);
                x.load(a.X + row * a.ldx + c, valid);
                dy.load(a.dY + row * a.lddy + c, valid);
                if (a.weight != nullptr) w.load(a.weight + c, valid);
                float out[n];
                if (pass == 1 && a.R != nullptr) res.load(a.R + row * a.ldr + c, valid);
#pragma unroll
                for (int e = 0; e < n; ++e) {
                    const float h = (x.at(e) - m) * r, g = dy.at(e) * (a.weight != nullptr ? w.at(e) : 1.f);
                    if (pass == 0) {
                        sg += g;
                        sgh += e < valid ? g * h : 0.f;
                    } else {
                        out[e] = r * (g - sg - h * sgh) + (a.R != nullptr ? res.at(e) : 0.f);
                    }
                }
                if (pass == 1) {
                    x.set(out);
                    x.store(a.dX + row * a.lddx + c, valid);
                }
            }
            if (pass == 0) {
                sg = block_sum(sg, part) / (float)a.cols;
                sgh = block_sum(sgh, part) / (float)a.cols;
            }
        }
    }
}

__device__ __forceinline__ void add_to(float* out, float beta, float v) {
    *out = beta == 0.f ? v : __builtin_fmaf(beta, *out, v);
}

// dweight and dbias of such rows: P columns to a workgroup, whose 256 / P rows of
// threads share its slice of the rows (blockIdx.y). The sums are taken in 64 bits,
// since a column may have millions of terms (262144 x 5: fp32 chains of 65536 were off by
// more than 3 steps of the terms' sum). Slices leave theirs in the workspace, P values
// of dweight and P of dbias each. 262144 x 5 bf16 0.58 ms with both kernels, 11 in one
// slice; 1024 x 40000 without R 114 us, 190 with a row at a time.
template <typename T, int P>
__global__ __launch_bounds__(256) void norm_grad_cols(NormGradArgs<T> a) {
    constexpr int kRows = 256 / P;
    __shared__ double part[2][kRows][P];
    const int lane = threadIdx.x % P, first = threadIdx.x / P;
    const int64_t slice = (a.rows + gridDim.y - 1) / gridDim.y, lo = blockIdx.y * slice;
    const int64_t hi = lo + slice < a.rows ? lo + slice : a.rows;
    for (int64_t c0 = (int64_t)blockIdx.x * P; c0 < a.cols; c0 += (int64_t)gridDim.x * P) {
        const int64_t c = c0 + lane;
        double dw = 0., db = 0.;
        if (c < a.cols) {
#pragma unroll 4
            for (int64_t row = lo + first; row < hi; row += kRows) {
                const float dy = elem_f32(a.dY[row * a.lddy + c]);
                const float h = (elem_f32(a.X[row * a.ldx + c]) - a.mean[row]) * a.rstd[row];
                db += (double)dy;
                dw += (double)dy * (double)h;
            }
        }
        __syncthreads();
        part[0][first][lane] = dw;
        part[1][first][lane] = db;
        __syncthreads();
        if (first != 0) continue;
#pragma unroll
        for (int q = 1; q < kRows; ++q) {
            dw += part[0][q][lane];
            db += part[1][q][lane];
        }
        if (gridDim.y > 1) {
            double* to = reinterpret_cast<double*>(a.ws) + (int64_t)blockIdx.y * 2 * P + lane;
            to[0] = dw;
            to[P] = db;
        } else if (c < a.cols) {
            if (a.dweight != nullptr) add_to(a.dweight + c, a.beta, (float)dw);
            if (a.dbias != nullptr) add_to(a.dbias + c, a.beta, (float)db);
        }
    }
}

// The slices of rows shorter than a vector added up, by one workgroup.
constexpr int kShort = 8;           // columns, and more than such rows have
constexpr int kMostSlices = 256;    // one to a compute unit
__global__ __launch_bounds__(256) void sum_slices(const double* slices, int count, int cols, float beta, float* dweight,
                                                  float* dbias) {
    constexpr int kWidth = 2 * kShort, kSets = 256 / kWidth;
    __shared__ double part[kSets][kWidth];
    const int at = threadIdx.x % kWidth, set = threadIdx.x / kWidth;
    double s = 0.;
    for (int b = set; b < count; b += kSets) s += slices[b * kWidth + at];
    part[set][at] = s;
    __syncthreads();
    if (set != 0) return;
#pragma unroll
    for (int q = 1; q < kSets; ++q) s += part[q][at];
    float* out = at < kShort ? dweight : dbias;
    if (out != nullptr && at % kShort < cols) add_to(out + at % kShort, beta, (float)s);
}
// Rows shorter than a vector fill one workgroup's columns, so the rows are shared out.
inline int slices_of(int64_t rows, int64_t cols) {
    if (cols >= kShort) return 1;
    const int64_t want = (rows + 1023) / 1024;
    return (int)(want < 1 ? 1 : (want < kMostSlices ? want : kMostSlices));
}

// Both at once, in one pass over X and dY: L threads to a row (16, or whole
// waves), V vectors to a thread, which keeps the row's values in registers
// between the row's sums and dX, and its columns' sums of dY h and dY in 2 V n
// more. PRE: the next row is on its way meanwhile (8192 x 4096 bf16 with a residual:
// 52 us with 32 values of a row to a thread and the next one on its way, 62 with 64
// and without). A workgroup of 512 threads takes
// 512 / L rows at a time and adds its threads' column sums up in LDS at the end,
// into one image of the registers for each workgroup; sum_images adds those.
template <typename T, int V, bool RES>
struct RowOf {
    Vec<T> x[V], dy[V], res[RES ? V : 1];
    float r, m;
    __device__ __forceinline__ void load(const NormGradArgs<T>& a, int64_t row, const int* col) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            x[i].load(a.X + row * a.ldx + col[i], Vec<T>::n);
            dy[i].load(a.dY + row * a.lddy + col[i], Vec<T>::n);
            if constexpr (RES) res[i].load(a.R + row * a.ldr + col[i], Vec<T>::n);
        }
        r = a.rstd[row];
        m = a.mean[row];
    }
    // Waits for every load of the row: a volatile statement that takes their
    // results and stays ahead of the barrier after it.
    __device__ __forceinline__ void landed() const {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            asm volatile("" ::"v"(x[i].w), "v"(dy[i].w));
            if constexpr (RES) asm volatile("" ::"v"(res[i].w));
        }
    }
};

template <typename T, int L, int V, bool RES, bool PRE>
__global__ __launch_bounds__(512, 2) void norm_grad(NormGradArgs<T> a) {
    constexpr int n = Vec<T>::n, kGroups = 512 / L, kWaves = L / 64;
    constexpr int kSets = L == 16 ? 8 : kGroups;                // of column sums, after the lanes of a wave have met
    constexpr int kImage = V * L * n / 4;                       // f32x4 of one sum
    __shared__ union {
        u32x4 w[V * L];
        f32x4 image[kSets > 1 ? kSets / 2 : 1][kSets > 1 ? 2 * kImage : 1];
    } lds;
    __shared__ float part[2][8][2];
    // Uniform in a wave, and kept in scalar registers, where a row has whole waves.
    const int t = threadIdx.x, lane = t % L, wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int group = L == 16 ? t / L : wave / (kWaves > 0 ? kWaves : 1);
    const int cols = (int)a.cols;
    int col[V];
#pragma unroll
    for (int i = 0; i < V; ++i) col[i] = (i * L + lane) * n;
    const LastVec last = last_vec(cols, col[V - 1], n);
    col[V - 1] = last.from;
    const int64_t step = (int64_t)gridDim.x * kGroups;
    int64_t row0 = (int64_t)blockIdx.x * kGroups, row = row0 + group;
    RowOf<T, V, RES> now;
    if (PRE && row < a.rows) now.load(a, row, col);
    if (group == 0) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            Vec<T> w;
            if (a.weight != nullptr) {
                w.load(a.weight + col[i], n);
            } else {
                float one[n];
#pragma unroll
                for (int e = 0; e < n; ++e) one[e] = 1.f;
                w.set(one);
            }
            lds.w[i * L + lane] = __builtin_bit_cast(u32x4, w.w);
        }
    }
    lds_only_barrier();
    float dw[V][n] = {}, db[V][n] = {};
    const float inv = 1.f / (float)cols;
    int turn = 0;
    // One row in each group, or (`on`) in some: the waves of a row meet in it.
    // Every lane stores whole vectors: where the last ones of a row overlap, they
    // hold the same bits. With that a turn's loads and stores are the same in
    // number on every path, and the wait for a row's loads leaves the
    // stores before and the loads after them in flight. dX may be dY or R, so
    // all the row's loads have to land before any wave stores to it: each wave
    // waits for its own before the barrier, which orders LDS alone.
    const auto one = [&](bool on) {
        float sg = 0.f, sgh = 0.f;
        if (on) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                Vec<T> w;
                w.w = __builtin_bit_cast(decltype(w.w), lds.w[i * L + lane]);
#pragma unroll
                for (int e = 0; e < n; ++e) {
                    const bool skip = i == V - 1 && e < last.skip;
                    const float h = (now.x[i].at(e) - now.m) * now.r;
                    const float d = now.dy[i].at(e), g = d * w.at(e);
                    sg += skip ? 0.f : g;
                    sgh = skip ? sgh : __builtin_fmaf(g, h, sgh);
                    db[i][e] += skip ? 0.f : d;
                    dw[i][e] = skip ? 0.f : __builtin_fmaf(d, h, dw[i][e]);
                }
            }
        }
        if constexpr (L == 16) {
            sg = sum_of_16(sg);
            sgh = sum_of_16(sgh);
        } else {
            sg = wave_sum(sg);
            sgh = wave_sum(sgh);
            if constexpr (kWaves > 1) {
                now.landed();
                if ((t & 63) == 0) {
                    part[turn][wave][0] = sg;
                    part[turn][wave][1] = sgh;
                }
                lds_only_barrier();
                sg = sgh = 0.f;
#pragma unroll
                for (int w = 0; w < kWaves; ++w) {
                    sg += part[turn][group * kWaves + w][0];
                    sgh += part[turn][group * kWaves + w][1];
                }
            }
        }
        turn ^= 1;
        if (!on) return;
        const float c1 = sg * inv, c2 = sgh * inv;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            // Unpacked again: the values of the first pass would take registers that spill.
            asm volatile("" : "+v"(now.x[i].w), "+v"(now.dy[i].w));
            Vec<T> w;
            w.w = __builtin_bit_cast(decltype(w.w), lds.w[i * L + lane]);
            float out[n];
#pragma unroll
            for (int e = 0; e < n; ++e) {
                const float h = (now.x[i].at(e) - now.m) * now.r;
                const float in = __builtin_fmaf(-h, c2, __builtin_fmaf(now.dy[i].at(e), w.at(e), -c1));
                out[e] = __builtin_fmaf(now.r, in, RES ? now.res[RES ? i : 0].at(e) : 0.f);
            }
            w.set(out);
            w.store(a.dX + row * a.lddx + col[i], n);
        }
    };
    for (; row0 + kGroups <= a.rows; row0 += step, row += step) {
        RowOf<T, V, RES> next;
        if constexpr (PRE) next.load(a, row + step < a.rows ? row + step : row, col);
        else now.load(a, row, col);
        one(true);
        if constexpr (PRE) now = next;
    }
    if (row0 < a.rows) {
        const bool on = row < a.rows;
        if (!PRE && on) now.load(a, row, col);
        one(on);
    }
    if (a.dweight == nullptr && a.dbias == nullptr) return;
    // The sets of column sums meet two by two.
    const int set = L == 16 ? wave : group;
    if constexpr (L == 16) {
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int e = 0; e < n; ++e) {
                dw[i][e] = add_lanes<32>(add_lanes<16>(dw[i][e]));
                db[i][e] = add_lanes<32>(add_lanes<16>(db[i][e]));
            }
    }
    const bool mine = L != 16 || (t & 63) < 16;
    const auto each = [&](auto&& f) {
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int q = 0; q < n / 4; ++q) {
                const int at = (i * (n / 4) + q) * L + lane;
                f(at, &dw[i][4 * q]);
                f(kImage + at, &db[i][4 * q]);
            }
    };
#pragma unroll
    for (int half = kSets / 2; half > 0; half /= 2) {
        lds_only_barrier();
        if (set >= half && set < 2 * half && mine)
            each([&](int at, const float* v) { lds.image[set - half][at] = f32x4{v[0], v[1], v[2], v[3]}; });
        lds_only_barrier();
        if (set < half && mine)
            each([&](int at, float* v) {
                const f32x4 o = lds.image[set][at];
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] += o[e];
            });
    }
    if (set != 0 || !mine) return;
    if (gridDim.x > 1) {
        f32x4* image = reinterpret_cast<f32x4*>(a.ws) + (int64_t)blockIdx.x * 2 * kImage;
        each([&](int at, const float* v) { image[at] = f32x4{v[0], v[1], v[2], v[3]}; });
        return;
    }
    // The only workgroup.
    const auto out = [&](float* to, const float* v, int i) {
        if (to == nullptr) return;
#pragma unroll
        for (int q = 0; q < n / 4; ++q) {
            float* p = to + col[i] + 4 * q;
            if (i < V - 1 || last.skip == 0) {
                f32x4 w = {v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
                if (a.beta != 0.f) {
                    const f32x4 o = *reinterpret_cast<const f32x4_a4*>(p);
#pragma unroll
                    for (int e = 0; e < 4; ++e) w[e] = __builtin_fmaf(a.beta, o[e], w[e]);
                }
                *reinterpret_cast<f32x4_a4*>(p) = w;
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (4 * q + e >= last.skip) add_to(p + e, a.beta, v[4 * q + e]);
            }
        }
    };
#pragma unroll
    for (int i = 0; i < V; ++i) {
        out(a.dweight, dw[i], i);
        out(a.dbias, db[i], i);
    }
}

// The workgroups' images added up: 4 f32x4 of an image to a workgroup, whose 64
// sets of 4 threads share the images.
template <int n>
__global__ __launch_bounds__(256) void sum_images(const f32x4* images, int count, int L, int V, int cols, float beta,
                                                  float* dweight, float* dbias) {
    __shared__ f32x4 part[64][4];
    const int each = V * L * n / 4, t = threadIdx.x, p = blockIdx.x * 4 + (t & 3);
    f32x4 s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int b = t >> 2; b < count; b += 64) s += images[(int64_t)b * 2 * each + p];
    part[t >> 2][t & 3] = s;
    __syncthreads();
    if (t >= 32) return;
#pragma unroll
    for (int g = 1; g < 8; ++g) s += part[(t >> 2) + 8 * g][t & 3];
    part[t >> 2][t & 3] = s;
    lds_wave_barrier();
    if (t >= 4) return;
#pragma unroll
    for (int g = 1; g < 8; ++g) s += part[g][t];
    const int which = p / each, at = p % each;
    const int lane = at % L, i = at / L / (n / 4), q = at / L % (n / 4);
    const LastVec last = last_vec(cols, (i * L + lane) * n, n);
    float* out = which == 0 ? dweight : dbias;
    if (out == nullptr) return;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if (4 * q + e < last.skip) continue;
        add_to(out + last.from + 4 * q + e, beta, s[e]);
    }
}

// Threads to a row and vectors to a thread: 16 lanes up to 16 vectors; then as few
// waves as hold the row in 32 values a thread; up to 64 in 8 waves. 0 threads: no such
// kernel (rows shorter than a vector, or longer than 32768 values in bf16, 16384 in fp32).
// Above 20480 values of bf16 registers spill. With a residual, 1024 rows of 20480, 24576, 28672 and
// 32768 take 58, 72, 111 and 154 us, the general kernels 84, 92, 100 and 107; 16 rows 13, 15, 19
// and 23 against 21, 24, 28 and 31; 4096 rows 148, 183, 338 and 456 against 320, 365, 411 and 452.
// fp32 does not spill (1024 x 16384 75 us, 104).
struct Width {
    int lanes, vecs;
};
inline Width width_of(int64_t cols, int n) {
    const int64_t vecs = (cols + n - 1) / n;
    if (cols < n || vecs > 512 * 8) return Width{0, 0};
    if (vecs <= 16) return Width{16, 1};
    int lanes = 64;
    while (lanes < 512 && vecs * n > lanes * 32) lanes *= 2;
    return Width{lanes, (int)((vecs + lanes - 1) / lanes)};
}

constexpr int64_t kManyRows = 512;
constexpr int kImages = 256;        // workgroups of norm_grad: one to a compute unit
// One alone up to two turns, where a second launch costs as much as the second turn
// or more, and a call less (bf16, two turns, alone and in two launches: 64 x 64 4.8
// and 6.0 us, 16 x 1024 5.8 and 6.8, 8 x 4096 9.05 and 9.0; four turns: 16 x 4096 14.1 and 9.1).
inline int64_t grad_blocks(int64_t rows, const Width& w) {
    const int groups = 512 / w.lanes;
    if (rows <= 2 * groups) return 1;
    const int64_t want = (rows + groups - 1) / groups;
    return want < kImages ? want : kImages;
}

template <typename T, int L, int V>
hipError_t launch_fused(const NormGradArgs<T>& a, unsigned blocks, hipStream_t s) {
    // Two rows (8 or, with R, 12 registers a vector) and the column sums fit 256
    // registers beside the rest.
    constexpr int kSums = 2 * V * Vec<T>::n;
    constexpr bool kPre = kSums <= 64, kPreRes = kPre && 24 * V + kSums <= 200;
    return a.R != nullptr ? launch_kernel(&norm_grad<T, L, V, true, kPreRes>, dim3(blocks), dim3(512), s, a)
                          : launch_kernel(&norm_grad<T, L, V, false, kPre>, dim3(blocks), dim3(512), s, a);
}
// The widths that width_of gives for L lanes: above a half of 32 values a thread
// (from one vector on with a single wave), with 8 waves up to 64.
template <typename T, int L, int V = L == 64 ? 1 : 16 / Vec<T>::n + 1>
hipError_t launch_fused(const NormGradArgs<T>& a, int vecs, unsigned blocks, hipStream_t s) {
    if (vecs == V) return launch_fused<T, L, V>(a, blocks, s);
    if constexpr (V < (L == 512 ? 8 : 32 / Vec<T>::n)) return launch_fused<T, L, V + 1>(a, vecs, blocks, s);
    return hipErrorInvalidConfiguration;
}

template <typename T>
hipError_t launch_grad(const NormGradArgs<T>& a, hipStream_t s) {
    constexpr int n = Vec<T>::n;
    const bool columns = a.dweight != nullptr || a.dbias != nullptr;
    const Width w = width_of(a.cols, n);
    if (w.lanes == 0 || a.rows == 0) {
        // The columns first: dX may take dY's place.
        if (columns) {
            const int slices = slices_of(a.rows, a.cols);
            hipError_t e = a.cols < kShort
                ? launch_kernel(&norm_grad_cols<T, kShort>, dim3(1, (unsigned)slices), dim3(256), s, a)
                : launch_kernel(&norm_grad_cols<T, 64>, dim3(grid_for((a.cols + 63) / 64)), dim3(256), s, a);
            if (e == hipSuccess && slices > 1)
                e = launch_kernel(&sum_slices, dim3(1), dim3(256), s, reinterpret_cast<const double*>(a.ws), slices,
                                  (int)a.cols, a.beta, a.dweight, a.dbias);
            if (e != hipSuccess) return e;
        }
        if (a.rows == 0) return hipSuccess;
        return launch_kernel(&norm_grad_rows<T>, dim3(grid_for(a.rows)), dim3(256), s, a);
    }
    const unsigned blocks = (unsigned)grad_blocks(a.rows, w);
    hipError_t e = hipErrorInvalidConfiguration;
    if (w.lanes == 16) e = launch_fused<T, 16, 1>(a, blocks, s);
    if (w.lanes == 64) e = launch_fused<T, 64>(a, w.vecs, blocks, s);
    if (w.lanes == 128) e = launch_fused<T, 128>(a, w.vecs, blocks, s);
    if (w.lanes == 256) e = launch_fused<T, 256>(a, w.vecs, blocks, s);
    if (w.lanes == 512) e = launch_fused<T, 512>(a, w.vecs, blocks, s);
    if (e != hipSuccess || !columns || blocks == 1) return e;
    const int each = w.vecs * w.lanes * n / 4;
    return launch_kernel(&sum_images<n>, dim3((unsigned)(2 * each / 4)), dim3(256), s,
                         reinterpret_cast<const f32x4*>(a.ws), (int)blocks, w.lanes, w.vecs, (int)a.cols, a.beta,
                         a.dweight, a.dbias);
}

// An image is at most the columns rounded up to 8 x 512 values (bf16 at 512
// lanes), twice, for each workgroup; sized alike for both types.
size_t workspace(int64_t rows, int64_t cols) {
    size_t most = 256;
    const int slices = slices_of(rows, cols);
    if (slices > 1) most = (size_t)slices * 2 * kShort * sizeof(double);
    for (int n : {Vec<uint16_t>::n, Vec<float>::n}) {
        const Width w = width_of(cols, n);
        if (w.lanes == 0) continue;
        const size_t bytes = (size_t)grad_blocks(rows, w) * 2 * w.vecs * w.lanes * n * sizeof(float);
        most = bytes > most ? bytes : most;
    }
    return most;
}

template <typename T>
hipError_t launch_general(const NormArgs<T>& a, hipStream_t s) {
    return launch_kernel(&norm_rows<T>, dim3(grid_for(a.rows)), dim3(256), s, a);
}
template <typename T, int L, int V>
hipError_t launch_rows(const NormArgs<T>& a, hipStream_t s) {
    constexpr int kThreads = L < 256 ? 256 : L, kGroups = kThreads / L;
    const int64_t blocks = (a.rows + kGroups - 1) / kGroups;
    if (blocks * kThreads > INT32_MAX) return launch_general(a, s);       // past what a launch takes
    return launch_kernel(&norm<T, L, V>, dim3((unsigned)blocks), dim3(kThreads), s, a, 1.f / (float)a.cols);
}
template <typename T, int L>
hipError_t launch_rows(const NormArgs<T>& a, int vecs, hipStream_t s) {
    switch ((vecs + L - 1) / L) {
        case 1: return launch_rows<T, L, 1>(a, s);
        case 2: return launch_rows<T, L, 2>(a, s);
        case 3: return launch_rows<T, L, 3>(a, s);
        case 4: return launch_rows<T, L, 4>(a, s);
        case 5: return launch_rows<T, L, 5>(a, s);
        case 6: return launch_rows<T, L, 6>(a, s);
        case 7: return launch_rows<T, L, 7>(a, s);
        case 8: return launch_rows<T, L, 8>(a, s);
    }
    return hipErrorInvalidConfiguration;
}

template <typename T>
hipError_t launch_norm(const NormArgs<T>& a, hipStream_t s) {
    constexpr int n = Vec<T>::n;
    const int64_t vecs = (a.cols + n - 1) / n;
    if (a.cols < n || vecs > 8 * 1024) return launch_general(a, s);
    if (vecs <= 16) return launch_rows<T, 16, 1>(a, s);
    // Up to 8 vectors to a thread where the rows fill the card, 2 where they don't
    // (bf16, inputs in the caches, 2 and 8: 256 rows of 4096 3.2 and 4.2 us, 512 rows 5.1
    // and 4.5, 4096 rows 25.8 and 13.1; 4096 rows of 8192 27.6 and 21.7).
    const int v = (int)vecs, most = a.rows >= kManyRows ? 8 : 2;
    if (v <= 64 * most) return launch_rows<T, 64>(a, v, s);
    if (v <= 256 * most) return launch_rows<T, 256>(a, v, s);
    return launch_rows<T, 1024>(a, v, s);
}

}  // namespace

size_t layernorm_grad_workspace(int64_t rows, int64_t cols) { return workspace(rows, cols); }

hipError_t launch_layernorm(const NormArgs<uint16_t>& a, hipStream_t s) { return launch_norm(a, s); }
hipError_t launch_layernorm(const NormArgs<float>& a, hipStream_t s) { return launch_norm(a, s); }
hipError_t launch_layernorm_grad(const NormGradArgs<uint16_t>& a, hipStream_t s) { return launch_grad(a, s); }
hipError_t launch_layernorm_grad(const NormGradArgs<float>& a, hipStream_t s) { return launch_grad(a, s); }

}  // namespace dg
