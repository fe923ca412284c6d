// Layer norm of the rows of a matrix, and its gradients.
//
//     m = mean(x),  r = 1 / sqrt(mean((x - m)^2) + eps),  y = (x - m) r w + b
//     dx = R + r (g - mean(g) - h mean(g h)),  g = dy w,  h = (x - m) r
//     dw = beta dw + sum over rows of dy h,    db = beta db + sum over rows of dy

#include "layer.hpp"

namespace dg {
namespace {

// Sum over a workgroup of 256 threads, in every thread. `part`: 4 values of LDS.
__device__ __forceinline__ float block_sum(float v, float* part) {
    v = wave_sum(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    return (part[0] + part[1]) + (part[2] + part[3]);
}

// One workgroup to a row, which it reads three times (from the caches after the
// first).
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
        s = 0.f;
        for (int64_t c = (int64_t)threadIdx.x * n; c < a.cols; c += 256 * n) {
            Vec<T> v;
            const int valid = inside(a.cols, c, n);
            v.load(x + c, valid);
#pragma unroll
            for (int e = 0; e < n; ++e) {
                const float d = v.at(e) - m;
                s += e < valid ? d * d : 0.f;
            }
        }
        const float r = 1.f / sqrtf(block_sum(s, part) / (float)a.cols + a.eps);
        if (threadIdx.x == 0) {
            if (a.mean != nullptr) a.mean[row] = m;
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
                const float h = (v.at(e) - m) * r;
                y[e] = __builtin_fmaf(h, a.weight != nullptr ? w.at(e) : 1.f, a.bias != nullptr ? b.at(e) : 0.f);
            }
            v.set(y);
            v.store(a.Y + row * a.ldy + c, valid);
        }
    }
}

// L threads to a row (16, or whole waves), V vectors to a thread: one read of X, whose
// values stay in registers between the mean, the squares and Y.
template <typename T, int L, int V>
__global__ __launch_bounds__(L < 256 ? 256 : L) void norm(NormArgs<T> a) {
    constexpr int n = Vec<T>::n, kThreads = L < 256 ? 256 : L, kGroups = kThreads / L, kWaves = L / 64;
    __shared__ float part[2][kThreads / 64];
    const int t = threadIdx.x, lane = t % L, cols = (int)a.cols;
    const int64_t row0 = (int64_t)blockIdx.x * kGroups + t / L;
    const bool on = row0 < a.rows;                      // kWaves <= 4 rows share no barrier that some skip
    const int64_t row = on ? row0 : a.rows - 1;
    int col[V];
#pragma unroll
    for (int i = 0; i < V; ++i) col[i] = (i * L + lane) * n;
    const LastVec last = last_vec(cols, col[V - 1], n);
    col[V - 1] = last.from;
    Vec<T> x[V], w[V], b[V];
#pragma unroll
    for (int i = 0; i < V; ++i) x[i].load(a.X + row * a.ldx + col[i], n);
    if (a.weight != nullptr) {
#pragma unroll
        for (int i = 0; i < V; ++i) w[i].load(a.weight + col[i], n);
    }
    if (a.bias != nullptr) {
#pragma unroll
        for (int i = 0; i < V; ++i) b[i].load(a.bias + col[i], n);
    }
    const auto row_sum = [&](float v, int turn) {
        if constexpr (L == 16) return sum_of_16(v);
        v = wave_sum(v);
        if constexpr (kWaves > 1) {
            if ((t & 63) == 0) part[turn][t >> 6] = v;
            __syncthreads();
            v = 0.f;
#pragma unroll
            for (int q = 0; q < kWaves; ++q) v += part[turn][t / L * kWaves + q];
        }
        return v;
    };
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int e = 0; e < n; ++e) s += i == V - 1 && e < last.skip ? 0.f : x[i].at(e);
    const float m = row_sum(s, 0) / (float)cols;
    s = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int e = 0; e < n; ++e) {
            const float d = x[i].at(e) - m;
            s = i == V - 1 && e < last.skip ? s : __builtin_fmaf(d, d, s);
        }
    const float r = 1.f / sqrtf(row_sum(s, 1) / (float)cols + a.eps);
    if (!on) return;
    if (lane == 0) {
        if (a.mean != nullptr) a.mean[row] = m;
        if (a.rstd != nullptr) a.rstd[row] = r;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        float y[n];
#pragma unroll
        for (int e = 0; e < n; ++e) {
            y[e] = (x[i].at(e) - m) * r;
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

// dX: one workgroup to a row, read twice.
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

// dweight and dbias: 64 columns to a workgroup, whose 4 waves share the rows.
template <typename T>
__global__ __launch_bounds__(256) void norm_grad_cols(NormGradArgs<T> a) {
    __shared__ float part[2][4][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int64_t c0 = (int64_t)blockIdx.x * 64; c0 < a.cols; c0 += (int64_t)gridDim.x * 64) {
        const int64_t c = c0 + lane;
        float dw = 0.f, db = 0.f;
        if (c < a.cols)
            for (int64_t row = wave; row < a.rows; row += 4) {
                const float dy = elem_f32(a.dY[row * a.lddy + c]);
                db += dy;
                dw += dy * ((elem_f32(a.X[row * a.ldx + c]) - a.mean[row]) * a.rstd[row]);
            }
        __syncthreads();
        part[0][wave][lane] = dw;
        part[1][wave][lane] = db;
        __syncthreads();
        if (wave != 0 || c >= a.cols) continue;
        dw = (part[0][0][lane] + part[0][1][lane]) + (part[0][2][lane] + part[0][3][lane]);
        db = (part[1][0][lane] + part[1][1][lane]) + (part[1][2][lane] + part[1][3][lane]);
        if (a.dweight != nullptr) a.dweight[c] = a.beta == 0.f ? dw : __builtin_fmaf(a.beta, a.dweight[c], dw);
        if (a.dbias != nullptr) a.dbias[c] = a.beta == 0.f ? db : __builtin_fmaf(a.beta, a.dbias[c], db);
    }
}

// Both at once, in one pass over X and dY: L threads to a row (16, or whole
// waves), V vectors to a thread, which keeps the row's values in registers
// between the row's sums and dX, and its columns' sums of dY h and dY in 2 V n
// more. A workgroup of 512 threads takes 512 / L rows at a time and adds its
// threads' column sums up in LDS at the end, into one image of the registers
// for each workgroup; sum_images adds those, in their order.
template <typename T, int L, int V, bool RES>
__global__ __launch_bounds__(512, 2) void norm_grad(NormGradArgs<T> a) {
    constexpr int n = Vec<T>::n, kGroups = 512 / L, kWaves = L / 64;
    constexpr int kImage = V * L * n / 4;                       // f32x4 of one sum
    __shared__ union {
        u32x4 w[V * L];
        f32x4 image[kImage];
    } lds;
    __shared__ float part[2][8][2];
    const int t = threadIdx.x, lane = t % L, group = t / L, wave = t >> 6;
    const int cols = (int)a.cols;
    int col[V];
#pragma unroll
    for (int i = 0; i < V; ++i) col[i] = (i * L + lane) * n;
    const LastVec last = last_vec(cols, col[V - 1], n);
    col[V - 1] = last.from;
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
    __syncthreads();
    float dw[V][n] = {}, db[V][n] = {};
    const float inv = 1.f / (float)cols;
    int turn = 0;
    for (int64_t row0 = (int64_t)blockIdx.x * kGroups; row0 < a.rows; row0 += (int64_t)gridDim.x * kGroups, turn ^= 1) {
        const int64_t row = row0 + group;
        const bool on = row < a.rows;
        Vec<T> x[V], dy[V], res[V];
        float r = 0.f, mr = 0.f, sg = 0.f, sgh = 0.f;
        if (on) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                x[i].load(a.X + row * a.ldx + col[i], n);
                dy[i].load(a.dY + row * a.lddy + col[i], n);
            }
            if constexpr (RES) {
#pragma unroll
                for (int i = 0; i < V; ++i) res[i].load(a.R + row * a.ldr + col[i], n);
            }
            r = a.rstd[row];
            mr = -a.mean[row];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                Vec<T> w;
                w.w = __builtin_bit_cast(decltype(w.w), lds.w[i * L + lane]);
#pragma unroll
                for (int e = 0; e < n; ++e) {
                    const float h = (x[i].at(e) + mr) * r;
                    float d = dy[i].at(e);
                    if (i == V - 1) d = e >= last.skip ? d : 0.f;
                    const float g = d * w.at(e);
                    sg += g;
                    sgh = i == V - 1 && e < last.skip ? sgh : __builtin_fmaf(g, h, sgh);
                    db[i][e] += d;
                    dw[i][e] = i == V - 1 && e < last.skip ? 0.f : __builtin_fmaf(d, h, dw[i][e]);
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
                if ((t & 63) == 0) {
                    part[turn][wave][0] = sg;
                    part[turn][wave][1] = sgh;
                }
                __syncthreads();
                sg = sgh = 0.f;
#pragma unroll
                for (int w = 0; w < kWaves; ++w) {
                    sg += part[turn][group * kWaves + w][0];
                    sgh += part[turn][group * kWaves + w][1];
                }
            }
        }
        if (!on) continue;
        const float c1 = sg * inv, c2 = sgh * inv;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            Vec<T> w;
            w.w = __builtin_bit_cast(decltype(w.w), lds.w[i * L + lane]);
            float out[n];
#pragma unroll
            for (int e = 0; e < n; ++e) {
                const float h = (x[i].at(e) + mr) * r;
                const float in = __builtin_fmaf(-h, c2, __builtin_fmaf(dy[i].at(e), w.at(e), -c1));
                out[e] = __builtin_fmaf(r, in, RES ? res[i].at(e) : 0.f);
            }
            x[i].set(out);
            T* p = a.dX + row * a.lddx + col[i];
            if (i < V - 1 || last.skip == 0) {
                x[i].store(p, n);
            } else {
#pragma unroll
                for (int e = 0; e < n; ++e)
                    if (e >= last.skip) x[i].store1(p + e, e);
            }
        }
    }
    if (a.dweight == nullptr && a.dbias == nullptr) return;
    // Rows of 16 lanes first: their sums meet within the wave.
    constexpr int kSets = L == 16 ? 8 : kGroups;
    const int set = L == 16 ? wave : group;
    if constexpr (L == 16) {
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int e = 0; e < n; ++e) {
                dw[i][e] += __shfl_xor(dw[i][e], 16, 64);
                dw[i][e] += __shfl_xor(dw[i][e], 32, 64);
                db[i][e] += __shfl_xor(db[i][e], 16, 64);
                db[i][e] += __shfl_xor(db[i][e], 32, 64);
            }
    }
    const bool mine = L != 16 || (t & 63) < 16;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        f32x4* image = reinterpret_cast<f32x4*>(a.ws) + ((int64_t)blockIdx.x * 2 + which) * kImage;
        for (int s = 0; s < kSets; ++s) {
            if (kSets > 1) __syncthreads();
            if (set != s || !mine) continue;
#pragma unroll
            for (int i = 0; i < V; ++i)
#pragma unroll
                for (int q = 0; q < n / 4; ++q) {
                    const int at = (i * (n / 4) + q) * L + lane;
                    f32x4 v;
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[e] = which == 0 ? dw[i][4 * q + e] : db[i][4 * q + e];
                    if (s > 0) v += lds.image[at];
                    if (s < kSets - 1) lds.image[at] = v;
                    else image[at] = v;
                }
        }
    }
}

// The workgroups' images added up: 8 f32x4 (128 bytes) of an image to a
// workgroup, whose 32 sets of 8 threads share the images.
template <int n>
__global__ __launch_bounds__(256) void sum_images(const f32x4* images, int count, int L, int V, int cols, float beta,
                                                  float* dweight, float* dbias) {
    __shared__ f32x4 part[32][8];
    const int each = V * L * n / 4, t = threadIdx.x, p = blockIdx.x * 8 + (t & 7);
    f32x4 s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
    for (int b = t >> 3; b < count; b += 32) s += images[(int64_t)b * 2 * each + p];
    part[t >> 3][t & 7] = s;
    __syncthreads();
    if (t >= 8) return;
#pragma unroll
    for (int g = 1; g < 32; ++g) s += part[g][t];
    const int which = p / each, at = p % each;
    const int lane = at % L, i = at / L / (n / 4), q = at / L % (n / 4);
    const int c = (i * L + lane) * n;
    const LastVec last = last_vec(cols, c, n);
    float* out = which == 0 ? dweight : dbias;
    if (out == nullptr) return;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if (4 * q + e < last.skip) continue;
        float* o = out + last.from + 4 * q + e;
        *o = beta == 0.f ? s[e] : __builtin_fmaf(beta, *o, s[e]);
    }
}

// Threads to a row and vectors to a thread of a width: 16 lanes up to 16
// vectors, a wave up to 8 vectors a lane, then 2, 4 and 8 waves; 0 threads: no
// such kernel (rows shorter than a vector, or longer than 4096 of them).
struct Width {
    int lanes, vecs;
};
inline Width width_of(int64_t cols, int n) {
    if (cols < n || cols > 4096 * n) return Width{0, 0};
    const int vecs = (int)((cols + n - 1) / n);
    if (vecs <= 16) return Width{16, 1};
    int lanes = 64;
    while (vecs > lanes * 8) lanes *= 2;
    return Width{lanes, (vecs + lanes - 1) / lanes};
}

constexpr int64_t kMaxNormRows = 1 << 22, kManyRows = 1024;
constexpr int kImages = 256;        // workgroups of norm_grad: one to a compute unit

template <typename T, int L, int V>
hipError_t launch_fused(const NormGradArgs<T>& a, unsigned blocks, hipStream_t s) {
    return a.R != nullptr ? launch_kernel(&norm_grad<T, L, V, true>, dim3(blocks), dim3(512), s, a)
                          : launch_kernel(&norm_grad<T, L, V, false>, dim3(blocks), dim3(512), s, a);
}

template <typename T>
hipError_t launch_grad(const NormGradArgs<T>& a, hipStream_t s) {
    constexpr int n = Vec<T>::n;
    const bool columns = a.dweight != nullptr || a.dbias != nullptr;
    const Width w = width_of(a.cols, n);
    if (w.lanes == 0 || a.rows == 0) {
        // The columns first: dX may take dY's place.
        if (columns) {
            const hipError_t e = launch_kernel(&norm_grad_cols<T>, dim3(grid_for((a.cols + 63) / 64)), dim3(256), s, a);
            if (e != hipSuccess) return e;
        }
        if (a.rows == 0) return hipSuccess;
        return launch_kernel(&norm_grad_rows<T>, dim3(grid_for(a.rows)), dim3(256), s, a);
    }
    const int groups = 512 / w.lanes;
    const int64_t want = (a.rows + groups - 1) / groups;
    const unsigned blocks = (unsigned)(want < kImages ? want : kImages);
    hipError_t e = hipErrorInvalidConfiguration;
    switch (w.lanes * 16 + w.vecs) {
        case 16 * 16 + 1: e = launch_fused<T, 16, 1>(a, blocks, s); break;
#define DG_WIDTH(L, V) case L * 16 + V: e = launch_fused<T, L, V>(a, blocks, s); break;
        DG_WIDTH(64, 1) DG_WIDTH(64, 2) DG_WIDTH(64, 3) DG_WIDTH(64, 4)
        DG_WIDTH(64, 5) DG_WIDTH(64, 6) DG_WIDTH(64, 7) DG_WIDTH(64, 8)
        DG_WIDTH(128, 5) DG_WIDTH(128, 6) DG_WIDTH(128, 7) DG_WIDTH(128, 8)
        DG_WIDTH(256, 5) DG_WIDTH(256, 6) DG_WIDTH(256, 7) DG_WIDTH(256, 8)
        DG_WIDTH(512, 5) DG_WIDTH(512, 6) DG_WIDTH(512, 7) DG_WIDTH(512, 8)
#undef DG_WIDTH
    }
    if (e != hipSuccess || !columns) return e;
    const int each = w.vecs * w.lanes * n / 4;
    return launch_kernel(&sum_images<n>, dim3((unsigned)(2 * each / 8)), dim3(256), s,
                         reinterpret_cast<const f32x4*>(a.ws), (int)blocks, w.lanes, w.vecs, (int)a.cols, a.beta,
                         a.dweight, a.dbias);
}

// An image is at most the columns rounded up to 8 x 512 values (bf16 at 512
// lanes), twice, for each workgroup; sized alike for both types.
size_t workspace(int64_t rows, int64_t cols) {
    size_t most = 256;
    for (int n : {Vec<uint16_t>::n, Vec<float>::n}) {
        const Width w = width_of(cols, n);
        if (w.lanes == 0) continue;
        const int groups = 512 / w.lanes;
        const int64_t want = (rows + groups - 1) / groups;
        const size_t bytes = (size_t)(want < kImages ? want : kImages) * 2 * w.vecs * w.lanes * n * sizeof(float);
        most = bytes > most ? bytes : most;
    }
    return most;
}

template <typename T, int L, int V>
hipError_t launch_rows(const NormArgs<T>& a, hipStream_t s) {
    constexpr int kThreads = L < 256 ? 256 : L, kGroups = kThreads / L;
    return launch_kernel(&norm<T, L, V>, dim3((unsigned)((a.rows + kGroups - 1) / kGroups)), dim3(kThreads), s, a);
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
    if (a.cols < n || vecs > 8 * 1024 || a.rows > kMaxNormRows)
        return launch_kernel(&norm_rows<T>, dim3(grid_for(a.rows)), dim3(256), s, a);
    if (vecs <= 16) return launch_rows<T, 16, 1>(a, s);
    // A wave to a row where the rows fill the card, more lanes where they don't.
    const int v = (int)vecs, most = a.rows >= kManyRows ? 8 : 1;
    if (v <= 64 * most) return launch_rows<T, 64>(a, v, s);
    if (v <= 256 * most) return launch_rows<T, 256>(a, v, s);
    return launch_rows<T, 1024>(a, v, s);
}

}  // namespace

size_t layernorm_grad_workspace(int64_t rows, int64_t cols) { return workspace(rows, cols); }

hipError_t launch_layernorm(const NormArgs<uint16_t>& a, int, hipStream_t s) { return launch_norm(a, s); }
hipError_t launch_layernorm(const NormArgs<float>& a, int, hipStream_t s) { return launch_norm(a, s); }
hipError_t launch_layernorm_grad(const NormGradArgs<uint16_t>& a, hipStream_t s) { return launch_grad(a, s); }
hipError_t launch_layernorm_grad(const NormGradArgs<float>& a, hipStream_t s) { return launch_grad(a, s); }

}  // namespace dg
