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

template <typename T>
hipError_t launch_grad(const NormGradArgs<T>& a, hipStream_t s) {
    // The columns first: dX may take dY's place.
    if (a.dweight != nullptr || a.dbias != nullptr) {
        const hipError_t e = launch_kernel(&norm_grad_cols<T>, dim3(grid_for((a.cols + 63) / 64)), dim3(256), s, a);
        if (e != hipSuccess) return e;
    }
    if (a.rows == 0) return hipSuccess;
    return launch_kernel(&norm_grad_rows<T>, dim3(grid_for(a.rows)), dim3(256), s, a);
}

}  // namespace

size_t layernorm_grad_workspace(int64_t, int64_t) { return 256; }

hipError_t launch_layernorm(const NormArgs<uint16_t>& a, int, hipStream_t s) {
    return launch_kernel(&norm_rows<uint16_t>, dim3(grid_for(a.rows)), dim3(256), s, a);
}
hipError_t launch_layernorm(const NormArgs<float>& a, int, hipStream_t s) {
    return launch_kernel(&norm_rows<float>, dim3(grid_for(a.rows)), dim3(256), s, a);
}
hipError_t launch_layernorm_grad(const NormGradArgs<uint16_t>& a, hipStream_t s) { return launch_grad(a, s); }
hipError_t launch_layernorm_grad(const NormGradArgs<float>& a, hipStream_t s) { return launch_grad(a, s); }

}  // namespace dg
