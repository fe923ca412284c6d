// Dropout whose mask is drawn from a counter wherever it is needed and never
// stored: Y = R + (u >= t ? X * 65536 / (65536 - t) : 0).
//
// u comes from Philox 4x32 with 10 rounds: each round multiplies two of the four
// counter words by constants, and the high halves, the other two words and the
// key are combined by exclusive or. One draw gives 8 columns 16 bits each: the
// chance to be dropped is a multiple of 2^-16, and the factor of what is kept is
// exactly its inverse, so that the mean is kept too.

#include "layer.hpp"

namespace dg {
namespace {


__device__ __forceinline__ u32x4 philox(uint32_t c0, uint32_t c1, uint32_t c2, uint32_t c3, uint64_t seed) {
    uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t a = (uint64_t)c0 * 0xD2511F53u, b = (uint64_t)c2 * 0xCD9E8D57u;
        const uint32_t n0 = (uint32_t)(b >> 32) ^ c1 ^ k0, n2 = (uint32_t)(a >> 32) ^ c3 ^ k1;
        c1 = (uint32_t)b;
        c3 = (uint32_t)a;
        c0 = n0;
        c2 = n2;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return u32x4{c0, c1, c2, c3};
}

// 8 columns to a thread.
template <typename T>
__global__ __launch_bounds__(256) void dropout(DropoutArgs<T> a, float scale) {
    constexpr int n = Vec<T>::n, per = 8 / n;
    const uint64_t seed = a.rng[0], offset = a.rng[1];
    const int64_t eights = (a.cols + 7) / 8, all = eights * a.rows;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < all; i += (int64_t)gridDim.x * 256) {
        const int64_t row = i / eights, col8 = i - row * eights;
        const u32x4 u = philox((uint32_t)col8, (uint32_t)row, (uint32_t)offset, (uint32_t)(offset >> 32), seed);
#pragma unroll
        for (int h = 0; h < per; ++h) {
            const int64_t c = col8 * 8 + h * n;
            const int valid = inside(a.cols, c, n);
            if (valid == 0) continue;
            Vec<T> x, r;
            x.load(a.X + row * a.ldx + c, valid);
            if (a.R != nullptr) r.load(a.R + row * a.ldr + c, valid);
            float y[n];
#pragma unroll
            for (int e = 0; e < n; ++e) {
                const int j = h * n + e;
                const uint32_t bits = (j & 1) ? u[j >> 1] >> 16 : u[j >> 1] & 0xffffu;
                y[e] = bits >= a.drop ? x.at(e) * scale : 0.f;
                if (a.R != nullptr) y[e] += r.at(e);
            }
            x.set(y);
            x.store(a.Y + row * a.ldy + c, valid);
        }
    }
}

template <typename T>
hipError_t launch(const DropoutArgs<T>& a, hipStream_t s) {
    const int64_t units = (a.cols + 7) / 8 * a.rows;
    const float scale = a.drop >= 65536 ? 0.f : 65536.f / (float)(65536 - a.drop);
    return launch_kernel(&dropout<T>, dim3(grid_for((units + 255) / 256)), dim3(256), s, a, scale);
}

}  // namespace

hipError_t launch_dropout(const DropoutArgs<uint16_t>& a, hipStream_t s) { return launch(a, s); }
hipError_t launch_dropout(const DropoutArgs<float>& a, hipStream_t s) { return launch(a, s); }

}  // namespace dg
