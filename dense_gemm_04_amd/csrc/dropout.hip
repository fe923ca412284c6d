// Dropout whose mask is drawn from a counter wherever it is needed and never
// stored: Y = R + (u >= t ? X * 65536 / (65536 - t) : 0).
//
// u comes from Philox 4x32 with 10 rounds: each round multiplies two of the four
// counter words by constants, and the high halves, the other two words and the
// key are combined by exclusive or. One draw gives 8 columns 16 bits each: the
// chance to be dropped is a multiple of 2^-16, and the factor of what is kept is
// exactly its inverse, so that the mean is kept too.
//
// Bound by memory: 8192 x 4096 bf16 with a residual 38 us (5.3 TB/s), of which the
// 180 vector instructions a thread, mostly the generator's, fill 19.

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

// A vector of 16 bytes to a thread, so that a wave reads and writes whole
// stretches: in fp32 two threads draw the same numbers and use half of them each
// (4095 x 1023 in fp32: 7.7 us, 9.0 with 8 columns to a thread, 32 bytes from lane to
// lane). I: the type that counts vectors.
template <typename T, typename I>
__global__ __launch_bounds__(256) void dropout(DropoutArgs<T> a, float scale, I vecs, I all) {
    constexpr int n = Vec<T>::n;
    const uint64_t seed = a.rng[0], offset = a.rng[1];
    for (I i = (I)blockIdx.x * 256 + threadIdx.x; i < all; i += (I)gridDim.x * 256) {
        const I row = i / vecs, v = i - row * vecs;
        const int64_t c = (int64_t)v * n;
        const int valid = inside(a.cols, c, n);
        Vec<T> x, r;
        x.load(a.X + (int64_t)row * a.ldx + c, valid);
        if (a.R != nullptr) r.load(a.R + (int64_t)row * a.ldr + c, valid);
        const u32x4 w = philox((uint32_t)(c / 8), (uint32_t)row, (uint32_t)offset, (uint32_t)(offset >> 32), seed);
        const bool second = c % 8 != 0;
        float y[n];
#pragma unroll
        for (int e = 0; e < n; ++e) {
            const uint32_t word = n == 8 ? w[e >> 1] : (second ? w[2 + (e >> 1 & 1)] : w[e >> 1]);
            const uint32_t u = (e & 1) ? word >> 16 : word & 0xffffu;
            y[e] = u >= a.drop ? x.at(e) * scale : 0.f;
            if (a.R != nullptr) y[e] += r.at(e);
        }
        x.set(y);
        x.store(a.Y + (int64_t)row * a.ldy + c, valid);
    }
}

template <typename T>
hipError_t launch(const DropoutArgs<T>& a, hipStream_t s) {
    constexpr int n = Vec<T>::n;
    const int64_t vecs = (a.cols + n - 1) / n, all = vecs * a.rows;
    const float scale = a.drop >= 65536 ? 0.f : 65536.f / (float)(65536 - a.drop);
    const dim3 grid(grid_for((all + 255) / 256));
    // 32 bits where the last step past the end stays inside them (8192 x 4096 bf16
    // 21.9 us with its input in the caches, 22.5 with a 64-bit division).
    if (all + (int64_t)grid.x * 256 <= (int64_t)UINT32_MAX)
        return launch_kernel(&dropout<T, uint32_t>, grid, dim3(256), s, a, scale, vecs, all);
    return launch_kernel(&dropout<T, int64_t>, grid, dim3(256), s, a, scale, vecs, all);
}

}  // namespace

hipError_t launch_dropout(const DropoutArgs<uint16_t>& a, hipStream_t s) { return launch(a, s); }
hipError_t launch_dropout(const DropoutArgs<float>& a, hipStream_t s) { return launch(a, s); }

}  // namespace dg
