// 8-bit floating point (OCP e4m3) helpers and kernel arguments shared by the
// quantiser and the block-scaled product.
#pragma once

#include "common.hpp"

namespace dg {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));

constexpr float kE4m3Max = 448.f;
constexpr int kScaleBlock = 128;             // values of K that share a scale
// Below this a block's largest magnitude no longer shrinks its scale, which
// therefore stays a normal number (2^-126).
constexpr float kMinTop = 0x1.cp-118f;       // 448 * 2^-126

// C <- act(alpha * sum_b SA(b,i) SB(b, j / b_rows) sum_{k in b} A(i,k) B(j,k)
//          + bias[j]) + beta * C; SA(b,i) = SA[b * ldsa + i], SB alike.
// Every kernel forms SA SB in fp32 and adds the block's sum times it in one
// fused step, so that scales at the ends of fp32's range give the same values
// whatever kernel the alignment chooses. (Scaling in two steps, or by mantissas
// and exponents where the product leaves the normal numbers, would hold a wider
// range: the first doubles the vector work of the tiles, the second's branch
// spills 42 to 215 registers of the two largest.)
struct Fp8Args {
    int64_t M, N, K;
    float alpha, beta;
    const uint8_t* A; int64_t lda;
    const float* SA; int64_t ldsa;
    const uint8_t* B; int64_t ldb;
    const float* SB; int64_t ldsb;
    int b_rows;                              // rows of B per scale: 1 or 128
    uint16_t* C; int64_t ldc;
    const uint16_t* bias;
    int act;
};

// One 16 x 16 block over 128 values of K: lane p + 16 g supplies 32 bytes of
// row p of `x` and of `y`, and receives D(row 4 g + r of x, row p of y) in
// register r. Which k a byte position means is free as long as both operands
// agree. The instruction aligns the products of each 8 k to the largest of
// them and keeps 13 bits below it (measured on in-range operands): a sum is
// within 8 * 2^-13 = 2^-10 of the sum of its terms' magnitudes at worst, which
// can exceed bf16's half step where the terms cancel. Measured over K of
// 1040 to 4100, normal values: 4.4e-5 to 6.1e-5 of C, root-mean-square, where
// rounding C to bf16 gives 1.7e-3. Everything after a block, over blocks, is fp32.
__device__ __forceinline__ f32x4 mfma_fp8(i32x8 x, i32x8 y) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
}

__device__ __forceinline__ i32x8 join16(u32x4 lo, u32x4 hi) {
    return i32x8{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
}

// Zeros the bytes at positions >= keep of a 16-byte chunk.
__device__ __forceinline__ u32x4 mask_bytes(u32x4 v, int keep) {
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        const int b = keep - 4 * w;
        v[w] &= b >= 4 ? ~0u : (b <= 0 ? 0u : (1u << (8 * b)) - 1u);
    }
    return v;
}

// Columns col .. col + 3 of one row of C: v[] holds alpha times the product.
// `wide`: C's rows (and base) are 8-byte aligned.
template <bool EPI>
__device__ __forceinline__ void store_c4(uint16_t* crow, int64_t col, int64_t N, float beta, const uint16_t* bias,
                                         int act, f32x4 v, bool wide) {
    if constexpr (EPI) {
#pragma unroll
        for (int r = 0; r < 4; ++r)
            v[r] = activate(v[r] + ((bias != nullptr && col + r < N) ? bf16_to_f32(bias[col + r]) : 0.f), act);
    }
    if (wide && col + 4 <= N) {
        u32x2* dst = reinterpret_cast<u32x2*>(crow + col);
        if (beta != 0.f) {
            const u32x2 c0 = *dst;
#pragma unroll
            for (int r = 0; r < 4; ++r) v[r] += beta * bf16_to_f32((uint16_t)(c0[r >> 1] >> (16 * (r & 1))));
        }
        *dst = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
        return;
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        if (col + r >= N) continue;
        float x = v[r];
        if (beta != 0.f) x += beta * bf16_to_f32(crow[col + r]);
        crow[col + r] = f32_to_bf16(x);
    }
}

}  // namespace dg
