// 8-bit block-scaled product for operands of any alignment: the same sums as
// the aligned kernels, each element loaded by itself.
//
//   C(i,j) = alpha sum_b SA(b,i) SB(b,j) sum_{k in b} A(i,k) B(j,k)   (+ epilogue)
//
// One workgroup of 4 waves per 64 x 64 tile, each wave a 32 x 32 quarter; K in
// blocks of 128, the block that shares a scale: its product (one
// v_mfma_f32_16x16x128_f8f6f4 per 16 x 16) is scaled by SA SB, formed first and
// in fp32 as in the aligned kernels, and added to the accumulator. B is the instruction's first operand, so a lane holds 4
// consecutive columns of one row of C. Elements past M, N and K are zeros.

#include "bf16_lds.hpp"
#include "fp8.hpp"
#include "ops.hpp"

namespace dg {
namespace {

constexpr int kT = 64;

// Byte offset of 16-byte chunk c of a 128-byte row (see bf16lds::a_off).
__device__ __forceinline__ int chunk_off(int row, int c) { return row * 128 + ((c ^ (row & 7)) << 4); }

__device__ __forceinline__ void load_tile(const uint8_t* X, int64_t ld, int64_t row0, int64_t rows, int64_t k0,
                                          int64_t K, uint8_t* dst, int t) {
    // 16 consecutive bytes of a row per thread and pass.
    for (int q = t; q < kT * 8; q += 256) {
        const int row = q >> 3, c = q & 7;
        u32x4 w = {0u, 0u, 0u, 0u};
        if (row0 + row < rows) {
            const uint8_t* p = X + (row0 + row) * ld + k0 + 16 * c;
            const int64_t left = K - k0 - 16 * c;
#pragma unroll
            for (int e = 0; e < 16; ++e)
                if (e < left) w[e >> 2] |= (uint32_t)p[e] << (8 * (e & 3));
        }
        *reinterpret_cast<u32x4*>(dst + chunk_off(row, c)) = w;
    }
}

template <bool EPI>
__global__ __launch_bounds__(256) void gemm_fp8_general_kernel(Fp8Args p, int tiles_m, int tiles_n) {
    __shared__ __attribute__((aligned(16))) uint8_t As[kT * 128], Bs[kT * 128];
    int tm, tn;
    tile_coords(blockIdx.x, gridDim.x, tiles_m, tiles_n, 4, tm, tn);
    const int64_t m0 = (int64_t)tm * kT, n0 = (int64_t)tn * kT;
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    const int pl = lane & 15, g = lane >> 4;
    const int wm = (wave >> 1) * 32, wn = (wave & 1) * 32;
    f32x4 acc[2][2];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i) acc[j][i] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int64_t nk = (p.K + kScaleBlock - 1) / kScaleBlock;
    for (int64_t kb = 0; kb < nk; ++kb) {
        __syncthreads();
        load_tile(p.A, p.lda, m0, p.M, kb * kScaleBlock, p.K, As, t);
        load_tile(p.B, p.ldb, n0, p.N, kb * kScaleBlock, p.K, Bs, t);
        __syncthreads();
        i32x8 fa[2], fb[2];
        float sa[2];
        f32x4 sb[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int ra = wm + 16 * i + pl, rb = wn + 16 * i + pl;
            fa[i] = join16(*reinterpret_cast<const u32x4*>(As + chunk_off(ra, g)),
                           *reinterpret_cast<const u32x4*>(As + chunk_off(ra, g + 4)));
            fb[i] = join16(*reinterpret_cast<const u32x4*>(Bs + chunk_off(rb, g)),
                           *reinterpret_cast<const u32x4*>(Bs + chunk_off(rb, g + 4)));
            sa[i] = m0 + ra < p.M ? p.SA[kb * p.ldsa + m0 + ra] : 0.f;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int64_t col = n0 + wn + 16 * i + 4 * g + r;
                sb[i][r] = col < p.N ? p.SB[kb * p.ldsb + (p.b_rows == 1 ? col : col / 128)] : 0.f;
            }
        }
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const f32x4 d = mfma_fp8(fb[j], fa[i]);
#pragma unroll
                for (int r = 0; r < 4; ++r) acc[j][i][r] = __builtin_fmaf(d[r], sa[i] * sb[j][r], acc[j][i][r]);
            }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int64_t row = m0 + wm + 16 * i + pl;
        if (row >= p.M) continue;
#pragma unroll
        for (int j = 0; j < 2; ++j)
            store_c4<EPI>(p.C + row * p.ldc, n0 + wn + 16 * j + 4 * g, p.N, p.beta, p.bias, p.act, p.alpha * acc[j][i],
                          false);
    }
}

}  // namespace

hipError_t launch_fp8_general(const Fp8Args& a, hipStream_t s) {
    const int64_t tm = (a.M + kT - 1) / kT, tn = (a.N + kT - 1) / kT;
    if (tm * tn > kMaxGrid) return hipErrorInvalidConfiguration;
    const bool epi = a.bias != nullptr || a.act != kActNone;
    return launch_kernel(epi ? &gemm_fp8_general_kernel<true> : &gemm_fp8_general_kernel<false>,
                         dim3((unsigned)(tm * tn)), dim3(256), s, a, tm, tn);
}

}  // namespace dg
