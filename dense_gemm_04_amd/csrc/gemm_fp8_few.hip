// 8-bit block-scaled product with few rows or few tiles, rows aligned to 16 bytes:
//
//   C(i,j) = alpha sum_b SA(b,i) SB(b, j / b_rows) sum_{k in b} A(i,k) B(j,k)   (+ epilogue)
//
// One workgroup per tile of 16 MF x 16 NF; its NW waves each compute the whole
// tile over every NW-th block of 128 k, and their partial tiles are added in
// wave order at the end. Both operands run along k, so a lane's 32 bytes of an
// MFMA operand are two 16-byte loads from global memory into registers: no LDS
// and no barrier in the loop, and with D blocks of loads in flight per wave a CU
// keeps 16 KB or more on the way.

#include "fp8.hpp"
#include "ops.hpp"

namespace dg {
namespace {

template <int MF, int NF, int NW, int D, bool EPI, bool B1>
__global__ __launch_bounds__(NW * 64) void gemm_fp8_few_kernel(Fp8Args p, int tiles_m, int tiles_n) {
    constexpr uint32_t kNowhere = 0x80000000u;       // past the end of every descriptor: loads give zeros
    __shared__ __attribute__((aligned(16))) f32x4 red[NW * NF * MF * 64];
    const int64_t M = p.M, N = p.N, K = p.K, lda = p.lda, ldb = p.ldb;
    int tm, tn;
    tile_coords(blockIdx.x, gridDim.x, tiles_m, tiles_n, 4, tm, tn);
    const int64_t m0 = (int64_t)tm * (16 * MF), n0 = (int64_t)tn * (16 * NF);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int pl = lane & 15, g = lane >> 4;
    const int nk = (int)((K + kScaleBlock - 1) / kScaleBlock);
    const int kr = (int)(K - (int64_t)(nk - 1) * kScaleBlock);

    const int64_t rows_a = M - m0 < 16 * MF ? M - m0 : 16 * MF, rows_b = N - n0 < 16 * NF ? N - n0 : 16 * NF;
    const rsrc_t da = make_rsrc(p.A + m0 * lda, (uint32_t)(((rows_a - 1) * lda + K + 15) & ~(int64_t)15));
    const rsrc_t db = make_rsrc(p.B + n0 * ldb, (uint32_t)(((rows_b - 1) * ldb + K + 15) & ~(int64_t)15));
    const uint32_t va = (uint32_t)(pl * lda + 16 * g), vb = (uint32_t)(pl * ldb + 16 * g);
    const int64_t scales_b = B1 ? rows_b : 1;
    const float* SB = p.SB + (B1 ? n0 : n0 / 128);

    u32x4 fa[D][MF][2], fb[D][NF][2];
    float sa[D][MF];
    f32x4 sb[D][B1 ? NF : 1];
    auto load = [&](int d, int kb) __attribute__((always_inline)) {
        const bool in = kb < nk;
        const uint32_t s0 = in ? (uint32_t)kb * 128u : kNowhere;
#pragma unroll
        for (int j = 0; j < NF; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h) fb[d][j][h] = buf_load16(db, vb + 64 * h + (uint32_t)(16 * j * ldb), s0);
#pragma unroll
        for (int i = 0; i < MF; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) fa[d][i][h] = buf_load16(da, va + 64 * h + (uint32_t)(16 * i * lda), s0);
        const int row = in ? kb : 0;
        const rsrc_t ra = make_rsrc(p.SA + row * p.ldsa + m0, in ? (uint32_t)(rows_a * 4) : 0u);
        const rsrc_t rb = make_rsrc(SB + row * p.ldsb, in ? (uint32_t)(scales_b * 4) : 0u);
#pragma unroll
        for (int i = 0; i < MF; ++i)
            sa[d][i] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(ra, 4 * (16 * i + pl), 0, 0));
        if constexpr (B1) {
#pragma unroll
            for (int j = 0; j < NF; ++j) sb[d][j] = __builtin_bit_cast(f32x4, buf_load16(rb, 4 * (16 * j + 4 * g), 0));
        } else {
            sb[d][0][0] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(rb, 0, 0, 0));
        }
    };
    f32x4 acc[NF][MF];
#pragma unroll
    for (int j = 0; j < NF; ++j)
#pragma unroll
        for (int i = 0; i < MF; ++i) acc[j][i] = f32x4{0.f, 0.f, 0.f, 0.f};
    auto compute = [&](int d, int kb) __attribute__((always_inline)) {
        if (kb == nk - 1 && kr < kScaleBlock) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int i = 0; i < MF; ++i) fa[d][i][h] = mask_bytes(fa[d][i][h], kr - 16 * g - 64 * h);
#pragma unroll
                for (int j = 0; j < NF; ++j) fb[d][j][h] = mask_bytes(fb[d][j][h], kr - 16 * g - 64 * h);
            }
        }
#pragma unroll
        for (int i = 0; i < MF; ++i) {
            const i32x8 x = join16(fa[d][i][0], fa[d][i][1]);
            const float s = B1 ? sa[d][i] : sa[d][i] * sb[d][0][0];
#pragma unroll
            for (int j = 0; j < NF; ++j) {
                const f32x4 v = mfma_fp8(join16(fb[d][j][0], fb[d][j][1]), x);
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    acc[j][i][r] = __builtin_fmaf(v[r], B1 ? s * sb[d][j][r] : s, acc[j][i][r]);
            }
        }
    };
#pragma unroll
    for (int d = 0; d < D; ++d) load(d, wave + NW * d);
    for (int kb = wave; kb < nk; kb += NW * D) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
            compute(d, kb + NW * d);
            load(d, kb + NW * (D + d));
        }
    }

    // Partial tiles: value (j, i) of lane l of wave w at ((w NF + j) MF + i) 64 + l.
#pragma unroll
    for (int j = 0; j < NF; ++j)
#pragma unroll
        for (int i = 0; i < MF; ++i) red[((wave * NF + j) * MF + i) * 64 + lane] = acc[j][i];
    __syncthreads();
    for (int q = wave; q < NF * MF; q += NW) {
        const int j = q / MF, i = q % MF;
        f32x4 sum = red[q * 64 + lane];
#pragma unroll
        for (int w = 1; w < NW; ++w) sum += red[(w * NF * MF + q) * 64 + lane];
        const int64_t row = m0 + 16 * i + pl;
        if (row < M)
            store_c4<EPI>(p.C + row * p.ldc, n0 + 16 * j + 4 * g, N, p.beta, p.bias, p.act, p.alpha * sum, true);
    }
}

template <int MF, int NF, int NW, int D>
hipError_t launch_cfg(const Fp8Args& a, hipStream_t s) {
    const int64_t tm = (a.M + 16 * MF - 1) / (16 * MF), tn = (a.N + 16 * NF - 1) / (16 * NF);
    if (tm * tn > kMaxGrid) return hipErrorInvalidConfiguration;
    const bool epi = a.bias != nullptr || a.act != kActNone, b1 = a.b_rows == 1;
    auto fn = epi ? (b1 ? &gemm_fp8_few_kernel<MF, NF, NW, D, true, true> : &gemm_fp8_few_kernel<MF, NF, NW, D, true, false>)
                  : (b1 ? &gemm_fp8_few_kernel<MF, NF, NW, D, false, true>
                        : &gemm_fp8_few_kernel<MF, NF, NW, D, false, false>);
    return launch_kernel(fn, dim3((unsigned)(tm * tn)), dim3(NW * 64), s, a, tm, tn);
}

}  // namespace

// M <= 32. Tiles of 16 or 32 columns: the wider ones read A half as often,
// the narrower ones are twice as many. 32 columns run where they make one round
// that fills more than half of the 256 CUs (129 to 256 tiles). One MI355X, us with 16 and with 32
// columns: 16 x 8192^2 18.0 and 14.2, 16 x 4096 x 8192 10.5 and 13.9, 5 x 12288 x
// 4096 12.3 and 13.5; 32 x 8192^2 27.7 and 17.9, 32 x 4096^2 9.4 and 10.7.
hipError_t launch_fp8_few(const Fp8Args& a, hipStream_t s) {
    const bool wide = a.N > 4096 && a.N <= 8192;
    if (a.M <= 16) return wide ? launch_cfg<1, 2, 8, 2>(a, s) : launch_cfg<1, 1, 8, 2>(a, s);
    return wide ? launch_cfg<2, 2, 8, 2>(a, s) : launch_cfg<2, 1, 8, 4>(a, s);
}

}  // namespace dg
