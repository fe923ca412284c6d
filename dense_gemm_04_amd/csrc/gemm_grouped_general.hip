// Products grouped by expert, and their weight gradients, for operands of any
// alignment: the same sums as the aligned kernels, each element loaded by
// itself. fp32 accumulation, one rounding at the end.
//
//   rows:  C(i,:) = act(alpha row_scale[i] A(i,:) B_e + bias_e) + beta C(i,:), i in group e
//   wgrad: C_e = alpha A_e^T B_e + beta C_e
//
// One workgroup of 4 waves per 64 x 64 tile, each wave a 32 x 32 quarter.
// Both operands are addressed as X(row, k) = X[row * rs + k * ks] with one of
// the strides 1, and staged k-contiguous in LDS. The group of a tile is found
// on the GPU (rows), or is part of the tile's number (wgrad); a group without
// rows has no row tiles, and its gradient is beta C_e.

#include <type_traits>

#include "bf16_lds.hpp"
#include "ops.hpp"

namespace dg {
namespace {

using namespace bf16lds;
constexpr int kT = 64;

__device__ __forceinline__ void load_tile(const uint16_t* X, int64_t rs, int64_t ks, int64_t rows, int64_t ks_left,
                                          uint16_t* dst, int t) {
    for (int q = t; q < kT * kBK; q += 256) {
        // Neighbouring threads along the operand's contiguous dimension.
        const int row = ks == 1 ? q >> 6 : q & 63, k = ks == 1 ? q & 63 : q >> 6;
        uint16_t v = 0;
        if (row < rows && k < ks_left) v = X[row * rs + k * ks];
        dst[a_off(row, k >> 3) + (k & 7)] = v;
    }
}

template <bool WGRAD, bool F32>
__global__ __launch_bounds__(256) void gemm_grouped_general_kernel(GroupedArgs p, int tiles_m, int tiles_n) {
    using CT = std::conditional_t<F32, float, uint16_t>;
    __shared__ __attribute__((aligned(16))) uint16_t As[kT * kBK], Bs[kT * kBK];
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    const int pl = lane & 15, g = lane >> 4;
    const int wm = (wave >> 1) * 32, wn = (wave & 1) * 32;
    const int tn = (int)blockIdx.x % tiles_n, rt = (int)blockIdx.x / tiles_n;
    const int64_t n0 = (int64_t)tn * kT, N = p.N;
    int e;
    int64_t rows, depth, ars, aks, brs, bks;           // rows of this tile of C; k's
    const uint16_t *A, *B;
    CT* C;
    const float* row_scale = nullptr;
    if constexpr (WGRAD) {
        e = rt / tiles_m;
        const int64_t m0 = (int64_t)(rt % tiles_m) * kT;
        int lo, hi;
        group_range(p.offsets, e, (int)p.M, lo, hi);
        rows = p.K - m0;
        depth = hi - lo;
        A = p.A + lo * p.lda + m0; ars = 1; aks = p.lda;
        B = p.B + lo * p.ldb + n0; brs = 1; bks = p.ldb;
        C = static_cast<CT*>(p.C) + e * p.stridec + m0 * p.ldc;
    } else {
        const RowTile w = find_row_tile(p.offsets, p.groups, (int)p.M, kT, rt, lane);
        if (w.group < 0) return;
        e = w.group;
        rows = w.end - w.m0;
        depth = p.K;
        A = p.A + w.m0 * p.lda; ars = p.lda; aks = 1;
        B = p.B + e * p.strideb + (p.tb ? n0 * p.ldb : n0);
        brs = p.tb ? p.ldb : 1; bks = p.tb ? 1 : p.ldb;
        C = static_cast<CT*>(p.C) + w.m0 * p.ldc;
        if (p.row_scale != nullptr) row_scale = p.row_scale + w.m0;
    }
    f32x4 acc[2][2];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i) acc[j][i] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int64_t k0 = 0; k0 < depth; k0 += kBK) {
        __syncthreads();
        load_tile(A + k0 * aks, ars, aks, rows, depth - k0, As, t);
        load_tile(B + k0 * bks, brs, bks, N - n0, depth - k0, Bs, t);
        __syncthreads();
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
            bf16x8 fa[2], fb[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                fa[i] = *reinterpret_cast<const bf16x8*>(As + a_off(wm + 16 * i + pl, 4 * ks + g));
                fb[i] = *reinterpret_cast<const bf16x8*>(Bs + a_off(wn + 16 * i + pl, 4 * ks + g));
            }
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    acc[j][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fb[j], fa[i], acc[j][i], 0, 0, 0);
        }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int64_t row = wm + 16 * i + pl;
        if (row >= rows) continue;
        const float alpha = WGRAD && depth == 0 ? 0.f : p.alpha;       // an empty sum is 0, also times inf
        const float fr = row_scale != nullptr ? alpha * row_scale[row] : alpha;
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int64_t col = n0 + wn + 16 * j + 4 * g + r;
                if (col >= N) continue;
                CT* c = C + row * p.ldc + col;
                float v = fr * acc[j][i][r];
                if constexpr (!WGRAD) {
                    if (p.bias != nullptr) v += bf16_to_f32(p.bias[e * p.stridebias + col]);
                    v = activate(v, p.act);
                }
                if (p.beta != 0.f) v += p.beta * elem_f32(*c);
                if constexpr (F32) *c = v;
                else *c = f32_to_bf16(v);
            }
    }
}

}  // namespace

hipError_t launch_grouped_general(const GroupedArgs& a, hipStream_t s) {
    const int64_t tn = (a.N + kT - 1) / kT;
    const int64_t tm = a.wgrad ? (a.K + kT - 1) / kT : row_tiles_bound(a.M, a.groups, kT);
    const int64_t grid = a.wgrad ? a.groups * tm * tn : tm * tn;
    if (grid > kMaxGrid) return hipErrorInvalidConfiguration;
    auto fn = !a.wgrad ? &gemm_grouped_general_kernel<false, false>
              : a.f32  ? &gemm_grouped_general_kernel<true, true>
                       : &gemm_grouped_general_kernel<true, false>;
    return launch_kernel(fn, dim3((unsigned)grid), dim3(256), s, a, tm, tn);
}

}  // namespace dg
