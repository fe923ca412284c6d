// Products grouped by expert whose groups have few rows (a decoding step), rows
// aligned to 16 bytes:
//
//   C(i,:) = act(alpha row_scale[i] A(i,:) op(B_e) + bias_e) + beta C(i,:), i in group e
//
// Bound by reading the matrices of the experts that have rows. One workgroup
// of 4 waves per tile of 16 MF rows by 64 columns; each wave computes the
// whole tile over its own quarter of K, with two LDS stages of its own that it
// fills with LDS-destined 128-bit copies and waits for by its own count: no
// barrier in the loop, and the 4 waves keep 4 slabs of 64 k on the way. Their
// partial tiles are added in wave order at the end.
//
// Layouts, edges and the search for a tile's group as in the tiled kernel
// (gemm_grouped.hip).

#include "bf16_lds.hpp"
#include "ops.hpp"

namespace dg {
namespace {

using namespace bf16lds;
constexpr int kN = 64;                       // columns of a tile
constexpr int kW = 4;                        // waves, one range of K each

template <int MF, bool TB, bool EPI>
__global__ __launch_bounds__(kW * 64) void gemm_grouped_few_kernel(GroupedArgs p, int tiles_n) {
    constexpr int kRows = 16 * MF;
    constexpr int kA = kRows * kBK, kB = kN * kBK;            // bf16 elements of a slab
    constexpr int kACopies = kA * 2 / 1024, kBCopies = kB * 2 / 1024;
    constexpr int kStage = kA + kB;
    __shared__ __attribute__((aligned(16))) uint16_t lds[kW * 2 * kStage];
    static_assert(kW * MF * 4 * 64 * 16 <= kW * 2 * kStage * 2, "partial tiles fit the stages");

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int pl = lane & 15, g = lane >> 4;
    int lo = 0, hi = 0;
    if (lane < p.groups) group_range(p.offsets, lane, (int)p.M, lo, hi);
    const RowPlace w = place_row_tile(p.offsets, p.groups, (int)p.M, kRows, tiles_n, 8, lo, hi, lane);
    if (w.tile.group < 0) return;
    const int e = w.tile.group, m0 = w.tile.m0;
    const int64_t n0 = (int64_t)w.tn * kN, N = p.N, K = p.K, lda = p.lda, ldb = p.ldb;
    const int rows = w.tile.end - m0 < kRows ? w.tile.end - m0 : kRows;
    const uint16_t* A = p.A + m0 * lda;
    const uint16_t* B = p.B + e * p.strideb + (TB ? n0 * ldb : n0);

    // This wave's slabs kb .. ke - 1 (none for the last waves when K is short).
    const int nk = (int)((K + kBK - 1) / kBK), per = (nk + kW - 1) / kW;
    const int kb = wave * per, ke = kb + per < nk ? kb + per : nk;
    uint16_t* const mine = lds + wave * 2 * kStage;
    const int64_t cols = N - n0 < kN ? N - n0 : kN;
    const rsrc_t a_desc = make_rsrc(A, (uint32_t)((((rows - 1) * lda + K) * 2 + 15) & ~(int64_t)15));
    const rsrc_t bt_desc = make_rsrc(B, (uint32_t)((((cols - 1) * ldb + K) * 2 + 15) & ~(int64_t)15));
    const int lrow = lane >> 3, pos = lane & 7;
    const uint32_t va = (uint32_t)(lrow * lda * 2 + ((pos ^ lrow) << 4));
    auto issue = [&](int kt, int st) __attribute__((always_inline)) {
        const int64_t k0 = (int64_t)kt * kBK;
        const uint32_t As = lds_addr(mine + st * kStage), Bs = As + kA * 2;
#pragma unroll
        for (int I = 0; I < kACopies; ++I) dma16(a_desc, va, (uint32_t)((8 * I * lda + k0) * 2), As + I * 1024);
        if constexpr (TB) {
#pragma unroll
            for (int I = 0; I < kBCopies; ++I)
                dma16(bt_desc, (uint32_t)(lrow * ldb * 2 + ((pos ^ lrow) << 4)), (uint32_t)((8 * I * ldb + k0) * 2),
                      Bs + I * 1024);
        } else {
            const int64_t bytes = (((K - k0 - 1) * ldb + N - n0) * 2 + 15) & ~(int64_t)15;
            const rsrc_t desc = make_rsrc(B + k0 * ldb, bytes < ((int64_t)1 << 31) ? (uint32_t)bytes : 0x80000000u);
#pragma unroll
            for (int I = 0; I < kBCopies; ++I)
                dma16(desc, (uint32_t)(lrow * ldb * 2 + ((pos ^ b_swz<kN>(8 * I + lrow)) << 4)),
                      (uint32_t)(8 * I * ldb * 2), Bs + I * 1024);
        }
        if constexpr (kLdsCheck == 2) __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
    };
    // Poison build: a stage is filled with NaN by its wave once it has read it.
    auto poison = [&](int st) {
        if constexpr (kLdsCheck == 1) {
            u32x4* q = reinterpret_cast<u32x4*>(mine + st * kStage);
            for (int i = lane; i < kStage / 8; i += 64) q[i] = u32x4{~0u, ~0u, ~0u, ~0u};
            __builtin_amdgcn_s_waitcnt(kWaitLgkm0);
        }
    };
    // k >= K of the last slab of k-contiguous operands: zeros in LDS.
    const int kr = (int)(K - (int64_t)(nk - 1) * kBK);
    const bool tail_here = ke == nk && kb < ke && kr < kBK;
    auto zero_tail = [&](int st) {
        auto zero = [&](uint16_t* S, int n) {
            if (lane >= n) return;
            for (int c = kr >> 3; c < 8; ++c) {
                u32x4* q = reinterpret_cast<u32x4*>(S + a_off(lane, c));
                *q = mask_tail(*q, kr - 8 * c);
            }
        };
        zero(mine + st * kStage, kRows);
        if constexpr (TB) zero(mine + st * kStage + kA, kN);
    };

    f32x4 acc[4][MF];
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < MF; ++i) acc[j][i] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int tr_row = pl >> 2, tr_col = (pl & 3) * 4;
    bf16x8 fa[2][MF], fb[2][4];
    auto read_frags = [&](int st, int ks) {
        const uint16_t *As = mine + st * kStage, *Bs = As + kA;
#pragma unroll
        for (int i = 0; i < MF; ++i)
            fa[ks][i] = *reinterpret_cast<const bf16x8*>(As + a_off(16 * i + pl, 4 * ks + g));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if constexpr (TB) fb[ks][j] = *reinterpret_cast<const bf16x8*>(Bs + a_off(16 * j + pl, 4 * ks + g));
            else fb[ks][j] = read_b_frag<kN>(Bs, 32 * ks + 8 * g + tr_row, 16 * j + tr_col);
        }
    };
    auto mfmas = [&](int ks) {
#pragma unroll
        for (int i = 0; i < MF; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                acc[j][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fb[ks][j], fa[ks][i], acc[j][i], 0, 0, 0);
    };
    if (kb < ke) {
        if constexpr (kLdsCheck == 1) { poison(0); poison(1); }
        issue(kb, 0);
        if (kb + 1 < ke) issue(kb + 1, 1);
        if (kb + 1 < ke) __builtin_amdgcn_s_waitcnt(waitcnt_vm(kACopies + kBCopies));
        else __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
        if (tail_here && kb + 1 == ke) zero_tail(0);
        read_frags(0, 0);
        auto slab = [&](int kt, int cur) {
            read_frags(cur, 1);
            mfmas(0);
            if (kt + 1 < ke) {
                // Both k steps of slab kt are in registers: its stage takes slab
                // kt + 2 while the wait below is for slab kt + 1 alone.
                __builtin_amdgcn_s_waitcnt(kWaitLgkm0);
                poison(cur);
                if (kt + 2 < ke) {
                    issue(kt + 2, cur);
                    __builtin_amdgcn_s_waitcnt(waitcnt_vm(kACopies + kBCopies));
                } else {
                    __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
                }
                if (tail_here && kt + 2 == ke) zero_tail(cur ^ 1);
                mfmas(1);
                read_frags(cur ^ 1, 0);
            } else {
                mfmas(1);
            }
        };
        for (int kt = kb; kt < ke; kt += 2) {
            slab(kt, 0);
            if (kt + 1 < ke) slab(kt + 1, 1);
        }
    }

    // Partial tiles: value (j, i) of lane l of wave w at ((4 w + j) MF + i) 64 + l,
    // in the stages every wave has finished with.
    __syncthreads();
    f32x4* red = reinterpret_cast<f32x4*>(lds);
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < MF; ++i) red[((4 * wave + j) * MF + i) * 64 + lane] = acc[j][i];
    __syncthreads();
    const uint16_t* bias = EPI && p.bias != nullptr ? p.bias + e * p.stridebias : nullptr;
    // Wave w finishes columns 16 w .. 16 w + 15: the partials in wave order.
    const int64_t col = n0 + 16 * wave + 4 * g;
#pragma unroll
    for (int i = 0; i < MF; ++i) {
        f32x4 sum = red[(wave * MF + i) * 64 + lane];
#pragma unroll
        for (int q = 1; q < kW; ++q) sum += red[((4 * q + wave) * MF + i) * 64 + lane];
        const int row = 16 * i + pl;
        if (row >= rows) continue;
        const float fr = EPI && p.row_scale != nullptr ? p.alpha * p.row_scale[m0 + row] : p.alpha;
        store_c4<EPI>(static_cast<uint16_t*>(p.C) + (m0 + row) * p.ldc, col, N, p.beta, bias, p.act, fr * sum, true);
    }
}

template <int MF>
hipError_t launch_rows(const GroupedArgs& a, hipStream_t s) {
    const int64_t tn = (a.N + kN - 1) / kN, grid = row_tiles_bound(a.M, a.groups, 16 * MF) * tn;
    if (grid > kMaxGrid) return hipErrorInvalidConfiguration;
    const bool epi = a.bias != nullptr || a.act != kActNone || a.row_scale != nullptr;
    auto fn = a.tb ? (epi ? &gemm_grouped_few_kernel<MF, true, true> : &gemm_grouped_few_kernel<MF, true, false>)
                   : (epi ? &gemm_grouped_few_kernel<MF, false, true> : &gemm_grouped_few_kernel<MF, false, false>);
    return launch_kernel(fn, dim3((unsigned)grid), dim3(kW * 64), s, a, tn);
}

}  // namespace

hipError_t launch_grouped_few(const GroupedArgs& a, int rows, hipStream_t s) {
    return rows == 16 ? launch_rows<1>(a, s) : launch_rows<4>(a, s);
}

}  // namespace dg
