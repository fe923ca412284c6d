// 8-bit block-scaled product, rows aligned to 16 bytes:
//
//   C(i,j) = alpha sum_b SA(b,i) SB(b, j / b_rows) sum_{k in b} A(i,k) B(j,k)   (+ epilogue)

#include "bf16_lds.hpp"
#include "fp8.hpp"
#include "kernels.hpp"

namespace dg {
namespace {

constexpr int kGroupM = 4;

__device__ __forceinline__ int chunk_off(int row, int c) { return row * 128 + ((c ^ (row & 7)) << 4); }

// B1: B has a scale for each row (128 rows share one otherwise).
template <int BM, int BN, int WAVES_M, int WAVES_N, bool EPI, bool B1>
__global__ __launch_bounds__(WAVES_M * WAVES_N * 64, BM == 256 ? 2 : 4)
void gemm_fp8_tiled_kernel(Fp8Args p, int tiles_m, int tiles_n) {
    constexpr int kWaves = WAVES_M * WAVES_N, kNT = kWaves * 64;
    constexpr int kWTM = BM / WAVES_M, kWTN = BN / WAVES_N;
    constexpr int kFM = kWTM / 16, kFN = kWTN / 16;
    constexpr int kDmaWaves = kWaves / 2;
    constexpr int kACopies = BM * 128 / 1024 / kDmaWaves, kBCopies = BN * 128 / 1024 / kDmaWaves;
    constexpr int kAScl = BM / 64, kBScl = BN / 64;            // 256-byte copies of the scales
    // Two stages, [A | B | scales] each.
    constexpr int kAB = BM * 128, kBB = BN * 128, kSB = (BM + (B1 ? BN : 0)) * 4;
    constexpr int kStage = kAB + kBB + kSB;
    __shared__ __attribute__((aligned(16))) uint8_t lds[2 * kStage];

    const int64_t M = p.M, N = p.N, K = p.K, lda = p.lda, ldb = p.ldb;
    const int nk = (int)((K + kScaleBlock - 1) / kScaleBlock);
    int tm, tn;
    tile_coords(blockIdx.x, gridDim.x, tiles_m, tiles_n, kGroupM, tm, tn);
    const int64_t m0 = (int64_t)tm * BM, n0 = (int64_t)tn * BN;
    const int t = threadIdx.x, lane = t & 63;
    const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int wm0 = (wave / WAVES_N) * kWTM, wn0 = (wave % WAVES_N) * kWTN;
    const int pl = lane & 15, g = lane >> 4;

    const int64_t rows_a = M - m0 < BM ? M - m0 : BM, rows_b = N - n0 < BN ? N - n0 : BN;
    const rsrc_t a_desc = make_rsrc(p.A + m0 * lda, (uint32_t)(((rows_a - 1) * lda + K + 15) & ~(int64_t)15));
    const rsrc_t b_desc = make_rsrc(p.B + n0 * ldb, (uint32_t)(((rows_b - 1) * ldb + K + 15) & ~(int64_t)15));
    const int lrow = lane >> 3, pos = lane & 7;
    const uint32_t va = (uint32_t)(lrow * lda + ((pos ^ lrow) << 4)), vb = (uint32_t)(lrow * ldb + ((pos ^ lrow) << 4));
    auto dma = [&](int kt, int st) __attribute__((always_inline)) {
        if (wave >= kDmaWaves) return;
        const uint32_t k0 = (uint32_t)kt * 128u;
        const uint32_t As = lds_addr(lds) + (uint32_t)(st * kStage), Bs = As + kAB, Ss = Bs + kBB;
#pragma unroll
        for (int i = 0; i < kACopies; ++i) {
            const int I = wave * kACopies + i;
            dma16(a_desc, va, (uint32_t)(8 * I * lda) + k0, As + I * 1024);
        }
#pragma unroll
        for (int i = 0; i < kBCopies; ++i) {
            const int I = wave * kBCopies + i;
            dma16(b_desc, vb, (uint32_t)(8 * I * ldb) + k0, Bs + I * 1024);
        }
        const rsrc_t sa = make_rsrc(p.SA + kt * p.ldsa + m0, (uint32_t)(rows_a * 4));
#pragma unroll
        for (int i = 0; i < kAScl; i += kDmaWaves)
            if (i + wave < kAScl) dma4(sa, (uint32_t)(lane * 4), (uint32_t)(i + wave) * 256, Ss + (i + wave) * 256);
        if constexpr (B1) {
            const rsrc_t sb = make_rsrc(p.SB + kt * p.ldsb + n0, (uint32_t)(rows_b * 4));
#pragma unroll
            for (int i = 0; i < kBScl; i += kDmaWaves)
                if (i + wave < kBScl)
                    dma4(sb, (uint32_t)(lane * 4), (uint32_t)(i + wave) * 256, Ss + BM * 4 + (i + wave) * 256);
        }
    };
    // Bytes at k >= K of a partial last block: zeros in LDS.
    auto zero_tail = [&](int st, int kr) {
        auto zero = [&](uint8_t* S, int rows) {
            for (int row = t; row < rows; row += kNT) {
                for (int c = kr >> 4; c < 8; ++c) {
                    u32x4* q = reinterpret_cast<u32x4*>(S + chunk_off(row, c));
                    u32x4 v = *q;
                    const int keep = kr - 16 * c;             // bytes of this chunk that stay
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        const int b = keep - 4 * w;
                        v[w] &= b >= 4 ? ~0u : (b <= 0 ? 0u : (1u << (8 * b)) - 1u);
                    }
                    *q = v;
                }
            }
        };
        zero(lds + st * kStage, BM);
        zero(lds + st * kStage + kAB, BN);
    };

    f32x4 acc[kFN][kFM];
#pragma unroll
    for (int j = 0; j < kFN; ++j)
#pragma unroll
        for (int i = 0; i < kFM; ++i) acc[j][i] = f32x4{0.f, 0.f, 0.f, 0.f};

    // A fragment of 16 rows: chunks g and g + 4 of row `pl`. Rows 16 apart have
    // the same swizzle, so a wave's fragments lie 2048 bytes apart.
    const int lo = ((g ^ (pl & 7)) << 4) + pl * 128, hi = (((g + 4) ^ (pl & 7)) << 4) + pl * 128;
    auto frag = [&](const uint8_t* S) {
        return join16(*reinterpret_cast<const u32x4*>(S + lo), *reinterpret_cast<const u32x4*>(S + hi));
    };
    const int64_t sb_col = (n0 + wn0) / 128;
    auto compute = [&](int kt, int st) __attribute__((always_inline)) {
        const uint8_t *As = lds + st * kStage + wm0 * 128, *Bs = lds + st * kStage + kAB + wn0 * 128;
        const float* Ss = reinterpret_cast<const float*>(lds + st * kStage + kAB + kBB);
        const float sb1 = B1 ? 1.f : (n0 + wn0 < N ? p.SB[kt * p.ldsb + sb_col] : 0.f);
        i32x8 fb[kFN], fa = frag(As);
        f32x4 sb[kFN], d[kFN], last[kFN];
        float sa = Ss[wm0 + pl] * sb1, last_sa = 0.f;
#pragma unroll
        for (int j = 0; j < kFN; ++j) {
            fb[j] = frag(Bs + 2048 * j);
            if constexpr (B1) sb[j] = *reinterpret_cast<const f32x4*>(Ss + BM + wn0 + 16 * j + 4 * g);
        }
        // Each MFMA is followed by the scaled additions of the one kFN before
        // it, whose result is there by then; the scheduling barriers keep the
        // compiler from running further ahead, which would not fit in the
        // registers.
        auto add = [&](int j, int i, float s, const f32x4& v) {
#pragma unroll
            for (int r = 0; r < 4; ++r) acc[j][i][r] = __builtin_fmaf(v[r], B1 ? s * sb[j][r] : s, acc[j][i][r]);
        };
#pragma unroll
        for (int i = 0; i < kFM; ++i) {
            i32x8 next = fa;
            float next_sa = 0.f;
            if (i + 1 < kFM) {
                next = frag(As + 2048 * (i + 1));
                next_sa = Ss[wm0 + 16 * (i + 1) + pl];
            }
#pragma unroll
            for (int j = 0; j < kFN; ++j) {
                d[j] = mfma_fp8(fb[j], fa);
                if (i > 0) add(j, i - 1, last_sa, last[j]);
                __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int j = 0; j < kFN; ++j) last[j] = d[j];
            last_sa = sa;
            sa = next_sa * sb1;
            fa = next;
        }
#pragma unroll
        for (int j = 0; j < kFN; ++j) add(j, kFM - 1, last_sa, last[j]);
    };

    const int kr = (int)(K - (int64_t)(nk - 1) * 128);
    if constexpr (kLdsCheck == 1) lds_retire(lds, 2 * kStage, t, kNT);
    copy_begin();
    dma(0, 0);
    copy_end();
    // The stage is a number, not a copy of the code for each: two copies let
    // the compiler move a slab's additions past the branch between them.
    for (int kt = 0, st = 0; kt < nk; ++kt, st ^= 1) {
        // Slab kt has landed and every read of slab kt - 1 is done.
        lds_barrier();
        if (kLdsCheck == 1 && kt > 0) lds_retire(lds + (st ^ 1) * kStage, kStage, t, kNT);
        if (kt + 1 == nk && kr < 128) {
            zero_tail(st, kr);
            lds_only_barrier();
        }
        if (kt + 1 < nk) {
            copy_begin();
            dma(kt + 1, st ^ 1);
            copy_end();
        }
        compute(kt, st);
    }
#pragma unroll
    for (int i = 0; i < kFM; ++i) {
        const int64_t row = m0 + wm0 + 16 * i + pl;
        if (row >= M) continue;
#pragma unroll
        for (int j = 0; j < kFN; ++j)
            store_c4<EPI>(p.C + row * p.ldc, n0 + wn0 + 16 * j + 4 * g, N, p.beta, p.bias, p.act, p.alpha * acc[j][i],
                          true);
    }
}

template <int BM, int BN, int WAVES_M, int WAVES_N>
hipError_t launch_tiles(const Fp8Args& a, hipStream_t s) {
    const int64_t tm = (a.M + BM - 1) / BM, tn = (a.N + BN - 1) / BN;
    if (tm * tn > kMaxGrid) return hipErrorInvalidConfiguration;
    const bool epi = a.bias != nullptr || a.act != kActNone, b1 = a.b_rows == 1;
    auto fn = epi ? (b1 ? &gemm_fp8_tiled_kernel<BM, BN, WAVES_M, WAVES_N, true, true>
                        : &gemm_fp8_tiled_kernel<BM, BN, WAVES_M, WAVES_N, true, false>)
                  : (b1 ? &gemm_fp8_tiled_kernel<BM, BN, WAVES_M, WAVES_N, false, true>
                        : &gemm_fp8_tiled_kernel<BM, BN, WAVES_M, WAVES_N, false, false>);
    return launch_kernel(fn, dim3((unsigned)(tm * tn)), dim3(WAVES_M * WAVES_N * 64), s, a, tm, tn);
}

}  // namespace

hipError_t launch_fp8(const Fp8Args& a, int, hipStream_t s) {
    auto at16 = [](const void* q, int64_t ld) { return reinterpret_cast<uintptr_t>(q) % 16 == 0 && ld % 16 == 0; };
    const bool rows16 = at16(a.A, a.lda) && at16(a.B, a.ldb);
    const bool c8 = reinterpret_cast<uintptr_t>(a.C) % 8 == 0 && a.ldc % 4 == 0;
    const int64_t lim = (int64_t)1 << 31;
    const bool fits = 256 * a.lda + a.K < lim && 256 * a.ldb + a.K < lim;
    if (!rows16 || !c8 || !fits) return launch_fp8_general(a, s);
    const int64_t t256 = ((a.M + 255) / 256) * ((a.N + 255) / 256);
    if (t256 > 128) return launch_tiles<256, 256, 2, 4>(a, s);
    return launch_tiles<128, 128, 2, 4>(a, s);
}

}  // namespace dg
