// 8-bit block-scaled product, rows aligned to 16 bytes:
//
//   C(i,j) = alpha sum_b SA(b,i) SB(b, j / b_rows) sum_{k in b} A(i,k) B(j,k)   (+ epilogue)
//
// The sum over a block b of 128 k is one v_mfma_f32_16x16x128_f8f6f4 per 16 x 16
// of C, from zero; its fp32 result times SA SB is added to the accumulator by
// the vector units. The block scales differ along k, so the matrix core cannot
// accumulate across blocks itself; 4 multiply-adds per lane take half the
// cycles of the MFMA they follow and run beside the next ones. With a scale for
// each row of B, SA SB differs by element: a multiply and a multiply-add each,
// as many cycles as the MFMAs (4096^2 x 8192 131 us, 110 without the multiply;
// with 128 rows to a scale 113).
//
// Bound: at 256 x 256 tiles a slab of 128 k holds 32 MFMAs per wave, 2048 cycles
// of each matrix core; 64 KB of copies into LDS and 192 KB of fragment reads
// pass beside them. On one MI355X a slab takes 1.7 us, about half of it MFMA:
// without the multiply-adds it takes 1.6, with copies that read nothing 1.25. So
// the copies' way through L2 is what is left, then the multiply-adds. Smaller
// tiles, one or two to a CU, wait for their copies at every slab's barrier:
// 509 x 4096 x 4000 on 64 x 128 tiles copies 768 KB per CU in 19.6 us, 40 GB/s.
//
//   * 8 waves, each 128 x 64 of a 256 x 256 tile (96 x 64 of 192 x 256, or a smaller
//     share of a smaller tile); K in slabs of 128 in a ring of NS LDS stages, copied with
//     LDS-destined 128-bit loads, A and B in rows of 128 bytes whose 16-byte
//     chunk c lies at c ^ (row mod 8): the fragment reads meet no bank conflict;
//   * the slab's scales travel with it: 256-byte copies from SA and SB, whose
//     layout keeps the scales of one block of k together. (Read from global
//     memory at their use they cost every slab 0.3 us: 4096^3 71 against 61 us.)
//   * B is the instruction's first operand, so a lane holds 4 consecutive
//     columns of one row of C, and one scale of A serves all of them;
//   * where 64 x 64 tiles have a CU each, two groups of 4 waves share a tile's K
//     (KS), so that one's MFMAs run in the other's waits;
//   * 256 x 256 and 192 x 256 tiles run one resident workgroup per CU that walks its tiles:
//     the ring runs on over them, so a tile's first slab lands while the one
//     before is stored;
//   * edges: descriptors end where the matrices end (rows past M and N arrive
//     as zeros), bytes at k >= K of a partial last block are zeroed in LDS.
//
// Operand layout of the MFMA: see mfma_fp8.

#include "fp8.hpp"
#include "ops.hpp"

namespace dg {
namespace {

constexpr int kGroupM = 4;

__device__ __forceinline__ int chunk_off(int row, int c) { return row * 128 + ((c ^ (row & 7)) << 4); }

// B1: B has a scale for each row (128 rows share one otherwise). The grid may
// be smaller than the number of tiles: workgroup w takes tiles w, w + grid, ..
// KS = 2: two groups of waves in one workgroup share a tile, group q over the
// slabs q, q + 2, .. with a ring of its own; group 1 hands its sums to group 0
// through LDS (one tile per workgroup). Both groups take every barrier.
template <int BM, int BN, int WAVES_M, int WAVES_N, int NS, int KS, bool EPI, bool B1>
__global__ __launch_bounds__(KS * WAVES_M * WAVES_N * 64, BM >= 192 ? 2 : 4)
void gemm_fp8_tiled_kernel(Fp8Args p, int tiles_m, int tiles_n) {
    constexpr int kWaves = WAVES_M * WAVES_N, kNT = kWaves * 64;
    constexpr int kWTM = BM / WAVES_M, kWTN = BN / WAVES_N;
    constexpr int kFM = kWTM / 16, kFN = kWTN / 16;
    constexpr int kACopies = BM * 128 / 1024 / kWaves, kBCopies = BN * 128 / 1024 / kWaves;
    constexpr int kAScl = BM / 64, kBScl = B1 ? BN / 64 : 1;    // 256-byte copies of the scales
    constexpr int kPerSlab = kACopies + kBCopies + 1;           // copies of each wave
    static_assert(kAScl + kBScl <= kWaves, "one copy of scales per wave");
    static_assert(kACopies * kWaves * 1024 == BM * 128 && kBCopies * kWaves * 1024 == BN * 128, "slabs split evenly");
    // Copies issued after each row of MFMAs: with two stages early in the slab,
    // as they have to land within it (4096^2 x 8192: all after the first row
    // 115.2 us, over 5 rows 114.1, over all 8 118.9).
    constexpr int kPerRow = (NS == 2 ? 2 : 1) * ((kPerSlab + kFM - 1) / kFM);
    // A ring of NS stages, [A | B | scales] each.
    constexpr int kAB = BM * 128, kBB = BN * 128, kSB = (kAScl + kBScl) * 256;
    constexpr int kStage = kAB + kBB + kSB;
    __shared__ __attribute__((aligned(16))) uint8_t all[KS * NS * kStage];

    const int64_t M = p.M, N = p.N, K = p.K, lda = p.lda, ldb = p.ldb;
    const int nk = (int)((K + kScaleBlock - 1) / kScaleBlock);
    const int kr = (int)(K - (int64_t)(nk - 1) * kScaleBlock);
    const int tiles = tiles_m * tiles_n, grid = (int)gridDim.x;
    // t and wave count within the group.
    const int grp = KS == 1 ? 0 : __builtin_amdgcn_readfirstlane((int)threadIdx.x / kNT);
    const int t = (int)threadIdx.x - grp * kNT, lane = t & 63;
    const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
    uint8_t* const lds = all + grp * (NS * kStage);
    const int turns = (nk + KS - 1) / KS;          // slabs of each group (one past the end where nk is odd)
    const int wm0 = (wave / WAVES_N) * kWTM, wn0 = (wave % WAVES_N) * kWTN;
    const int pl = lane & 15, g = lane >> 4;

    // Rows and columns of tile `id`: each round of `grid` tiles is spread over
    // the XCDs in contiguous runs.
    auto place = [&](int id, int64_t& m0, int64_t& n0) {
        const int first = id - (int)blockIdx.x;
        const int round = tiles - first < grid ? tiles - first : grid;
        int tm, tn;
        raster_tile(first + xcd_slot((int)blockIdx.x, round), tiles_m, tiles_n, kGroupM, tm, tn);
        m0 = (int64_t)tm * BM;
        n0 = (int64_t)tn * BN;
    };

    // ---- copies ----
    // The ring is filled NS - 1 slabs ahead by a cursor over this workgroup's
    // slabs: slab c_kt of tile c_id.
    const int lrow = lane >> 3, pos = lane & 7;
    const uint32_t va = (uint32_t)(lrow * lda + ((pos ^ lrow) << 4)), vb = (uint32_t)(lrow * ldb + ((pos ^ lrow) << 4));
    const int scl_slot = wave % (kAScl + kBScl);
    const bool scl_a = scl_slot < kAScl;
    const uint32_t scl_chunk = (uint32_t)(scl_a ? scl_slot : scl_slot - kAScl) * 256;
    const int64_t scl_ld = scl_a ? p.ldsa : p.ldsb;
    int c_id = (int)blockIdx.x, c_kt = grp;
    rsrc_t a_desc, b_desc;
    const float* scl_base;
    uint32_t scl_bytes;
    auto aim = [&](int id) __attribute__((always_inline)) {
        int64_t m0 = 0, n0 = 0;
        if (id < tiles) place(id, m0, n0);
        const int64_t rows_a = M - m0 < BM ? M - m0 : BM, rows_b = N - n0 < BN ? N - n0 : BN;
        a_desc = make_rsrc(p.A + m0 * lda, id < tiles ? (uint32_t)(((rows_a - 1) * lda + K + 15) & ~(int64_t)15) : 0u);
        b_desc = make_rsrc(p.B + n0 * ldb, id < tiles ? (uint32_t)(((rows_b - 1) * ldb + K + 15) & ~(int64_t)15) : 0u);
        scl_base = scl_a ? p.SA + m0 : p.SB + (B1 ? n0 : n0 / 128);
        const uint32_t entries = scl_a ? (uint32_t)rows_a : (uint32_t)(B1 ? rows_b : (n0 % 128 + rows_b + 127) / 128);
        scl_bytes = id < tiles ? 4u * entries : 0u;
    };
    // Copy q (0 .. kPerSlab - 1) of this wave for the cursor's slab into stage
    // st. Every wave issues the same number of copies for a slab, so that a
    // count of outstanding copies is a number of slabs: waves past the last
    // chunk of scales copy an earlier one again (the same bytes to the same
    // place), and past the last tile all copies lie outside their descriptors
    // and put zeros into a stage that nothing reads any more. With 128 rows to
    // a scale the tile's one or two scales of B lie at the start of their copy.
    auto copy = [&](int q, int st) __attribute__((always_inline)) {
        const bool in = KS == 1 || c_kt < nk;
        const uint32_t k0 = in ? (uint32_t)c_kt * 128u : 0x80000000u;
        const uint32_t As = lds_addr(lds) + (uint32_t)(st * kStage), Bs = As + kAB, Ss = Bs + kBB;
        if (q == 0) {
            dma4(make_rsrc(scl_base + (in ? c_kt : 0) * scl_ld, in ? scl_bytes : 0u), (uint32_t)(lane * 4), scl_chunk,
                 Ss + (scl_a ? 0 : BM * 4) + scl_chunk);
        } else if (q <= kACopies) {
            const int I = wave * kACopies + q - 1;
            dma16(a_desc, va, (uint32_t)(8 * I * lda) + k0, As + I * 1024);
        } else {
            const int I = wave * kBCopies + q - 1 - kACopies;
            dma16(b_desc, vb, (uint32_t)(8 * I * ldb) + k0, Bs + I * 1024);
        }
    };
    auto advance = [&]() __attribute__((always_inline)) {
        c_kt += KS;
        if (KS == 1 && c_kt == nk) {
            c_kt = 0;
            c_id += grid;
            aim(c_id);
        }
    };
    auto copy_all = [&](int st) __attribute__((always_inline)) {
        copy_begin();
#pragma unroll
        for (int q = 0; q < kPerSlab; ++q) copy(q, st);
        copy_end();
    };
    // Bytes at k >= K of a partial last block: zeros in LDS.
    auto zero_tail = [&](int st) {
        auto zero = [&](uint8_t* S, int rows) {
            for (int row = t; row < rows; row += kNT) {
                for (int c = kr >> 4; c < 8; ++c) {
                    u32x4* q = reinterpret_cast<u32x4*>(S + chunk_off(row, c));
                    *q = mask_bytes(*q, kr - 16 * c);
                }
            }
        };
        zero(lds + st * kStage, BM);
        zero(lds + st * kStage + kAB, BN);
    };

    // ---- one slab ----
    f32x4 acc[kFN][kFM];
    // A fragment of 16 rows: chunks g and g + 4 of row `pl`. Rows 16 apart have
    // the same swizzle, so a wave's fragments lie 2048 bytes apart.
    const int lo = ((g ^ (pl & 7)) << 4) + pl * 128, hi = (((g + 4) ^ (pl & 7)) << 4) + pl * 128;
    auto frag = [&](const uint8_t* S) {
        return join16(*reinterpret_cast<const u32x4*>(S + lo), *reinterpret_cast<const u32x4*>(S + hi));
    };
    // Each MFMA is followed by the scaled additions of the one kFN before it,
    // whose result is there by then; the scheduling barriers keep the compiler
    // from running further ahead, which would not fit in the registers. The
    // last row's additions wait for the next slab's first row, where they pass
    // the time of its first reads (with a scale for each row of B its 16 more
    // registers would not fit, and they end the slab).
    constexpr bool kCarry = !B1;
    f32x4 sb[kFN], last[kFN];
    float last_sa = 0.f;
    auto add = [&](int j, int i) __attribute__((always_inline)) {
#pragma unroll
        for (int r = 0; r < 4; ++r)
            acc[j][i][r] = __builtin_fmaf(last[j][r], B1 ? last_sa * sb[j][r] : last_sa, acc[j][i][r]);
    };
    // The slab in stage st; meanwhile the copies of the cursor's slab into
    // stage `to`, a few after each row of MFMAs.
    auto compute = [&](int st, int to) __attribute__((always_inline)) {
        const uint8_t *As = lds + st * kStage + wm0 * 128, *Bs = lds + st * kStage + kAB + wn0 * 128;
        const float* Ss = reinterpret_cast<const float*>(lds + st * kStage + kAB + kBB);
        const float sb1 = B1 ? 1.f : Ss[BM + wn0 / 128];
        i32x8 fb[kFN], fa = frag(As);
        f32x4 d[kFN];
        fb[0] = frag(Bs);
        __builtin_amdgcn_sched_barrier(0);
        float sa = Ss[wm0 + pl] * sb1;
#pragma unroll
        for (int j = 1; j < kFN; ++j) {
            fb[j] = frag(Bs + 2048 * j);
            __builtin_amdgcn_sched_barrier(0);
        }
        if constexpr (B1) {
#pragma unroll
            for (int j = 0; j < kFN; ++j) sb[j] = *reinterpret_cast<const f32x4*>(Ss + BM + wn0 + 16 * j + 4 * g);
        }
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
                if (i > 0) add(j, i - 1);
                else if (kCarry) add(j, kFM - 1);
                __builtin_amdgcn_sched_barrier(0);
            }
            if constexpr (kLdsCheck != 2) {
#pragma unroll
                for (int q = i * kPerRow; q < (i + 1) * kPerRow && q < kPerSlab; ++q) copy(q, to);
            }
#pragma unroll
            for (int j = 0; j < kFN; ++j) last[j] = d[j];
            last_sa = sa;
            sa = next_sa * sb1;
            fa = next;
        }
        if constexpr (!kCarry) {
#pragma unroll
            for (int j = 0; j < kFN; ++j) add(j, kFM - 1);
        }
    };

    if constexpr (kLdsCheck == 1) lds_retire(lds, NS * kStage, t, kNT);
    aim(c_id);
    for (int q = 0; q < NS - 1; ++q) {
        if (q > 0) advance();
        copy_all(q);
    }
    // Stores that the tile before left on their way, issued after this tile's
    // first copies (0 where they are not counted).
    bool stores = false;
    constexpr int kStores = 2 * kFM;
    int st = 0;
    for (int id = (int)blockIdx.x; id < tiles; id += grid) {
        int64_t m0, n0;
        place(id, m0, n0);
#pragma unroll
        for (int j = 0; j < kFN; ++j)
#pragma unroll
            for (int i = 0; i < kFM; ++i) acc[j][i] = f32x4{0.f, 0.f, 0.f, 0.f};
        if constexpr (kCarry) {
#pragma unroll
            for (int j = 0; j < kFN; ++j) last[j] = f32x4{0.f, 0.f, 0.f, 0.f};
            last_sa = 0.f;
        }
        // The stage is a number, not a copy of the code for each: copies let
        // the compiler move a slab's additions past the branch between them.
        for (int turn = 0; turn < turns; ++turn) {
            // This slab has landed (NS - 2 later ones may be on their way), and
            // every read of the slab before, whose stage the cursor's slab
            // takes, is done.
            if (NS == 2 && stores) __builtin_amdgcn_s_waitcnt(waitcnt_vm(kStores));
            else __builtin_amdgcn_s_waitcnt(waitcnt_vm(kPerSlab * (NS - 2)));
            stores = false;
            lds_only_barrier();
            const int before = st == 0 ? NS - 1 : st - 1;
            if (kLdsCheck == 1) lds_retire(lds + before * kStage, kStage, t, kNT);
            advance();
            if (turn + 1 == turns && kr < kScaleBlock) {
                if (KS == 1 || turn * KS + grp == nk - 1) zero_tail(st);
                lds_only_barrier();
            }
            if constexpr (kLdsCheck == 2) copy_all(before);
            compute(st, before);
            st = st + 1 == NS ? 0 : st + 1;
        }

        if constexpr (kCarry) {
#pragma unroll
            for (int j = 0; j < kFN; ++j) add(j, kFM - 1);
        }

        if constexpr (KS == 2) {
            // Group 1's sums to group 0 through the rings, which both have read
            // to the end and whose last copies (zeros) have landed: value c of
            // lane l of wave w at (c waves + w) 64 + l. First half + second half,
            // the same bits on every call.
            static_assert(kFM * kFN * kNT * 16 <= KS * NS * kStage, "sums fit");
            f32x4* const hand = reinterpret_cast<f32x4*>(all) + wave * 64 + lane;
            lds_barrier();
            if (grp == 1) {
#pragma unroll
                for (int j = 0; j < kFN; ++j)
#pragma unroll
                    for (int i = 0; i < kFM; ++i) hand[(j * kFM + i) * kNT] = acc[j][i];
            }
            lds_only_barrier();
            if (grp == 1) return;
#pragma unroll
            for (int j = 0; j < kFN; ++j)
#pragma unroll
                for (int i = 0; i < kFM; ++i) acc[j][i] += hand[(j * kFM + i) * kNT];
        }

        // ---- epilogue ----
        if constexpr (kWTN == 64 && KS == 1) {
            if (m0 + BM <= M && n0 + BN <= N) {
                // Whole tiles: each 16-row block of a wave's results goes
                // through LDS into row order, so that a lane stores 8 columns
                // and 8 lanes a row's 128 bytes, instead of 16 rows of 32 bytes
                // per instruction. The scratch is the last slab's stage (all
                // its reads are done after the barrier; the copies on their way
                // go to other stages): 16 rows of 64 floats per wave, 16-byte
                // chunk c of row r at c ^ r.
                static_assert(kWaves * 4096 <= kStage, "scratch fits a stage");
                const int cc = lane & 7, rr = lane >> 3;
                const int64_t gcol = n0 + wn0 + 8 * cc;
                float bias[8];
                if constexpr (EPI) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) bias[e] = p.bias != nullptr ? bf16_to_f32(p.bias[gcol + e]) : 0.f;
                }
                lds_only_barrier();
                float* scr = reinterpret_cast<float*>(lds + (st == 0 ? NS - 1 : st - 1) * kStage + wave * 4096);
#pragma unroll
                for (int i = 0; i < kFM; ++i) {
                    uint16_t* crow = p.C + (m0 + wm0 + 16 * i + rr) * p.ldc + gcol;
                    u32x4 c0[2];
                    if (p.beta != 0.f) {
#pragma unroll
                        for (int h = 0; h < 2; ++h) c0[h] = *reinterpret_cast<const u32x4_a4*>(crow + 8 * h * p.ldc);
                    }
#pragma unroll
                    for (int j = 0; j < kFN; ++j)
                        *reinterpret_cast<f32x4*>(scr + pl * 64 + 4 * ((4 * j + g) ^ pl)) = acc[j][i];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int r = rr + 8 * h;
                        const f32x4 x = *reinterpret_cast<const f32x4*>(scr + r * 64 + 4 * ((2 * cc) ^ r));
                        const f32x4 y = *reinterpret_cast<const f32x4*>(scr + r * 64 + 4 * ((2 * cc + 1) ^ r));
                        float v[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            v[e] = p.alpha * (e < 4 ? x[e] : y[e - 4]);
                            if constexpr (EPI) v[e] = activate(v[e] + bias[e], p.act);
                        }
                        if (p.beta != 0.f) {
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                v[e] += p.beta * bf16_to_f32((uint16_t)(c0[h][e >> 1] >> (16 * (e & 1))));
                        }
                        // C would push operands out of L2: 8192 x 12288 x 4096 364 -> 354 us.
                        const u32x4_a4 out = u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                   pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
                        __builtin_nontemporal_store(out, reinterpret_cast<u32x4_a4*>(crow + 8 * h * p.ldc));
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
                stores = true;
                continue;
            }
        }
#pragma unroll
        for (int i = 0; i < kFM; ++i) {
            const int64_t row = m0 + wm0 + 16 * i + pl;
            if (row >= M) continue;
#pragma unroll
            for (int j = 0; j < kFN; ++j)
                store_c4<EPI>(p.C + row * p.ldc, n0 + wn0 + 16 * j + 4 * g, N, p.beta, p.bias, p.act,
                              p.alpha * acc[j][i], true);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    // No copy may land in LDS after the workgroup has left it.
    __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
}

template <int BM, int BN, int WAVES_M, int WAVES_N, int NS, int KS>
hipError_t launch_tiles(const Fp8Args& a, int64_t most, hipStream_t s) {
    const int64_t tm = (a.M + BM - 1) / BM, tn = (a.N + BN - 1) / BN;
    if (tm * tn > kMaxGrid) return hipErrorInvalidConfiguration;
    const bool epi = a.bias != nullptr || a.act != kActNone, b1 = a.b_rows == 1;
#define DG_F(...) &gemm_fp8_tiled_kernel<BM, BN, WAVES_M, WAVES_N, NS, KS, __VA_ARGS__>
    auto fn = epi ? (b1 ? DG_F(true, true) : DG_F(true, false)) : (b1 ? DG_F(false, true) : DG_F(false, false));
#undef DG_F
    const int64_t grid = most > 0 && tm * tn > most ? most : tm * tn;
    return launch_kernel(fn, dim3((unsigned)grid), dim3(KS * WAVES_M * WAVES_N * 64), s, a, tm, tn);
}

// Time of a product's tiles in us per slab of K, at 256 CUs: whole rounds of
// `per_round` resident tiles at `round`, and the rest by how many share a CU.
double rounds(int64_t M, int64_t N, int bm, int bn, int per_round, double round, double one, double two) {
    const int64_t tiles = ((M + bm - 1) / bm) * ((N + bn - 1) / bn);
    const int64_t full = tiles / per_round, rem = tiles % per_round;
    return (double)full * round + (rem == 0 ? 0.0 : rem <= 256 ? one : rem <= 512 ? two : round);
}

}  // namespace

// Which kernel. Few rows stream B straight into registers; the others run the
// tile size whose rounds of resident workgroups cost least. Measured on one
// MI355X (us): 24 x 12288 x 4096 12.7 on 64 x 64 tiles, 17.6 on the few-row
// kernel, but 32 x 8192^2 22.4 and 17.9; 48 x 8192^2 22.5 and 23.0.
// 96 x 8192^2: 64 x 64 22.8, 64 x 128 28.4, 128 x 128 36.0, 256 x 256 83;
// 700 x 2048^2: 11.1, 10.1, 12.6, 29.5; 1500^3: 14.7, 14.4, 11.6, 26.5;
// 2048 x 2560 x 4096: 41.4, 38.1, 40.8, 51.1; 3500 x 3700 x 2000: 65, 56, 54, 34.6;
// 64 x 64, 64 x 128 and 128 x 128: 509 x 4096 x 4000 23.5, 19.6, 23.9, 512 x 4096 x 8192
// 32.8, 29.7, 39.5. The model counts 256 CUs, the whole card.
// A tile size's time per slab with one, two or a CU's fill of workgroups:
// 64 x 64 0.28, 0.66, 0.9 (three); 64 x 128 0.5, 0.8; 128 x 128 0.72, 1.3 (two of
// two stages); 192 x 256 1.4; 256 x 256 1.75. 192 x 256 saves what 256 x 256 leaves
// empty in a last round (3346 x 6144 x 4912 142 -> 124 us, 6000^2 x 3000 with a scale
// per row of B 162 -> 135, 5550 x 1478 x 5756 70 -> 60, 4813 x 3710 x 720 38 -> 29).
// One 64 x 64 tile to a CU runs as two groups of 4 waves that share its K
// (128 x 8192^2 23.3 -> 18.3 us, 1024^2 x 4096 13.5 -> 10.9; two to a CU 509 x 4096 x
// 4000 23.4 -> 24.5, and at 64 x 128 and 128 x 128 no gain).
hipError_t launch_fp8(const Fp8Args& a, int cus, hipStream_t s) {
    auto at16 = [](const void* q, int64_t ld) { return reinterpret_cast<uintptr_t>(q) % 16 == 0 && ld % 16 == 0; };
    const bool rows16 = at16(a.A, a.lda) && at16(a.B, a.ldb);
    const bool c8 = reinterpret_cast<uintptr_t>(a.C) % 8 == 0 && a.ldc % 4 == 0;
    const int64_t lim = (int64_t)1 << 31;
    const bool fits = 256 * a.lda + a.K < lim && 256 * a.ldb + a.K < lim;
    if (!rows16 || !c8 || !fits) return launch_fp8_general(a, s);
    if (a.M <= 16 || (a.M <= 32 && a.N <= 8192)) return launch_fp8_few(a, s);
    const double c64 = rounds(a.M, a.N, 64, 64, 768, 0.9, 0.28, 0.66);
    const double c64w = rounds(a.M, a.N, 64, 128, 512, 0.8, 0.5, 0.8);
    const double c128 = rounds(a.M, a.N, 128, 128, 512, 1.3, 0.72, 1.3);
    const double c256 = rounds(a.M, a.N, 256, 256, 256, 1.75, 1.75, 1.75);
    const double c192 = rounds(a.M, a.N, 192, 256, 256, 1.4, 1.4, 1.4);
    if (c192 < c256 && c192 <= c128 && c192 <= c64w && c192 <= c64)
        return launch_tiles<192, 256, 2, 4, 2, 1>(a, cus, s);
    if (c256 <= c128 && c256 <= c64w && c256 <= c64) return launch_tiles<256, 256, 2, 4, 2, 1>(a, cus, s);
    if (c128 <= c64w && c128 <= c64) {
        const int64_t t128 = ((a.M + 127) / 128) * ((a.N + 127) / 128);
        if (t128 <= 256) return launch_tiles<128, 128, 2, 4, 3, 1>(a, 0, s);
        return launch_tiles<128, 128, 2, 4, 2, 1>(a, 0, s);
    }
    if (c64w <= c64) return launch_tiles<64, 128, 2, 4, 3, 1>(a, 0, s);
    if (((a.M + 63) / 64) * ((a.N + 63) / 64) <= 256) return launch_tiles<64, 64, 2, 2, 3, 2>(a, 0, s);
    return launch_tiles<64, 64, 2, 4, 3, 1>(a, 0, s);
}

}  // namespace dg
