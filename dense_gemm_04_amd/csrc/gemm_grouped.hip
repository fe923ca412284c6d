// Products grouped by expert and their weight gradients on bf16 matrix cores,
// rows aligned to 16 bytes, fp32 accumulation, one rounding at the end:
//
//   rows:  C(i,:) = act(alpha row_scale[i] A(i,:) op(B_e) + bias_e) + beta C(i,:), i in group e
//   wgrad: C_e = alpha A_e^T B_e + beta C_e (bf16 or fp32)
//
// Both are bound by the matrix cores once a group has a few hundred rows, and
// by reading the experts' matrices (rows) or writing them (wgrad) below that.
//
//   * rows: every group is cut into tiles of BM rows of its own, numbered in
//     group order; each wave finds its tile's group from the offsets, which its
//     lanes hold (lane e group e's; past 64 groups they are read again), by a
//     prefix sum and a ballot. So the host needs to know no group's size and
//     nothing is launched to lay out tiles. The grid covers the most tiles that
//     M rows and `groups` groups can make; workgroups past the last leave;
//   * wgrad: one workgroup per tile of every group's matrix, summing over that
//     group's rows, the longest group's tiles first, so that the last ones to
//     end are short; each group's tiles are spread over the XCDs by
//     themselves, so a long group is not one XCD's alone;
//   * 256 x 256 or 192 x 256 tiles of 8 waves (128 or 96 x 64 each), or 128 x 128 of 8
//     waves (64 x 32, two workgroups per CU); K in slabs of 64 through two LDS stages, copied
//     with LDS-destined 128-bit loads one slab ahead; one barrier per slab, the
//     next k step's fragments read while the current one's MFMAs run;
//   * an operand whose rows run along k lies as [row][k] in LDS and is read
//     with 128-bit reads, one whose rows run along m or n as [k][row], read
//     with transposing reads (layouts: bf16_lds.hpp, without bank conflicts);
//   * the MFMA takes B first, so a lane holds 4 consecutive columns of C;
//   * edges: descriptors end where a group's rows and the matrices end, so rows
//     past them are zeros; k >= K of k-contiguous operands is zeroed in LDS.

#include "grouped_tiled.hpp"
#include "ops.hpp"

namespace dg {
namespace {

template <int BM, int BN, int WAVES_M, int WAVES_N>
hipError_t launch_tiles(const GroupedArgs& a, hipStream_t s) {
    const int64_t tn = (a.N + BN - 1) / BN;
    const int64_t tm = a.wgrad ? (a.K + BM - 1) / BM : row_tiles_bound(a.M, a.groups, BM);
    const int64_t grid = a.wgrad ? a.groups * tm * tn : tm * tn;
    if (grid > kMaxGrid) return hipErrorInvalidConfiguration;
    const bool epi = a.bias != nullptr || a.act != kActNone || a.row_scale != nullptr;
#define DG_G(...) &gemm_grouped_kernel<BM, BN, WAVES_M, WAVES_N, __VA_ARGS__>
    auto fn = a.wgrad ? (a.f32 ? DG_G(true, false, false, true) : DG_G(true, false, false, false))
              : a.tb  ? (epi ? DG_G(false, true, true, false) : DG_G(false, true, false, false))
                      : (epi ? DG_G(false, false, true, false) : DG_G(false, false, false, false));
#undef DG_G
    return launch_kernel(fn, dim3((unsigned)grid), dim3(WAVES_M * WAVES_N * 64), s, a, tm, tn);
}

// Modelled time (us) of `tiles` tiles of `slabs` slabs of K: whole rounds of
// `per_round` resident workgroups at `full` a slab, and the rest at `one` where
// they have a CU each, `two` where two share one; `edge` for every round's start
// and stores.
double rounds_us(double tiles, double slabs, int per_round, double full, double one, double two, double edge) {
    const double whole = (double)(int64_t)(tiles / per_round), rem = tiles - whole * per_round;
    const double last = rem < 0.5 ? 0.0 : rem <= 256 ? one : rem <= 512 ? two : full;
    return whole * (full * slabs + edge) + (rem < 0.5 ? 0.0 : last * slabs + edge);
}

// The tile size whose rounds of resident workgroups cost least, on 256 CUs (the
// whole card). The host does
// not know the groups' sizes: with M rows in E groups it counts on M / bm + E / 2
// row tiles (a last one for each group, half full), at least one for each group
// that can have rows. Measured on one MI355X (us; 256, 128 and 64 rows and
// columns to a tile). Rows, E x M x N x K: 16 x 16384 x 4096^2 520, 610, 1075;
// 8 x 8001 x 4096 x 2048 150, 170, 247; 8 x 4096 x 1024 x 2048 46.6, 28.7, 40.6;
// 32 x 1024 x 4096 x 2048 127, 132, 124; 8 x 16 x 1024 x 4096 83, 41, 34.
// Gradients: 16 x 16384 x 2048 x 4096 306, 407, 615; 8 x 999 x 1024^2 15.6, 10.2,
// 12.6; 8 x 8192 x 512^2 50, 27, 20; 2 x 16384 x 2048^2 224, 154, 239. 0 is the
// few-row kernel on tiles of 64 rows (rows only), one workgroup to a CU whose
// waves share K: with few tiles, 64 x 64 here and there: 4 x 400 x 1024 x 4096 34.2
// and 16.6, 2 x 1749 x 256 x 1536 15.2 and 9.2, 3 x 600 x 1024 x 3264 (B stored N x K)
// 27.4 and 13.2, 8 x 256 x 2048^2 20.4 and 16.8; 6 x 812 x 2560 x 1544 22.7 and 27.9.
// 192 rows by 256 columns (rows only), against 256: 8 x 8001 x 4096 x 2048 with B
// stored N x K 143 and 149, 4 x 12000 x 2816 x 2048 131 and 149, 8 x 5000 x 4096^2 184
// and 196, 2 x 2500 x 4096 x 2048 40 and 47; 16 x 16384 x 4096^2 522 and 517,
// 8 x 6000 x 4096 x 1024 66 and 56.
// A gradient's workgroup sums all of its group's rows, so few small matrices
// with many rows leave CUs empty: 2 x 16384 x 256^2 takes 74 us on 32 workgroups
// of 128 slabs, for 17 MB of operands; 2 x 16384 x 512^2 75, 8 x 16384 x 256^2 33.
int pick_tile(const GroupedArgs& a) {
    const double E = (double)a.groups, M = (double)a.M;
    auto edges = [](int64_t n, int b) { return (double)((n + b - 1) / b); };
    auto tiles = [&](int b) {
        if (a.wgrad) return E * edges(a.K, b) * edges(a.N, b);
        const double used = M < E ? M : E, cut = M / b + used / 2;
        return (double)(int64_t)(cut > used ? cut : used) * edges(a.N, b);
    };
    const double slabs = a.wgrad ? (M / E > 64 ? M / E / 64 : 1.0) : edges(a.K, 64);
    const double t256 = rounds_us(tiles(256), slabs, 256, 1.8, a.wgrad ? 1.8 : 1.3, 1.8, 8);
    const double t128 = rounds_us(tiles(128), slabs, 512, 1.18, 0.65, 1.1, 5);
    const double t64 = rounds_us(tiles(64), slabs, 1024, 1.05, 0.55, a.wgrad ? 0.6 : 1.05, 3);
    const double few = a.wgrad ? 1e30 : rounds_us(tiles(64), slabs, 256, 0.32, 0.24, 0.24, 4);
    if (few < t256 && few < t128 && few < t64) return 0;
    if (!a.wgrad) {
        const double t192 = rounds_us((double)(int64_t)(M / 192 + (M < E ? M : E) / 2) * edges(a.N, 256), slabs, 256, 1.5,
                                      1.1, 1.5, 6);
        if (t192 < t256 && t192 < t128 && t192 < t64) return 192;
    }
    return t256 <= t128 && t256 <= t64 ? 256 : t128 <= t64 ? 128 : 64;
}

}  // namespace

hipError_t launch_grouped(const GroupedArgs& a, int, hipStream_t s) {
    auto at16 = [](const void* q, int64_t stride, int esz) {
        return reinterpret_cast<uintptr_t>(q) % 16 == 0 && stride * esz % 16 == 0;
    };
    const int esz = a.f32 ? 4 : 2;
    const bool many = a.groups > 1;
    const bool rows16 = at16(a.A, a.lda, 2) && at16(a.B, a.ldb, 2) && at16(a.C, a.ldc, esz) &&
                        (!many || (a.wgrad ? a.stridec * esz % 16 == 0 : a.strideb * 2 % 16 == 0));
    // Offsets inside a tile's descriptors stay below 2^31: 256 rows plus K
    // elements of a k-contiguous operand, 64 rows plus their length otherwise.
    const int64_t lim = (int64_t)1 << 31;
    auto kc = [&](int64_t ld) { return (256 * ld + a.K) * 2 < lim; };
    auto mn = [&](int64_t ld, int64_t extent) { return (kBK * ld + 256 + extent) * 2 < lim; };
    const bool fits = 256 * a.ldc * esz < lim &&
                      (a.wgrad ? mn(a.lda, a.K) && mn(a.ldb, a.N)
                               : kc(a.lda) && (a.tb ? kc(a.ldb) : mn(a.ldb, a.N)));
    if (!rows16 || !fits) return launch_grouped_general(a, s);
    // Few rows for each group: the few-row kernel, on tiles of 16 rows where most
    // groups fit one and of 64 otherwise (us; 128 x 128 and 64 x 64 tiles, then
    // 16, 32 and 64 rows of the few-row kernel; E x M x N x K): 32 x 64 x 4096 x 2048
    // 84, 82, 82, 81, 87 and with B stored N x K 108, 104, 73, 81, 86;
    // 8 x 16 x 1024 x 4096 40.7, 34.4, 13.6, 13.8, 14.9; 64 x 512 x 1408 x 2048 79, 77,
    // 67, 74, 78; 8 x 128 x 2048^2 23.9, 20.3, 18.9, 15.3, 14.4; 16 x 512 x 2048^2 36.1,
    // 36.1, 52.7, 40.1, 36.7; 16 x 2048 x 1024 x 2048 24.9, 24.7, 41.4, 37.7, 29.8.
    if (!a.wgrad && a.M <= (int64_t)24 * a.groups)
        return launch_grouped_few(a, a.M <= 16 || a.M <= (int64_t)8 * a.groups ? 16 : 64, s);
    switch (pick_tile(a)) {
        case 256: return launch_tiles<256, 256, 2, 4>(a, s);
        case 192: return launch_grouped_192(a, s);
        case 128: return launch_tiles<128, 128, 2, 4>(a, s);
        case 0: return launch_grouped_few(a, 64, s);
        default: return launch_tiles<64, 64, 2, 2>(a, s);
    }
}

}  // namespace dg
