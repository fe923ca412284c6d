// Row groups of the products grouped by expert: arguments, and the search for
// the group that a tile of rows belongs to.
#pragma once

#include "common.hpp"

namespace dg {

// Rows offsets[e] .. offsets[e + 1] - 1 belong to group e.
//   rows (wgrad == false): C(i,:) <- act(alpha row_scale[i] A(i,:) B_e + bias_e) + beta C(i,:)
//   wgrad:                 C_e <- alpha A_e^T B_e + beta C_e, A_e and B_e the group's rows
struct GroupedArgs {
    bool wgrad;
    int groups;
    int64_t M, N, K;                         // rows of A; columns of C; columns of A
    float alpha, beta;
    const uint16_t* A; int64_t lda;
    const uint16_t* B; int64_t ldb;          // rows: group e's matrix at B + e * strideb
    int64_t strideb;
    void* C; int64_t ldc;                    // wgrad: group e's matrix at C + e * stridec
    int64_t stridec;
    const int32_t* offsets;
    bool tb;                                 // rows: B_e stored N x K
    bool f32;                                // wgrad: C in fp32, bf16 otherwise
    const float* row_scale;
    const uint16_t* bias; int64_t stridebias;
    int act;
};

// Group e's rows [lo, hi), cut to [0, M) whatever the offsets hold: a kernel
// then stays inside its operands even where the offsets are not valid.
__device__ __forceinline__ void group_range(const int32_t* offsets, int e, int M, int& lo, int& hi) {
    const int a = offsets[e], b = offsets[e + 1];
    lo = a < 0 ? 0 : (a > M ? M : a);
    hi = b < lo ? lo : (b > M ? M : b);
}

// Tiles of bm rows of every group, numbered in group order. Their number is at
// most M / bm + groups when the offsets are valid (each group adds at most one
// tile that is not full).
inline int64_t row_tiles_bound(int64_t M, int64_t groups, int bm) {
    const int64_t by_groups = M / bm + groups;
    return by_groups < M ? by_groups : M;
}

__device__ __forceinline__ int wave_scan(int v, int lane) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int u = __shfl_up(v, d, 64);
        v += lane >= d ? u : 0;
    }
    return v;
}

// The number of row tiles of all groups (every lane of the wave calls it).
__device__ __forceinline__ int count_row_tiles(const int32_t* offsets, int groups, int M, int bm, int lane) {
    int total = 0;
    for (int base = 0; base < groups; base += 64) {
        int lo = 0, hi = 0;
        if (base + lane < groups) group_range(offsets, base + lane, M, lo, hi);
        total += (int)(((unsigned)(hi - lo) + bm - 1) / bm);
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) total += __shfl_xor(total, d, 64);
    return __builtin_amdgcn_readfirstlane(total);
}

struct RowTile {
    int group;       // -1: no such tile
    int m0;          // first row
    int end;         // the group's end: rows m0 .. min(end, m0 + bm) - 1
};

// Row tile `id`, found by one wave: 64 groups at a time, a prefix sum of their
// tile counts and a ballot of the groups whose sum passes `id`.
__device__ __forceinline__ RowTile find_row_tile(const int32_t* offsets, int groups, int M, int bm, int id, int lane) {
    for (int base = 0; base < groups; base += 64) {
        int lo = 0, hi = 0;
        if (base + lane < groups) group_range(offsets, base + lane, M, lo, hi);
        const int mine = (int)(((unsigned)(hi - lo) + bm - 1) / bm);
        const int upto = wave_scan(mine, lane);
        const unsigned long long past = __ballot(upto > id);
        if (past != 0) {
            const int w = __builtin_ctzll(past);
            const int first = __builtin_amdgcn_readlane(upto - mine, w);
            RowTile t;
            t.group = __builtin_amdgcn_readfirstlane(base + w);
            t.m0 = __builtin_amdgcn_readfirstlane(__builtin_amdgcn_readlane(lo, w) + (id - first) * bm);
            t.end = __builtin_amdgcn_readfirstlane(__builtin_amdgcn_readlane(hi, w));
            return t;
        }
        id -= __builtin_amdgcn_readlane(upto, 63);
    }
    return RowTile{-1, 0, 0};
}

// The row tile and column of this workgroup: tiles of bm rows by tiles_n
// columns of tiles, spread over the XCDs in contiguous runs. A group's tiles lie
// together and are walked column by column in bands of up to `band` of its row
// tiles, so that neighbours share their expert's columns and their rows. lo, hi: the
// rows of group `lane` (group_range), from which the tile's group is found where
// there are at most 64; with more the offsets are read again and the bands
// run over the groups' ends.
struct RowPlace {
    RowTile tile;
    int tn;
};
__device__ __forceinline__ RowPlace place_row_tile(const int32_t* offsets, int groups, int M, int bm, int tiles_n,
                                                   int band, int lo, int hi, int lane) {
    const int mine = (int)(((unsigned)(hi - lo) + bm - 1) / bm);
    const int upto = wave_scan(mine, lane);
    const bool in_lanes = groups <= 64;
    const int have = in_lanes ? __builtin_amdgcn_readlane(upto, 63) : count_row_tiles(offsets, groups, M, bm, lane);
    const int64_t all = (int64_t)have * tiles_n;
    RowPlace w{RowTile{-1, 0, 0}, 0};
    if ((int64_t)blockIdx.x >= all) return w;
    const int id = xcd_slot((int)blockIdx.x, (int)(all < gridDim.x ? all : gridDim.x));
    int tm;
    if (in_lanes) {
        const int e = __builtin_ctzll(__ballot((int64_t)upto * tiles_n > id));
        const int of = __builtin_amdgcn_readlane(mine, e), first = __builtin_amdgcn_readlane(upto, e) - of;
        const int bands = (of + band - 1) / band;
        raster_tile(id - first * tiles_n, of, tiles_n, (of + bands - 1) / bands, tm, w.tn);
        w.tile.group = e;
        w.tile.end = __builtin_amdgcn_readlane(hi, e);
        w.tile.m0 = __builtin_amdgcn_readlane(lo, e) + tm * bm;
    } else {
        raster_tile(id, have, tiles_n, band, tm, w.tn);
        w.tile = find_row_tile(offsets, groups, M, bm, tm, lane);
    }
    return w;
}

}  // namespace dg
