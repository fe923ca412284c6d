// Rows between the tokens' order and the experts': gather, combine and its
// gradient. Each works from the tokens' side, so that a token's row is read (or
// written) once for all its choices.
//
//     gather    Y(slot_tj) = X(t)
//     combine   C(t) = R(t) + sum_j gate_tj Y(slot_tj)
//     gradient  dY(slot_tj) = gate_tj dC(t),  dgate_tj = dC(t) . Y(slot_tj)
//
// Bound by memory. A token's k slots are read first and held in scalar registers
// (K: k rounded up to a power of two), so that the k rows' loads of whole vectors
// leave together. One MI355X: gather of 8191 x 4096, 2 choices 38.6 us (5.2 TB/s),
// combine of 4096 x 2048, 8 choices 29.4 (5.7), its gradient of 8192 x 4096, 2
// choices 64 (5.3).
//
// Where that does not hold: a row's last, partial vector is read element by
// element, one choice after the other (4096 x 2047, 8 choices: gather 45 us, combine 51,
// gradient 117, against 32, 30 and 63 for 2048 columns); combine of more than 8
// choices keeps its rows in private memory (4096 x 2048, 16 choices 147 us, its
// bytes 60); and rows much narrower than the 2048 columns of a workgroup leave
// threads idle (16384 x 256, 8 choices: 28, 35 and 86 us for bytes of 15, 17 and 28).

#include "layer.hpp"

namespace dg {
namespace {

constexpr int kVec = Vec<uint16_t>::n;
constexpr int kColumns = 256 * kVec;             // of a workgroup at a time

// A vector of a sorted row. Its last reader in a pass is combine, and in the
// backward pass combine's gradient, so rows of whole cache lines are read past
// the caches and leave what is there to the next products. One MI355X, 16 experts, cached
// and past the caches: product, combine and norm of 2048 tokens x 2048, 8 choices 182 and
// 174 us, of 8192 x 4096, 2 choices 620 and 616; the gradient, its product and the sum after
// it 195 and 175, 638 and 618; alone, combine of 4096 x 2048, 8 choices 34.5 and
// 29.4. Rows that share lines lose by it (a pass over rows of 4092 bytes 13.4 and 17.6).
// Stores past the caches are not used: alone they gain more (gather of 8191 x 4096,
// 2 choices 41 and 31), but the product that reads the rows next loses it (with it 556
// and 566).
__device__ __forceinline__ void load_sorted(Vec<uint16_t>& v, const RowsArgs& a, int slot, int64_t c, int valid) {
    const uint16_t* p = a.Y + slot * a.ldy + c;
    if (a.once) v.load_once(p);
    else v.load(p, valid);
}

// A token's slots as scalars: -1 where absent, outside the rows or past k.
template <int K>
__device__ __forceinline__ void load_slots(const RowsArgs& a, int64_t t, int* slot) {
#pragma unroll
    for (int j = 0; j < K; ++j) slot[j] = a.slots[t * a.k + (j < a.k ? j : 0)];
#pragma unroll
    for (int j = 0; j < K; ++j) {
        slot[j] = __builtin_amdgcn_readfirstlane(slot[j]);
        if (j >= a.k || slot[j] < 0 || slot[j] >= a.rows) slot[j] = -1;
    }
}
template <int K>
__device__ __forceinline__ void load_gates(const RowsArgs& a, int64_t t, float* gate) {
#pragma unroll
    for (int j = 0; j < K; ++j) gate[j] = j >= a.k ? 0.f : (a.gates != nullptr ? a.gates[t * a.k + j] : 1.f);
}

template <int K>
__device__ __forceinline__ void gather_one(const RowsArgs& a, int64_t t, int64_t c) {
    const int valid = inside(a.cols, c, kVec);
    Vec<uint16_t> x;
    x.load(a.X + t * a.ldx + (valid > 0 ? c : 0), valid);
    int slot[K];
    load_slots<K>(a, t, slot);
    if (valid == 0) return;
#pragma unroll
    for (int j = 0; j < K; ++j)
        if (slot[j] >= 0) x.store(a.out + slot[j] * a.ldo + c, valid);
}

template <int K>
__device__ __forceinline__ void combine_one(const RowsArgs& a, int64_t t, int64_t c) {
    const int valid = inside(a.cols, c, kVec);
    int slot[K];
    float gate[K];
    load_slots<K>(a, t, slot);
    load_gates<K>(a, t, gate);
    if (valid == 0) return;
    Vec<uint16_t> y[K], r;
    float sum[kVec] = {};
#pragma unroll
    for (int j = 0; j < K; ++j) {
        y[j].w = u32x4{0, 0, 0, 0};
        if (slot[j] >= 0) load_sorted(y[j], a, slot[j], c, valid);
    }
    if (a.X != nullptr) r.load(a.X + t * a.ldx + c, valid);
#pragma unroll
    for (int j = 0; j < K; ++j) {
        if (j >= a.k) break;
#pragma unroll
        for (int e = 0; e < kVec; ++e) sum[e] = __builtin_fmaf(gate[j], y[j].at(e), sum[e]);
    }
    if (a.X != nullptr) {
#pragma unroll
        for (int e = 0; e < kVec; ++e) sum[e] += r.at(e);
    }
    r.set(sum);
    r.store(a.out + t * a.ldo + c, valid);
}

// A workgroup takes kColumns columns of a token (tokens over grid.y; both
// strides are for sizes past the grid).
template <int K, bool COMBINE>
__global__ __launch_bounds__(256) void rows(RowsArgs a) {
    for (int64_t t = blockIdx.y; t < a.tokens; t += gridDim.y)
        for (int64_t c0 = (int64_t)blockIdx.x * kColumns; c0 < a.cols; c0 += (int64_t)gridDim.x * kColumns) {
            if constexpr (COMBINE) combine_one<K>(a, t, c0 + threadIdx.x * kVec);
            else gather_one<K>(a, t, c0 + threadIdx.x * kVec);
        }
}

// A token's gradients, by a workgroup: the products with all its rows are sums
// over the whole row. part: LDS that the token before did not use.
template <int K>
__device__ __forceinline__ void combine_grad_one(const RowsArgs& a, int64_t t, float (*part)[K]) {
    int slot[K];
    float gate[K], dot[K] = {};
    load_slots<K>(a, t, slot);
    load_gates<K>(a, t, gate);
    for (int64_t c = threadIdx.x * kVec; c < a.cols; c += kColumns) {
        const int valid = inside(a.cols, c, kVec);
        Vec<uint16_t> dc, y[K];
        dc.load(a.X + t * a.ldx + c, valid);
        if (a.dgates != nullptr) {
#pragma unroll
            for (int j = 0; j < K; ++j) {
                y[j].w = u32x4{0, 0, 0, 0};
                if (slot[j] >= 0) load_sorted(y[j], a, slot[j], c, valid);
            }
        }
#pragma unroll
        for (int j = 0; j < K; ++j) {
            if (slot[j] < 0) continue;
            float dy[kVec];
            if (a.dgates != nullptr) {
#pragma unroll
                for (int e = 0; e < kVec; ++e) dot[j] = __builtin_fmaf(dc.at(e), y[j].at(e), dot[j]);
            }
#pragma unroll
            for (int e = 0; e < kVec; ++e) dy[e] = gate[j] * dc.at(e);
            y[j].set(dy);
            y[j].store(a.out + slot[j] * a.ldo + c, valid);
        }
    }
    if (a.dgates == nullptr) return;
#pragma unroll
    for (int j = 0; j < K; ++j) {
        const float s = wave_sum(dot[j]);
        if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6][j] = s;
    }
    lds_only_barrier();
    const int j = threadIdx.x;
    if (j < a.k) a.dgates[t * a.k + j] = (part[0][j] + part[1][j]) + (part[2][j] + part[3][j]);
}

template <int K>
__global__ __launch_bounds__(256) void combine_grad(RowsArgs a) {
    __shared__ float part[2][4][K];
    int turn = 0;
    for (int64_t t = blockIdx.x; t < a.tokens; t += gridDim.x, turn ^= 1) combine_grad_one<K>(a, t, part[turn]);
}

// K: k rounded up to a power of two.
template <typename F>
hipError_t with_choices(int k, F&& launch) {
    if (k == 1) return launch(std::integral_constant<int, 1>{});
    if (k == 2) return launch(std::integral_constant<int, 2>{});
    if (k <= 4) return launch(std::integral_constant<int, 4>{});
    if (k <= 8) return launch(std::integral_constant<int, 8>{});
    return launch(std::integral_constant<int, 16>{});
}

bool whole_lines(const RowsArgs& a) {
    constexpr int64_t kLine = 128;
    return reinterpret_cast<uintptr_t>(a.Y) % kLine == 0 && 2 * a.ldy % kLine == 0 && 2 * a.cols % kLine == 0;
}

dim3 rows_grid(const RowsArgs& a) {
    const int64_t chunks = (a.cols + kColumns - 1) / kColumns;
    return dim3((unsigned)(chunks < 64 ? chunks : 64), (unsigned)(a.tokens < 65535 ? a.tokens : 65535));
}

}  // namespace

hipError_t launch_gather(const RowsArgs& a, hipStream_t s) {
    return with_choices(a.k, [&](auto k) { return launch_kernel(&rows<k(), false>, rows_grid(a), dim3(256), s, a); });
}
hipError_t launch_combine(const RowsArgs& args, hipStream_t s) {
    RowsArgs a = args;
    a.once = whole_lines(a);
    return with_choices(a.k, [&](auto k) { return launch_kernel(&rows<k(), true>, rows_grid(a), dim3(256), s, a); });
}
hipError_t launch_combine_grad(const RowsArgs& args, hipStream_t s) {
    RowsArgs a = args;
    a.once = whole_lines(a);
    return with_choices(a.k, [&](auto k) {
        return launch_kernel(&combine_grad<k()>, dim3(grid_for(a.tokens)), dim3(256), s, a);
    });
}

}  // namespace dg
