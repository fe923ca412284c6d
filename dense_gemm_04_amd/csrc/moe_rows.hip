// Rows between the tokens' order and the experts': gather, combine and its
// gradient. Each works from the tokens' side, so that a token's row is read (or
// written) once for all its choices.
//
//     gather    Y(slot_tj) = X(t)
//     combine   C(t) = R(t) + sum_j gate_tj Y(slot_tj)
//     gradient  dY(slot_tj) = gate_tj dC(t),  dgate_tj = dC(t) . Y(slot_tj)

#include "layer.hpp"

namespace dg {
namespace {

constexpr int kVec = Vec<uint16_t>::n;

__global__ __launch_bounds__(256) void gather(RowsArgs a) {
    for (int64_t t = blockIdx.x; t < a.tokens; t += gridDim.x)
        for (int64_t c = (int64_t)threadIdx.x * kVec; c < a.cols; c += 256 * kVec) {
            const int valid = inside(a.cols, c, kVec);
            Vec<uint16_t> x;
            x.load(a.X + t * a.ldx + c, valid);
            for (int j = 0; j < a.k; ++j) {
                const int64_t slot = a.slots[t * a.k + j];
                if (slot >= 0 && slot < a.rows) x.store(a.out + slot * a.ldo + c, valid);
            }
        }
}

__global__ __launch_bounds__(256) void combine(RowsArgs a) {
    for (int64_t t = blockIdx.x; t < a.tokens; t += gridDim.x)
        for (int64_t c = (int64_t)threadIdx.x * kVec; c < a.cols; c += 256 * kVec) {
            const int valid = inside(a.cols, c, kVec);
            Vec<uint16_t> v;
            float sum[kVec] = {};
            for (int j = 0; j < a.k; ++j) {
                const int64_t slot = a.slots[t * a.k + j];
                const bool there = slot >= 0 && slot < a.rows;
                const float gate = a.gates != nullptr ? a.gates[t * a.k + j] : 1.f;
                v.load(there ? a.Y + slot * a.ldy + c : a.Y, there ? valid : 0);
#pragma unroll
                for (int e = 0; e < kVec; ++e) sum[e] = __builtin_fmaf(gate, v.at(e), sum[e]);
            }
            if (a.X != nullptr) {
                v.load(a.X + t * a.ldx + c, valid);
#pragma unroll
                for (int e = 0; e < kVec; ++e) sum[e] += v.at(e);
            }
            v.set(sum);
            v.store(a.out + t * a.ldo + c, valid);
        }
}

__global__ __launch_bounds__(256) void combine_grad(RowsArgs a) {
    __shared__ float part[4];
    for (int64_t t = blockIdx.x; t < a.tokens; t += gridDim.x)
        for (int j = 0; j < a.k; ++j) {
            const int64_t slot = a.slots[t * a.k + j];
            const bool there = slot >= 0 && slot < a.rows;
            const float gate = a.gates != nullptr ? a.gates[t * a.k + j] : 1.f;
            float dot = 0.f;
            if (there)
                for (int64_t c = (int64_t)threadIdx.x * kVec; c < a.cols; c += 256 * kVec) {
                    const int valid = inside(a.cols, c, kVec);
                    Vec<uint16_t> dc, y;
                    float dy[kVec];
                    dc.load(a.X + t * a.ldx + c, valid);
                    if (a.dgates != nullptr) {
                        y.load(a.Y + slot * a.ldy + c, valid);
#pragma unroll
                        for (int e = 0; e < kVec; ++e) dot = __builtin_fmaf(dc.at(e), y.at(e), dot);
                    }
#pragma unroll
                    for (int e = 0; e < kVec; ++e) dy[e] = gate * dc.at(e);
                    y.set(dy);
                    y.store(a.out + slot * a.ldo + c, valid);
                }
            if (a.dgates == nullptr) continue;
            dot = wave_sum(dot);
            __syncthreads();
            if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = dot;
            __syncthreads();
            if (threadIdx.x == 0) a.dgates[t * a.k + j] = (part[0] + part[1]) + (part[2] + part[3]);
        }
}

}  // namespace

hipError_t launch_gather(const RowsArgs& a, hipStream_t s) {
    return launch_kernel(&gather, dim3(grid_for(a.tokens)), dim3(256), s, a);
}
hipError_t launch_combine(const RowsArgs& a, hipStream_t s) {
    return launch_kernel(&combine, dim3(grid_for(a.tokens)), dim3(256), s, a);
}
hipError_t launch_combine_grad(const RowsArgs& a, hipStream_t s) {
    return launch_kernel(&combine_grad, dim3(grid_for(a.tokens)), dim3(256), s, a);
}

}  // namespace dg
