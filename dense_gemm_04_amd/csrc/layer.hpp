// Layer norm, dropout, the router and its rows (internal to the library):
// arguments, launchers, and what their kernels share.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "common.hpp"
#include "ops.hpp"

namespace dg {

template <typename T>
struct NormArgs {
    int64_t rows, cols;
    float eps;
    const T* X; int64_t ldx;
    const T* weight;                // or null
    const T* bias;                  // or null
    T* Y; int64_t ldy;
    float* mean;                    // or null
    float* rstd;                    // or null
};
hipError_t launch_layernorm(const NormArgs<uint16_t>& a, hipStream_t s);
hipError_t launch_layernorm(const NormArgs<float>& a, hipStream_t s);

template <typename T>
struct NormGradArgs {
    int64_t rows, cols;
    const T* X; int64_t ldx;
    const T* weight;                // or null
    const float* mean;
    const float* rstd;
    const T* dY; int64_t lddy;
    const T* R; int64_t ldr;        // or null
    T* dX; int64_t lddx;
    float beta;
    float* dweight;                 // or null
    float* dbias;                   // or null
    float* ws;                      // layernorm_grad_workspace bytes, where dweight or dbias is wanted
};
size_t layernorm_grad_workspace(int64_t rows, int64_t cols);
hipError_t launch_layernorm_grad(const NormGradArgs<uint16_t>& a, hipStream_t s);
hipError_t launch_layernorm_grad(const NormGradArgs<float>& a, hipStream_t s);

template <typename T>
struct DropoutArgs {
    int64_t rows, cols;
    uint32_t drop;                  // of 65536
    const uint64_t* rng;
    const T* X; int64_t ldx;
    const T* R; int64_t ldr;        // or null
    T* Y; int64_t ldy;
};
hipError_t launch_dropout(const DropoutArgs<uint16_t>& a, hipStream_t s);
hipError_t launch_dropout(const DropoutArgs<float>& a, hipStream_t s);

constexpr int kMaxExperts = 1024, kMaxChoices = 16;

template <typename T>
struct RouteArgs {
    int tokens, experts, k;
    bool renormalize;
    const T* logits; int64_t ldl;
    float* gates;
    int32_t* choice;
    int32_t* slots;
    int32_t* offsets;
    int32_t* counts;
    float* loss;                    // or null
    void* ws;                       // route_workspace bytes
};
size_t route_workspace(int64_t tokens, int64_t experts, int k);
hipError_t launch_route(const RouteArgs<uint16_t>& a, hipStream_t s);
hipError_t launch_route(const RouteArgs<float>& a, hipStream_t s);

template <typename T>
struct RouteGradArgs {
    int tokens, experts, k;
    bool renormalize;
    const T* logits; int64_t ldl;
    const int32_t* choice;
    const int32_t* counts;
    const float* dgates;            // or null
    const float* dloss;             // or null
    T* dlogits; int64_t lddl;
};
hipError_t launch_route_grad(const RouteGradArgs<uint16_t>& a, hipStream_t s);
hipError_t launch_route_grad(const RouteGradArgs<float>& a, hipStream_t s);

// Rows between the tokens' order (X, R, C, dC: tokens x cols) and the experts'
// (Y, dY: rows x cols).
struct RowsArgs {
    int64_t tokens, cols, rows;
    int k;
    const int32_t* slots;
    const float* gates;                      // or null: 1
    const uint16_t* X; int64_t ldx;          // gather: X; combine: R or null; gradient: dC
    const uint16_t* Y; int64_t ldy;          // combine, gradient
    uint16_t* out; int64_t ldo;              // gather: Y; combine: C; gradient: dY
    float* dgates;                           // gradient, or null
    bool once;                               // Y's rows are whole cache lines, read past the caches
};
hipError_t launch_gather(const RowsArgs& a, hipStream_t s);
hipError_t launch_combine(const RowsArgs& a, hipStream_t s);
hipError_t launch_combine_grad(const RowsArgs& a, hipStream_t s);

// ---- device helpers -----------------------------------------------------------

// Vectors of 16 bytes: 8 bf16 or 4 fp32 values, at addresses aligned to their
// element (one 128-bit access either way). Elements at `valid` and past it are
// read as zero and not written.
template <typename T>
struct Vec;
template <>
struct Vec<uint16_t> {
    static constexpr int n = 8;
    u32x4 w;
    __device__ __forceinline__ float at(int e) const {
        return __builtin_bit_cast(float, (e & 1) ? (w[e >> 1] & 0xffff0000u) : (w[e >> 1] << 16));
    }
    __device__ __forceinline__ void load(const uint16_t* p, int valid) {
        if (valid >= 8) {
            w = *reinterpret_cast<const u32x4_a2*>(p);
            return;
        }
#pragma unroll
        for (int q = 0; q < 4; ++q)
            w[q] = (2 * q < valid ? (uint32_t)p[2 * q] : 0u) | ((2 * q + 1 < valid ? (uint32_t)p[2 * q + 1] : 0u) << 16);
    }
    // A whole vector that is not kept in the caches.
    __device__ __forceinline__ void load_once(const uint16_t* p) {
        w = __builtin_nontemporal_load(reinterpret_cast<const u32x4_a2*>(p));
    }
    __device__ __forceinline__ void set(const float* v) {
#pragma unroll
        for (int q = 0; q < 4; ++q) w[q] = pack_bf16x2(v[2 * q], v[2 * q + 1]);
    }
    __device__ __forceinline__ void store(uint16_t* p, int valid) const {
        if (valid >= 8) {
            *reinterpret_cast<u32x4_a2*>(p) = w;
            return;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < valid) store1(p + e, e);
    }
    __device__ __forceinline__ void store1(uint16_t* p, int e) const { *p = (uint16_t)(w[e >> 1] >> (16 * (e & 1))); }
};
template <>
struct Vec<float> {
    static constexpr int n = 4;
    f32x4 w;
    __device__ __forceinline__ float at(int e) const { return w[e]; }
    __device__ __forceinline__ void load(const float* p, int valid) {
        if (valid >= 4) {
            w = *reinterpret_cast<const f32x4_a4*>(p);
            return;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = e < valid ? p[e] : 0.f;
    }
    __device__ __forceinline__ void set(const float* v) {
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = v[e];
    }
    __device__ __forceinline__ void store(float* p, int valid) const {
        if (valid >= 4) {
            *reinterpret_cast<f32x4_a4*>(p) = w;
            return;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (e < valid) p[e] = w[e];
    }
    __device__ __forceinline__ void store1(float* p, int e) const { *p = w[e]; }
};

// Elements of a vector at column c0 that lie inside a row of `cols`.
__device__ __forceinline__ int inside(int64_t cols, int64_t c0, int n) {
    const int64_t left = cols - c0;
    return left >= n ? n : (left > 0 ? (int)left : 0);
}

// Where a lane's vector at column c of a row of `cols` >= n values is read: the
// last n of the row where it would pass their end, so that no lane reads
// element by element; its first `skip` elements then belong to the vector
// before (all of them where c lies past the end).
struct LastVec {
    int from, skip;
};
__device__ __forceinline__ LastVec last_vec(int cols, int c, int n) {
    const int from = c + n <= cols ? c : cols - n;
    return LastVec{from, c - from < n ? c - from : n};
}

// Lane exchanges that the vector unit does on its own (DPP): sums over 16
// neighbouring lanes, in all of them, and over the wave, as a scalar.
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_add(float v) {
    return v + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, ROWS, 0xf, false));
}
__device__ __forceinline__ float sum_of_16(float v) {
    v = dpp_add<0xB1, 0xf>(v);         // lane ^ 1
    v = dpp_add<0x4E, 0xf>(v);         // lane ^ 2
    v = dpp_add<0x141, 0xf>(v);        // mirrored in 8
    return dpp_add<0x140, 0xf>(v);     // mirrored in 16
}
__device__ __forceinline__ float wave_sum(float v) {
    v = sum_of_16(v);
    v = dpp_add<0x142, 0xa>(v);        // rows 1 and 3 take the row before
    v = dpp_add<0x143, 0xc>(v);        // rows 2 and 3 take the first half
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 63));
}
// Sums of two values over the wave, as scalars: half the lanes go on with each.
__device__ __forceinline__ void wave_sums(float& a, float& b) {
    const auto w = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b),
                                                    false, false);
    const uint32_t x = w[0], y = w[1];                 // lower half: a's, upper half: b's
    float v = sum_of_16(__builtin_bit_cast(float, x) + __builtin_bit_cast(float, y));
    v = dpp_add<0x142, 0xa>(v);
    a = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 31));
    b = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 63));
}

// A value and that of the lane 16 or 32 lanes away: of both results, one is v
// and the other the partner's, alike in both lanes.
template <int APART>
__device__ __forceinline__ void both_lanes(uint32_t v, uint32_t& x, uint32_t& y) {
    if constexpr (APART == 16) {
        const auto b = __builtin_amdgcn_permlane16_swap(v, v, false, false);
        x = b[0];
        y = b[1];
    } else {
        const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        x = b[0];
        y = b[1];
    }
}
template <int APART>
__device__ __forceinline__ float add_lanes(float v) {
    uint32_t x, y;
    both_lanes<APART>(__builtin_bit_cast(uint32_t, v), x, y);
    return __builtin_bit_cast(float, x) + __builtin_bit_cast(float, y);
}

// What a wave's lanes wrote to LDS before is seen by its other lanes behind. They
// run in step, so this costs no instruction: it keeps the compiler from moving
// LDS accesses across.
__device__ __forceinline__ void lds_wave_barrier() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
}

// Workgroups for `units` independent pieces: as many, up to what a grid
// dimension takes; the kernels stride over the rest.
inline unsigned grid_for(int64_t units) {
    constexpr int64_t kMost = 1 << 20;
    return (unsigned)(units < 1 ? 1 : (units < kMost ? units : kMost));
}

}  // namespace dg
