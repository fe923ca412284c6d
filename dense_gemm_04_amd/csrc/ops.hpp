// Host-side launchers of the 8-bit and the grouped operators (internal to the
// library; the dense products' are in kernels.hpp).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <tuple>

#include "fp8.hpp"
#include "grouped.hpp"
#include "kernels.hpp"

namespace dg {

// Launches a kernel with its arguments converted to its parameter types, and
// returns that launch's own status (not an error left by an earlier call).
template <typename... P, typename... A>
hipError_t launch_kernel(void (*fn)(P...), dim3 grid, dim3 block, hipStream_t s, A... args) {
    std::tuple<P...> vals(static_cast<P>(args)...);
    return std::apply(
        [&](auto&... v) {
            void* kargs[] = {static_cast<void*>(&v)...};
            return hipLaunchKernel(reinterpret_cast<const void*>(fn), grid, block, kargs, 0, s);
        },
        vals);
}

// Quantisation to e4m3 (quantize_fp8.hip): Q is rows x cols, or with
// `transpose` cols x rows; blocks of 128 along Q's rows by block_rows of them.
template <typename T>
struct QuantArgs {
    bool transpose;
    int block_rows;                 // 1 or 128
    int64_t rows, cols;             // of X
    const T* X; int64_t ldx;
    uint8_t* Q; int64_t ldq;
    float* S; int64_t lds;
};
hipError_t launch_quantize(const QuantArgs<uint16_t>& a, hipStream_t s);
hipError_t launch_quantize(const QuantArgs<float>& a, hipStream_t s);

// The 8-bit block-scaled product: rows of A and B aligned to 16 bytes and of C
// to 8, or any alignment (general).
hipError_t launch_fp8(const Fp8Args& a, int cus, hipStream_t s);
hipError_t launch_fp8_general(const Fp8Args& a, hipStream_t s);
hipError_t launch_fp8_few(const Fp8Args& a, hipStream_t s);

// Products grouped by expert and their weight gradients.
hipError_t launch_grouped(const GroupedArgs& a, int cus, hipStream_t s);
hipError_t launch_grouped_general(const GroupedArgs& a, hipStream_t s);
hipError_t launch_grouped_192(const GroupedArgs& a, hipStream_t s);    // rows only, called by launch_grouped
// Groups of few rows (rows only; alignment as for launch_grouped): tiles of 16
// or 64 rows by 64 columns, K split over the waves of a workgroup.
hipError_t launch_grouped_few(const GroupedArgs& a, int rows, hipStream_t s);

}  // namespace dg
