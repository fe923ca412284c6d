// Quantisation to e4m3 with one fp32 scale per block of 128 values along the
// dimension a product sums over (or per 128 x 128 block):
//
//     top = max(largest |x| of the block, 448 * 2^-126)
//     S   = top / 448,   Q = e4m3(448 x / top), to nearest, ties to even.
//
// A block that holds an infinity or a NaN gets S = NaN and Q = 0, so a product
// that reads it gives NaN in the rows it belongs to and nowhere else.
//
// The quotient: with bf16 inputs 448 x / top is often exactly half way between
// two e4m3 values, where a product with a rounded reciprocal would fall to
// either side. Each element therefore takes one correction step,
//     q0 = y r,  q = q0 + (y - q0 t) r   (y = 0.875 x, t = top / 512, r ~ 1/t),
// whose two fused multiply-adds give the correctly rounded quotient; y is exact
// for bf16, never overflows, and r stays a normal number for every top. Where
// top is below 2^-60, y and t are both taken 2^64 times as large: y - q0 t can
// be 2^-34 of t where q is small, and has to be held exactly (a residual lost
// below the smallest fp32 number would leave q on either side of a tie).
//
// Bound by memory: one read of X and one write of Q, every value held in
// registers between the two; 4 fp32 operations, an unpack and half a
// conversion per element, below half of what the vector units do in the time
// of the copy.

#include "fp8.hpp"
#include "ops.hpp"

namespace dg {
namespace {

// Eight consecutive elements as they lie in memory.
template <typename T>
struct Raw8;
template <>
struct Raw8<uint16_t> {
    u32x4 w;
    __device__ __forceinline__ float at(int e) const {
        return __builtin_bit_cast(float, (e & 1) ? (w[e >> 1] & 0xffff0000u) : (w[e >> 1] << 16));
    }
};
template <>
struct Raw8<float> {
    f32x4 lo, hi;
    __device__ __forceinline__ float at(int e) const { return e < 4 ? lo[e] : hi[e - 4]; }
};

// `wide`: p is 16-byte aligned. Elements at `valid` and past it are zero.
__device__ __forceinline__ Raw8<uint16_t> load8(const uint16_t* p, int valid, bool wide) {
    Raw8<uint16_t> x;
    if (valid >= 8) {
        x.w = wide ? *reinterpret_cast<const u32x4*>(p) : (u32x4)*reinterpret_cast<const u32x4_a2*>(p);
        return x;
    }
#pragma unroll
    for (int q = 0; q < 4; ++q)
        x.w[q] = (2 * q < valid ? (uint32_t)p[2 * q] : 0u) |
                 ((2 * q + 1 < valid ? (uint32_t)p[2 * q + 1] : 0u) << 16);
    return x;
}
__device__ __forceinline__ Raw8<float> load8(const float* p, int valid, bool wide) {
    Raw8<float> x;
    if (valid >= 8) {
        x.lo = wide ? *reinterpret_cast<const f32x4*>(p) : (f32x4)*reinterpret_cast<const f32x4_a4*>(p);
        x.hi = wide ? *reinterpret_cast<const f32x4*>(p + 4) : (f32x4)*reinterpret_cast<const f32x4_a4*>(p + 4);
        return x;
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        x.lo[q] = q < valid ? p[q] : 0.f;
        x.hi[q] = 4 + q < valid ? p[4 + q] : 0.f;
    }
    return x;
}

// Magnitudes as integers: they order like the values, infinities above every
// finite one and NaNs above those.
__device__ __forceinline__ uint32_t mag(float x) { return __builtin_bit_cast(uint32_t, x) & 0x7fffffffu; }
__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t top8(const Raw8<uint16_t>& x) {
    u16x2 m = {0, 0};
#pragma unroll
    for (int q = 0; q < 4; ++q)
        m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, x.w[q] & 0x7fff7fffu));
    return (uint32_t)(m[0] > m[1] ? m[0] : m[1]) << 16;
}
__device__ __forceinline__ uint32_t top8(const Raw8<float>& x) {
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) m = umax(m, mag(x.at(e)));
    return m;
}

struct Block {
    float t, r, s;     // top / 512 (times 2^64 where top is small), its reciprocal, the scale
    float f;           // y = f x
    bool bad;          // an infinity or NaN in the block
};

__device__ __forceinline__ Block block_of(uint32_t bits) {
    Block b;
    b.bad = bits >= 0x7f800000u;
    float top = __builtin_bit_cast(float, bits);
    top = (b.bad || top < kMinTop) ? kMinTop : top;
    b.s = b.bad ? __builtin_nanf("") : top / kE4m3Max;
    const bool small = top < 0x1p-60f;
    b.f = small ? 0.875f * 0x1p64f : 0.875f;
    b.t = top * (small ? 0x1p55f : 0x1p-9f);
    b.r = 1.f / b.t;
    return b;
}

__device__ __forceinline__ float quotient(float x, const Block& b) {
    const float y = b.f * x, q0 = y * b.r;
    return __builtin_fmaf(__builtin_fmaf(-q0, b.t, y), b.r, q0);
}

__device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d, bool bad) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
    return bad ? 0u : (uint32_t)w;
}

// Largest of 16 neighbouring lanes, in all of them.
__device__ __forceinline__ uint32_t top_of_16(uint32_t m) {
#pragma unroll
    for (int d = 1; d < 16; d <<= 1) m = umax(m, (uint32_t)__shfl_xor((int)m, d, 64));
    return m;
}

__device__ __forceinline__ void store8(uint8_t* p, uint32_t lo, uint32_t hi, int valid, bool wide) {
    if (valid >= 8 && wide) {
        *reinterpret_cast<u32x2*>(p) = u32x2{lo, hi};
        return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (e < valid) p[e] = (uint8_t)((e < 4 ? lo >> (8 * e) : hi >> (8 * e - 32)) & 0xffu);
}

// Blocks of 1 x 128 along the rows of X: 16 lanes take a block, 8 values each.
// One workgroup of 256 threads takes 16 blocks of one row; rows stride over
// grid.y.
template <typename T>
__global__ __launch_bounds__(256) void quantize_rows(int64_t rows, int64_t cols, const T* X, int64_t ldx,
                                                     uint8_t* Q, int64_t ldq, float* S, int64_t lds, bool wide) {
    const int64_t kb = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4);
    const int64_t c0 = kb * kScaleBlock + (threadIdx.x & 15) * 8;
    for (int64_t row = blockIdx.y; row < rows; row += gridDim.y) {
        const int64_t left = cols - c0;
        const int valid = left >= 8 ? 8 : (left > 0 ? (int)left : 0);
        const Raw8<T> x = load8(X + row * ldx + (valid > 0 ? c0 : 0), valid, wide);
        const Block b = block_of(top_of_16(top8(x)));
        float q[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) q[e] = quotient(x.at(e), b);
        store8(Q + row * ldq + c0, pack4(q[0], q[1], q[2], q[3], b.bad), pack4(q[4], q[5], q[6], q[7], b.bad), valid,
               wide);
        if ((threadIdx.x & 15) == 0 && kb * kScaleBlock < cols) S[kb * lds + row] = b.s;
    }
}

// Blocks of 128 x 128 of X: one workgroup of 256 threads each, 16 lanes per
// row and 16 rows per pass, the whole block in registers.
template <typename T>
__global__ __launch_bounds__(256) void quantize_square(int64_t rows, int64_t cols, const T* X, int64_t ldx,
                                                       uint8_t* Q, int64_t ldq, float* S, int64_t lds, int64_t nb,
                                                       bool wide) {
    __shared__ uint32_t part[4];
    const int64_t kb = (int64_t)blockIdx.x % nb, rb = (int64_t)blockIdx.x / nb;
    const int t = threadIdx.x;
    const int64_t c0 = kb * 128 + (t & 15) * 8, r0 = rb * 128 + (t >> 4);
    const int64_t left = cols - c0;
    const int valid = left >= 8 ? 8 : (left > 0 ? (int)left : 0);
    Raw8<T> x[8];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t row = r0 + 16 * i;
        const int v = row < rows ? valid : 0;
        x[i] = load8(v > 0 ? X + row * ldx + c0 : X, v, wide);
        m = umax(m, top8(x[i]));
    }
    m = top_of_16(m);
    m = umax(m, (uint32_t)__shfl_xor((int)m, 16, 64));
    m = umax(m, (uint32_t)__shfl_xor((int)m, 32, 64));
    if ((t & 63) == 0) part[t >> 6] = m;
    __syncthreads();
    const Block b = block_of(umax(umax(part[0], part[1]), umax(part[2], part[3])));
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t row = r0 + 16 * i;
        if (row >= rows) continue;
        float q[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) q[e] = quotient(x[i].at(e), b);
        store8(Q + row * ldq + c0, pack4(q[0], q[1], q[2], q[3], b.bad), pack4(q[4], q[5], q[6], q[7], b.bad), valid,
               wide);
    }
    if (t == 0) S[kb * lds + rb] = b.s;
}

// Q = X^T: blocks of 128 run down the columns of X. One workgroup takes 128
// rows by 8 CW columns (CW threads across, 32 down, 4 consecutive rows each):
// every thread packs its 4 rows of a column into a dword, and the tile goes
// through LDS ([column][128 bytes], 16-byte chunk c of column j at chunk
// c ^ (j / 8 mod 8)) so that Q too is written in runs of 128 bytes. The 16 chunks
// that a wave's dword writes touch fall on 8 places, two lanes to a bank (27% of
// the LDS cycles at 8191 x 4096, which runs at 83% of a copy's rate). SQUARE: one scale for the
// whole 128 x 128 block (CW = 16).
template <typename T, int CW, bool SQUARE>
__global__ __launch_bounds__(CW * 32) void quantize_cols(int64_t rows, int64_t cols, const T* X, int64_t ldx,
                                                         uint8_t* Q, int64_t ldq, float* S, int64_t lds,
                                                         int64_t col_tiles, bool wide_x, bool wide_q) {
    constexpr int kCols = 8 * CW, kWaves = CW / 2;
    static_assert(!SQUARE || kCols == 128, "square blocks");
    __shared__ uint32_t tops[kWaves][kCols];
    __shared__ __attribute__((aligned(16))) uint8_t tile[kCols * 128];
    const int64_t rb = (int64_t)blockIdx.x / col_tiles, cb = (int64_t)blockIdx.x % col_tiles;
    const int t = threadIdx.x, a = t % CW, quad = t / CW;        // columns 8 a .., rows 4 quad ..
    const int64_t c0 = cb * kCols + 8 * a, r0 = rb * 128 + 4 * quad;
    const int64_t left = cols - c0;
    const int valid = left >= 8 ? 8 : (left > 0 ? (int)left : 0);
    Raw8<T> x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int v = r0 + i < rows ? valid : 0;
        x[i] = load8(v > 0 ? X + (r0 + i) * ldx + c0 : X, v, wide_x);
    }
    uint32_t m[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        m[e] = umax(umax(mag(x[0].at(e)), mag(x[1].at(e))), umax(mag(x[2].at(e)), mag(x[3].at(e))));
#pragma unroll
        for (int d = CW; d < 64; d <<= 1) m[e] = umax(m[e], (uint32_t)__shfl_xor((int)m[e], d, 64));
    }
    if ((t & 63) < CW) {
#pragma unroll
        for (int e = 0; e < 8; ++e) tops[t >> 6][8 * a + e] = m[e];
    }
    __syncthreads();
    Block b[8];
    if constexpr (SQUARE) {
        uint32_t all = 0;
        for (int i = t & 63; i < kWaves * kCols; i += 64) all = umax(all, tops[i / kCols][i % kCols]);
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) all = umax(all, (uint32_t)__shfl_xor((int)all, d, 64));
        const Block one = block_of(all);
#pragma unroll
        for (int e = 0; e < 8; ++e) b[e] = one;
        if (t == 0) S[rb * lds + cb] = one.s;
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            uint32_t all = 0;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) all = umax(all, tops[w][8 * a + e]);
            b[e] = block_of(all);
            if (quad == 0 && e < valid) S[rb * lds + c0 + e] = b[e].s;
        }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const uint32_t w = pack4(quotient(x[0].at(e), b[e]), quotient(x[1].at(e), b[e]), quotient(x[2].at(e), b[e]),
                                 quotient(x[3].at(e), b[e]), b[e].bad);
        const int chunk = (quad >> 2) ^ (a & 7);
        *reinterpret_cast<uint32_t*>(tile + (8 * a + e) * 128 + chunk * 16 + (quad & 3) * 4) = w;
    }
    __syncthreads();
    // 4 threads per column, 32 bytes each.
    const int j = t >> 2;
    const int64_t col = cb * kCols + j;
    if (col >= cols) return;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int c = 2 * (t & 3) + h;
        const u32x4 v = *reinterpret_cast<const u32x4*>(tile + j * 128 + ((c ^ ((j >> 3) & 7)) << 4));
        const int64_t k = rb * 128 + c * 16;
        uint8_t* dst = Q + col * ldq + k;
        if (wide_q && k + 16 <= rows) {
            *reinterpret_cast<u32x4*>(dst) = v;
        } else {
#pragma unroll
            for (int e = 0; e < 16; ++e)
                if (k + e < rows) dst[e] = (uint8_t)(v[e >> 2] >> (8 * (e & 3)));
        }
    }
}

template <typename T>
hipError_t launch(const QuantArgs<T>& a, hipStream_t s) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.X), q = reinterpret_cast<uintptr_t>(a.Q);
    const bool wide_x = x % 16 == 0 && (a.ldx * (int64_t)sizeof(T)) % 16 == 0;
    const bool wide = wide_x && q % 8 == 0 && a.ldq % 8 == 0;
    const bool wide_q = q % 16 == 0 && a.ldq % 16 == 0;
    const int64_t rb = (a.rows + 127) / 128, cb = (a.cols + 127) / 128;
    if (!a.transpose && a.block_rows == 1) {
        const dim3 grid((unsigned)((cb + 15) / 16), (unsigned)(a.rows < 65535 ? a.rows : 65535));
        return launch_kernel(&quantize_rows<T>, grid, dim3(256), s, a.rows, a.cols, a.X, a.ldx, a.Q, a.ldq, a.S, a.lds,
                             wide);
    }
    const int64_t tiles = a.transpose && a.block_rows == 1 ? (a.cols + 63) / 64 : cb;
    if (rb * tiles > kMaxGrid) return hipErrorInvalidConfiguration;
    const dim3 grid((unsigned)(rb * tiles));
    if (!a.transpose)
        return launch_kernel(&quantize_square<T>, grid, dim3(256), s, a.rows, a.cols, a.X, a.ldx, a.Q, a.ldq, a.S,
                             a.lds, tiles, wide);
    if (a.block_rows == 1)
        return launch_kernel(&quantize_cols<T, 8, false>, grid, dim3(256), s, a.rows, a.cols, a.X, a.ldx, a.Q, a.ldq,
                             a.S, a.lds, tiles, wide_x, wide_q);
    return launch_kernel(&quantize_cols<T, 16, true>, grid, dim3(512), s, a.rows, a.cols, a.X, a.ldx, a.Q, a.ldq, a.S,
                         a.lds, tiles, wide_x, wide_q);
}

}  // namespace

hipError_t launch_quantize(const QuantArgs<uint16_t>& a, hipStream_t s) { return launch<uint16_t>(a, s); }
hipError_t launch_quantize(const QuantArgs<float>& a, hipStream_t s) { return launch<float>(a, s); }

}  // namespace dg
