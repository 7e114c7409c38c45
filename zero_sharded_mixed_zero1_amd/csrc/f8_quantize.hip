// f8_quantize.hip -- matrices into 8-bit floating point with a power of two for
// each block of 128 (f8.h), along their rows, across them (the transpose), or both
// from one read.
//
// A workgroup takes a 128 x 128 tile: whatever the blocks' shape, each lies in one
// tile whole.  A lane holds 8 x 8 of it: rows 8 g + i, columns 8 c + j of lane
// 16 g + c, so that its codes are 8 bytes of a row of either output.  The
// transpose goes through LDS to leave as whole rows.
//
// HBM-bound: 2 or 4 bytes an element in, one out for each output.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "f8.h"
#include "internal.h"

#pragma clang fp contract(off)

namespace z1 {
namespace {

constexpr uint32_t kInf = 0x7f800000u;
constexpr int kPitch = kF8Block + 16;     // bytes of a row of the transposed codes in LDS

typedef uint16_t u16x8 __attribute__((ext_vector_type(8), aligned(2)));
typedef float f32x4 __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ uint32_t wide(uint16_t h) { return (uint32_t)h << 16; }
__device__ __forceinline__ uint32_t wide(float x) { return __float_as_uint(x); }

// Eight neighbouring values as binary32 bits.
__device__ __forceinline__ void load8(const uint16_t* p, uint32_t (&x)[8])
{
    const u16x8 v = *reinterpret_cast<const u16x8*>(p);
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = wide((uint16_t)v[j]);
}

__device__ __forceinline__ void load8(const float* p, uint32_t (&x)[8])
{
    const f32x4 a = *reinterpret_cast<const f32x4*>(p), b = *reinterpret_cast<const f32x4*>(p + 4);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        x[j] = __float_as_uint(a[j]);
        x[4 + j] = __float_as_uint(b[j]);
    }
}

// Largest over the 16 lanes of a row of the wave, in each of them.
__device__ __forceinline__ uint32_t row_max(uint32_t x)
{
    x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x128, 0xf, 0xf, false));   // row_ror:8
    x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x124, 0xf, 0xf, false));
    x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x122, 0xf, 0xf, false));
    x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x121, 0xf, 0xf, false));
    return x;
}

// The exponent byte that brings a block's largest magnitude to at most the
// format's largest value (1.75 * 2^8 or 1.75 * 2^15), and over half of that.
__device__ __forceinline__ uint32_t exponent(uint32_t top, int e5m2)
{
    const int b = (int)(top >> 23) - (e5m2 ? 15 : 8) + ((top & 0x7fffffu) > 0x600000u ? 1 : 0);
    return (uint32_t)(b > 1 ? b : 1);
}

__device__ __forceinline__ float inverse(uint32_t b) { return __uint_as_float((254u - b) << 23); }

// Four codes, to the nearest, ties to even.  What is infinite is NaN in e4m3, which
// has no infinity.
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d, int e5m2)
{
    if (e5m2) {
        const int lo = __builtin_amdgcn_cvt_pk_bf8_f32(a, b, 0, false);
        return (uint32_t)__builtin_amdgcn_cvt_pk_bf8_f32(c, d, lo, true);
    }
    const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, lo, true);
}

template <typename T>
__global__ __launch_bounds__(kThreads) void quantize_kernel(const T* __restrict__ src, int64_t rows, int64_t cols,
                                                            int64_t ld, F8 q, F8 qt, uint32_t col_blocks)
{
    __shared__ uint32_t tops[16][kF8Block];                       // a group of 8 rows' largest of each column
    __shared__ uint32_t tile_top[kThreads / 64];
    __shared__ __attribute__((aligned(16))) uint8_t turned[kF8Block * kPitch];
    const uint32_t rb = blockIdx.x / col_blocks, cb = blockIdx.x % col_blocks;
    const int c = threadIdx.x & 15, g = threadIdx.x >> 4;
    const int64_t r0 = (int64_t)rb * kF8Block + 8 * g, c0 = (int64_t)cb * kF8Block + 8 * c;
    uint32_t x[8][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const T* p = src + (r0 + i) * ld + c0;
        if (r0 + i < rows && c0 + 8 <= cols) {
            load8(p, x[i]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) x[i][j] = r0 + i < rows && c0 + j < cols ? wide(p[j]) : 0u;
        }
    }
    uint32_t row[8], col[8];
    auto tops_of = [&](auto magnitude) {
#pragma unroll
        for (int i = 0; i < 8; ++i) row[i] = col[i] = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t a = magnitude(x[i][j]);
                row[i] = max(row[i], a);
                col[j] = max(col[j], a);
            }
#pragma unroll
        for (int i = 0; i < 8; ++i) row[i] = row_max(row[i]);
    };
    tops_of([](uint32_t u) { return u & 0x7fffffffu; });
    uint32_t all = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) all = max(all, row[i]);
    if (__any(all >= kInf)) {   // what is not finite does not set the scale
        tops_of([](uint32_t u) { return (u & 0x7fffffffu) >= kInf ? 0u : u & 0x7fffffffu; });
        all = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) all = max(all, row[i]);
    }
    all = max(all, (uint32_t)__shfl_xor((int)all, 16, 64));
    all = max(all, (uint32_t)__shfl_xor((int)all, 32, 64));
    if ((threadIdx.x & 63) == 0) tile_top[threadIdx.x >> 6] = all;
    if (qt.codes) {
#pragma unroll
        for (int j = 0; j < 8; ++j) tops[g][8 * c + j] = col[j];
    }
    __syncthreads();
    all = max(max(tile_top[0], tile_top[1]), max(tile_top[2], tile_top[3]));
    if (q.codes) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (r0 + i >= rows) continue;
            const uint32_t b = exponent(q.shift ? all : row[i], q.e5m2);
            const float inv = inverse(b);
            float y[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = __uint_as_float(x[i][j]) * inv;
            *reinterpret_cast<u32x2*>(q.codes + (r0 + i) * q.ld + c0) =
                u32x2{codes4(y[0], y[1], y[2], y[3], q.e5m2), codes4(y[4], y[5], y[6], y[7], q.e5m2)};
            if (c == 0 && !q.shift) q.scales[(r0 + i) * q.ld_scales + cb] = (uint8_t)b;
        }
        if (q.shift && threadIdx.x == 0) q.scales[(int64_t)rb * q.ld_scales + cb] = (uint8_t)exponent(all, q.e5m2);
    }
    if (qt.codes) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            uint32_t top = all;
            if (!qt.shift) {
                top = 0;
                for (int k = 0; k < 16; ++k) top = max(top, tops[k][8 * c + j]);
            }
            const uint32_t b = exponent(top, qt.e5m2);
            const float inv = inverse(b);
            float y[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = __uint_as_float(x[i][j]) * inv;
            *reinterpret_cast<u32x2*>(turned + (8 * c + j) * kPitch + 8 * g) =
                u32x2{codes4(y[0], y[1], y[2], y[3], qt.e5m2), codes4(y[4], y[5], y[6], y[7], qt.e5m2)};
            if (!qt.shift && g == 0 && c0 + j < cols) qt.scales[(c0 + j) * qt.ld_scales + rb] = (uint8_t)b;
        }
        if (qt.shift && threadIdx.x == 0) qt.scales[(int64_t)cb * qt.ld_scales + rb] = (uint8_t)exponent(all, qt.e5m2);
        __syncthreads();
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            const int at = threadIdx.x + h * kThreads, line = at >> 3, seg = (at & 7) * 16;
            const int64_t out = (int64_t)cb * kF8Block + line;
            if (out < cols)
                *reinterpret_cast<u32x4*>(qt.codes + out * qt.ld + (int64_t)rb * kF8Block + seg) =
                    *reinterpret_cast<const u32x4*>(turned + line * kPitch + seg);
        }
    }
}

}  // namespace

hipError_t launch_f8_quantize(const void* src, bool f32, int64_t rows, int64_t cols, int64_t ld, const F8& q,
                              const F8& qt, hipStream_t s)
{
    const int64_t rb = (rows + kF8Block - 1) / kF8Block, cb = (cols + kF8Block - 1) / kF8Block;
    const dim3 grid((uint32_t)(rb * cb));
    if (f32) quantize_kernel<float><<<grid, kThreads, 0, s>>>(static_cast<const float*>(src), rows, cols, ld, q, qt, (uint32_t)cb);
    else quantize_kernel<uint16_t><<<grid, kThreads, 0, s>>>(static_cast<const uint16_t*>(src), rows, cols, ld, q, qt, (uint32_t)cb);
    return hipGetLastError();
}

}  // namespace z1
