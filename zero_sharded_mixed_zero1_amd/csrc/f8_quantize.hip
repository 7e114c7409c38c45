// f8_quantize.hip -- matrices into 8-bit floating point with a power of two for
// each block of 128 (f8.h), along their rows, across them (the transpose), or both
// from one read.
//
// A workgroup takes a 128 x 128 tile: whatever the blocks' shape, each lies in one
// tile whole.  A lane holds 8 x 8 of it: rows 8 g + i, columns 8 c + j of lane
// 16 g + c, so that its codes are 8 bytes of a row of either output.  The
// transpose goes through LDS to leave as whole rows.  bf16 stays packed in pairs all
// the way (magnitudes are compared as 16-bit numbers, codes made from pairs).
//
// HBM-bound: 2 or 4 bytes an element in, one out for each output.  8192 x 4096 bf16 into
// both 32 us (4.2 TB/s; without the pairs, an element at a time, 48), 11008 x 4096 fp32
// with blocks of 128 x 128 into both 54.2 (5.0 TB/s).  A forward pass multiplies the codes
// next and the backward pass reads the transpose much later, so the transpose is stored
// non-temporally and the codes are not: into the transpose alone 19.2 us (23.8), and the
// weight's and the input's conversion with the product behind them, 2048 x 4096 x 4096,
// 57.9 (59.2).  Both so: 8192 x 4096 27.0 us alone, but the product then reads from
// memory (512 x 4096 x 4096 38.5 all together, 35.8 without either, 35.4 as it is).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "f8.h"
#include "internal.h"

#pragma clang fp contract(off)

namespace z1 {
namespace {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef u32x4 u32x4u __attribute__((aligned(2)));
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
typedef short s16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

template <typename A, typename B>
__device__ __forceinline__ A bits(B b)
{
    static_assert(sizeof(A) == sizeof(B), "size");
    return __builtin_bit_cast(A, b);
}

// Eight neighbouring values of a row, in kWords registers; their magnitudes' maxima
// as numbers that compare like them; and codes of pairs.
struct Half {   // bf16, in pairs
    static constexpr int kWords = 4;
    typedef uint16_t Elem;
    static constexpr uint32_t kMagnitude = 0x7fff7fffu;
    static __device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b)
    {
        return bits<uint32_t>(__builtin_elementwise_max(bits<u16x2>(a), bits<u16x2>(b)));
    }
    // of the two values of a pair, as binary32's magnitude
    static __device__ __forceinline__ uint32_t one(uint32_t a) { return max(a << 16, a & 0xffff0000u); }
    // magnitudes, zero for what is not finite
    static __device__ __forceinline__ uint32_t finite(uint32_t a)
    {
        if ((a & 0x7fffu) >= 0x7f80u) a &= 0xffff0000u;
        return a >= 0x7f800000u ? a & 0xffffu : a;
    }
    static __device__ __forceinline__ uint32_t column(const uint32_t* w, int j) { return j & 1 ? w[j >> 1] & 0xffff0000u : w[j >> 1] << 16; }
    static __device__ __forceinline__ uint32_t word(uint32_t lo, uint32_t hi) { return lo >> 16 | (hi & 0xffff0000u); }
};

struct Single {   // fp32
    static constexpr int kWords = 8;
    typedef float Elem;
    static constexpr uint32_t kMagnitude = 0x7fffffffu;
    static __device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) { return max(a, b); }
    static __device__ __forceinline__ uint32_t one(uint32_t a) { return a; }
    static __device__ __forceinline__ uint32_t finite(uint32_t a) { return a >= 0x7f800000u ? 0u : a; }
    static __device__ __forceinline__ uint32_t column(const uint32_t* w, int j) { return w[j]; }
};

constexpr uint32_t kInf = 0x7f800000u;

__device__ __forceinline__ uint32_t widened(uint16_t h) { return (uint32_t)h << 16; }
__device__ __forceinline__ uint32_t widened(float x) { return __float_as_uint(x); }

__device__ __forceinline__ void load_row(const uint16_t* p, uint32_t (&w)[4])
{
    const u32x4 v = *reinterpret_cast<const u32x4u*>(p);
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = v[k];
}

__device__ __forceinline__ void load_row(const float* p, uint32_t (&w)[8])
{
    const u32x4 a = *reinterpret_cast<const u32x4u*>(p), b = *reinterpret_cast<const u32x4u*>(p + 4);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        w[k] = a[k];
        w[4 + k] = b[k];
    }
}

// Two codes, to the nearest, ties to even, of values over their scale, into the low or
// high half of `old`.
template <bool HI>
__device__ __forceinline__ uint32_t codes_of_pair(uint32_t old, uint32_t pair, float scale, int e5m2)
{
    const bf16x2 v = bits<bf16x2>(pair);
    return bits<uint32_t>(e5m2 ? __builtin_amdgcn_cvt_scalef32_pk_bf8_bf16(bits<s16x2>(old), v, scale, HI)
                               : __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(bits<s16x2>(old), v, scale, HI));
}

template <bool HI>
__device__ __forceinline__ uint32_t codes_of_two(uint32_t old, uint32_t a, uint32_t b, float scale, int e5m2)
{
    const float x = __uint_as_float(a), y = __uint_as_float(b);
    return bits<uint32_t>(e5m2 ? __builtin_amdgcn_cvt_scalef32_pk_bf8_f32(bits<s16x2>(old), x, y, scale, HI)
                               : __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(bits<s16x2>(old), x, y, scale, HI));
}

// Codes of a row's eight values, and of the eight rows' values of column j.
__device__ __forceinline__ u32x2 codes_along(const uint32_t (&w)[4], float scale, int e5m2)
{
    return u32x2{codes_of_pair<true>(codes_of_pair<false>(0, w[0], scale, e5m2), w[1], scale, e5m2),
                 codes_of_pair<true>(codes_of_pair<false>(0, w[2], scale, e5m2), w[3], scale, e5m2)};
}

__device__ __forceinline__ u32x2 codes_along(const uint32_t (&w)[8], float scale, int e5m2)
{
    return u32x2{codes_of_two<true>(codes_of_two<false>(0, w[0], w[1], scale, e5m2), w[2], w[3], scale, e5m2),
                 codes_of_two<true>(codes_of_two<false>(0, w[4], w[5], scale, e5m2), w[6], w[7], scale, e5m2)};
}

__device__ __forceinline__ u32x2 codes_across(const uint32_t (&x)[8][4], int j, float scale, int e5m2)
{
    const uint32_t sel = j & 1 ? 0x07060302u : 0x05040100u;   // both words' high or low halves
    uint32_t p[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = __builtin_amdgcn_perm(x[2 * i + 1][j >> 1], x[2 * i][j >> 1], sel);
    return codes_along(p, scale, e5m2);
}

__device__ __forceinline__ u32x2 codes_across(const uint32_t (&x)[8][8], int j, float scale, int e5m2)
{
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = x[i][j];
    return codes_along(w, scale, e5m2);
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

// Largest over a wave's four rows of 16 lanes, in each of them.
template <typename F>
__device__ __forceinline__ uint32_t rows_max(uint32_t x)
{
    const auto a = __builtin_amdgcn_permlane32_swap(x, x, false, false);
    x = F::larger(a[0], a[1]);
    const auto b = __builtin_amdgcn_permlane16_swap(x, x, false, false);
    return F::larger(b[0], b[1]);
}

// The exponent byte that brings a block's largest magnitude to at most the
// format's largest value (1.75 * 2^8 or 1.75 * 2^15), and over half of that.
__device__ __forceinline__ uint32_t exponent(uint32_t top, int e5m2)
{
    const int b = (int)(top >> 23) - (e5m2 ? 15 : 8) + ((top & 0x7fffffu) > 0x600000u ? 1 : 0);
    return (uint32_t)(b > 1 ? b : 1);
}

__device__ __forceinline__ float power(uint32_t b) { return __uint_as_float(b << 23); }

template <typename F, bool Q, bool QT>
__global__ __launch_bounds__(kThreads) void quantize_kernel(const typename F::Elem* __restrict__ src, int64_t rows,
                                                            int64_t cols, int64_t ld, F8 q, F8 qt, uint32_t col_blocks)
{
    constexpr int W = F::kWords;
    __shared__ __attribute__((aligned(16))) uint32_t tops[QT ? kThreads / 64 : 1][16][W];   // a wave's largest of each column
    __shared__ uint32_t tile_top[kThreads / 64];
    __shared__ __attribute__((aligned(16))) uint8_t turned[QT ? kF8Block * kF8Block : 16];
    const uint32_t rb = blockIdx.x / col_blocks, cb = blockIdx.x % col_blocks;
    const int c = threadIdx.x & 15, g = threadIdx.x >> 4, wave = threadIdx.x >> 6;
    const int64_t r0 = (int64_t)rb * kF8Block + 8 * g, c0 = (int64_t)cb * kF8Block + 8 * c;
    uint32_t x[8][W];
    if (r0 + 8 <= rows && c0 + 8 <= cols) {
#pragma unroll
        for (int i = 0; i < 8; ++i) load_row(src + (r0 + i) * ld + c0, x[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            uint32_t v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = r0 + i < rows && c0 + j < cols ? widened(src[(r0 + i) * ld + c0 + j]) : 0u;
#pragma unroll
            for (int k = 0; k < W; ++k) {
                if constexpr (W == 4) x[i][k] = F::word(v[2 * k], v[2 * k + 1]);
                else x[i][k] = v[k];
            }
        }
    }
    uint32_t row[8], col[W];
    auto tops_of = [&](auto magnitude) {
#pragma unroll
        for (int k = 0; k < W; ++k) col[k] = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            uint32_t r = 0;
#pragma unroll
            for (int k = 0; k < W; ++k) {
                const uint32_t a = magnitude(x[i][k]);
                r = F::larger(r, a);
                if constexpr (QT) col[k] = F::larger(col[k], a);
            }
            row[i] = row_max(F::one(r));
        }
    };
    tops_of([](uint32_t w) { return w & F::kMagnitude; });
    uint32_t all = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) all = max(all, row[i]);
    if (__any(all >= kInf)) {   // what is not finite does not set the scale
        tops_of([](uint32_t w) { return F::finite(w & F::kMagnitude); });
        all = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) all = max(all, row[i]);
    }
    if (QT || q.shift) {
        all = rows_max<Single>(all);
        if ((threadIdx.x & 63) == 0) tile_top[wave] = all;
        if constexpr (QT) {
#pragma unroll
            for (int k = 0; k < W; ++k) col[k] = rows_max<F>(col[k]);
            if ((threadIdx.x & 48) == 0) {
#pragma unroll
                for (int k = 0; k < W; k += 4)
                    *reinterpret_cast<u32x4*>(&tops[wave][c][k]) = u32x4{col[k], col[k + 1], col[k + 2], col[k + 3]};
            }
        }
        __syncthreads();
        all = max(max(tile_top[0], tile_top[1]), max(tile_top[2], tile_top[3]));
    }
    if constexpr (Q) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (r0 + i >= rows) continue;
            const uint32_t b = exponent(q.shift ? all : row[i], q.e5m2);
            *reinterpret_cast<u32x2*>(q.codes + (r0 + i) * q.ld + c0) = codes_along(x[i], power(b), q.e5m2);
            if (c == 0 && !q.shift) q.scales[(r0 + i) * q.ld_scales + cb] = (uint8_t)b;
        }
        if (q.shift && threadIdx.x == 0) q.scales[(int64_t)rb * q.ld_scales + cb] = (uint8_t)exponent(all, q.e5m2);
    }
    if constexpr (QT) {
#pragma unroll
        for (int w = 0; w < kThreads / 64; ++w)
#pragma unroll
            for (int k = 0; k < W; k += 4) {
                const u32x4 v = *reinterpret_cast<const u32x4*>(&tops[w][c][k]);
#pragma unroll
                for (int e = 0; e < 4; ++e) col[k + e] = F::larger(w ? col[k + e] : 0u, v[e]);
            }
        // Column 8 c + j of the tile is line 8 c + j of `turned`, 16 slots of 8 bytes, one
        // a group of rows, XORed with c: lanes of one j write 16 lines a multiple of
        // 1 KiB apart, which would all begin in one bank.
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t b = exponent(qt.shift ? all : F::column(col, j), qt.e5m2);
            *reinterpret_cast<u32x2*>(turned + (8 * c + j) * kF8Block + 8 * (g ^ c)) = codes_across(x, j, power(b), qt.e5m2);
            if (!qt.shift && g == 0 && c0 + j < cols) qt.scales[(c0 + j) * qt.ld_scales + rb] = (uint8_t)b;
        }
        if (qt.shift && threadIdx.x == 0) qt.scales[(int64_t)cb * qt.ld_scales + rb] = (uint8_t)exponent(all, qt.e5m2);
        __syncthreads();
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            const int at = threadIdx.x + h * kThreads, line = at >> 3, seg = at & 7, key = line >> 3;
            const int64_t out = (int64_t)cb * kF8Block + line;
            u32x4 v = *reinterpret_cast<const u32x4*>(turned + line * kF8Block + 16 * (seg ^ (key >> 1)));
            if (key & 1) v = u32x4{v[2], v[3], v[0], v[1]};
            if (out < cols) __builtin_nontemporal_store(v, reinterpret_cast<u32x4*>(qt.codes + out * qt.ld + (int64_t)rb * kF8Block + 16 * seg));
        }
    }
}

template <typename F>
void launch(const void* src, int64_t rows, int64_t cols, int64_t ld, const F8& q, const F8& qt, hipStream_t s)
{
    const int64_t rb = (rows + kF8Block - 1) / kF8Block, cb = (cols + kF8Block - 1) / kF8Block;
    const dim3 grid((uint32_t)(rb * cb));
    const typename F::Elem* x = static_cast<const typename F::Elem*>(src);
    if (q.codes && qt.codes) quantize_kernel<F, true, true><<<grid, kThreads, 0, s>>>(x, rows, cols, ld, q, qt, (uint32_t)cb);
    else if (q.codes) quantize_kernel<F, true, false><<<grid, kThreads, 0, s>>>(x, rows, cols, ld, q, qt, (uint32_t)cb);
    else quantize_kernel<F, false, true><<<grid, kThreads, 0, s>>>(x, rows, cols, ld, q, qt, (uint32_t)cb);
}

}  // namespace

hipError_t launch_f8_quantize(const void* src, bool f32, int64_t rows, int64_t cols, int64_t ld, const F8& q,
                              const F8& qt, hipStream_t s)
{
    if (f32) launch<Single>(src, rows, cols, ld, q, qt, s);
    else launch<Half>(src, rows, cols, ld, q, qt, s);
    return hipGetLastError();
}

}  // namespace z1
