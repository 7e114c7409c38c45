// f8_product.hip -- D = A B^T of matrices in 8-bit floating point with a power of
// two for each block of 128 (f8.h) on gfx950's matrix cores.
//
// Into bf16: v_mfma_scale_f32_16x16x128_f8f6f4 multiplies 16 x 128 codes by 16 x 128
// and takes a scale for each operand's row, so one instruction is one block of
// 128, scales included.  It adds groups of eight products after aligning them to the
// group's largest, and what lies below 2^-13 of that is dropped (found by adding
// powers of two; beyond the groups sums keep fp32's 24 bits): 1e-5 to 6e-5 of the
// result on random operands, a hundredth of bf16's own rounding.
// Into fp32 that would be the largest error there is, so codes are widened to bf16
// with their scales (each exactly) and multiplied as bf16, which adds to
// 24 bits (7e-8), at half the rate.
//
// The operands are swapped (B's rows first), so that a lane holds four neighbouring
// columns of D: acc[x][y][r] = D[16 x + (lane & 15)][16 y + 4 (lane >> 4) + r].
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "f8.h"
#include "internal.h"

namespace z1 {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kTileRows = 128;
constexpr int kLine = kF8Block;    // bytes of a row of a stage in LDS

// What the 16-byte slots of row r are XORed with: sixteen lanes read one slot of 16
// neighbouring rows, 128 bytes apart (64 banks: two rows), and the key takes each
// value twice over them.
__device__ __forceinline__ int slot_key(int r) { return (r >> 1) & 7; }

// Rows [r0, r0 + 128) of a block of 128 columns into LDS; rows past the end: zeros.
__device__ __forceinline__ void stage(const F8& m, int64_t r0, int64_t kb, uint8_t* lds)
{
#pragma unroll
    for (int h = 0; h < 4; ++h) {
        const int at = threadIdx.x + h * kThreads, r = at >> 3, slot = at & 7;
        u32x4 v = {0, 0, 0, 0};
        if (r0 + r < m.rows) v = *reinterpret_cast<const u32x4*>(m.codes + (r0 + r) * m.ld + kb * kF8Block + 16 * slot);
        *reinterpret_cast<u32x4*>(lds + r * kLine + 16 * (slot ^ slot_key(r))) = v;
    }
}

// 16 rows of a stage: lane l gets 32 bytes of row l & 15 (which of its 128 bytes is
// the same for both operands, so the sum is over the whole block either way).
__device__ __forceinline__ i32x8 fragment(const uint8_t* lds, int r0)
{
    const int lane = threadIdx.x & 63, r = r0 + (lane & 15), h = lane >> 4;
    union { u32x4 v[2]; i32x8 f; } u;
    u.v[0] = *reinterpret_cast<const u32x4*>(lds + r * kLine + 16 * (h ^ slot_key(r)));
    u.v[1] = *reinterpret_cast<const u32x4*>(lds + r * kLine + 16 * ((4 + h) ^ slot_key(r)));
    return u.f;
}

// The scale of row r of a block (of the last row for rows past the end).
__device__ __forceinline__ int scale_of(const F8& m, int64_t r, int64_t kb)
{
    r = r < m.rows ? r : m.rows - 1;
    return m.scales[(r >> m.shift) * m.ld_scales + kb];
}

// Eight codes (two registers) times their scale in bf16, which holds each exactly.
template <int E5M2>
__device__ __forceinline__ bf16x8 widen8(uint32_t lo, uint32_t hi, float scale)
{
    union { bf16x2 p[4]; bf16x8 v; } u;
    if constexpr (E5M2) {
        u.p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(lo, scale, false);
        u.p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(lo, scale, true);
        u.p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(hi, scale, false);
        u.p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(hi, scale, true);
    } else {
        u.p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, false);
        u.p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, true);
        u.p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, false);
        u.p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, true);
    }
    return u.v;
}

// 2^(b-127); NaN for 255.
__device__ __forceinline__ float power(int b)
{
    return __uint_as_float(b == 255 ? 0x7fc00000u : b == 0 ? 0x00400000u : (uint32_t)b << 23);
}

template <typename T>
__device__ __forceinline__ T narrow(float x);
template <>
__device__ __forceinline__ float narrow<float>(float x) { return x; }
template <>
__device__ __forceinline__ __bf16 narrow<__bf16>(float x) { return (__bf16)x; }

template <int FA, int FB, typename D>
__global__ __launch_bounds__(kThreads) void product_kernel(F8Product p)
{
    __shared__ __attribute__((aligned(16))) uint8_t sa[kTileRows * kLine], sb[kTileRows * kLine];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t tiles_n = (p.b.rows + kTileRows - 1) / kTileRows;
    const int64_t m0 = blockIdx.x / tiles_n * kTileRows, n0 = blockIdx.x % tiles_n * kTileRows;
    const int wm = 64 * (wave >> 1), wn = 64 * (wave & 1);
    f32x4 acc[4][4];
#pragma unroll
    for (int x = 0; x < 4; ++x)
#pragma unroll
        for (int y = 0; y < 4; ++y) acc[x][y] = f32x4{0, 0, 0, 0};
    const int64_t blocks = (p.a.cols + kF8Block - 1) / kF8Block;
    for (int64_t kb = 0; kb < blocks; ++kb) {
        __syncthreads();
        stage(p.a, m0, kb, sa);
        stage(p.b, n0, kb, sb);
        __syncthreads();
        i32x8 fa[4], fb[4];
        int ea[4], eb[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            fa[x] = fragment(sa, wm + 16 * x);
            ea[x] = scale_of(p.a, m0 + wm + 16 * x + (lane & 15), kb);
            fb[x] = fragment(sb, wn + 16 * x);
            eb[x] = scale_of(p.b, n0 + wn + 16 * x + (lane & 15), kb);
        }
        if constexpr (sizeof(D) == 2) {
#pragma unroll
            for (int x = 0; x < 4; ++x)
#pragma unroll
                for (int y = 0; y < 4; ++y)
                    acc[x][y] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fb[y], fa[x], acc[x][y], FB, FA, 0, eb[y], 0, ea[x]);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                bf16x8 wa[4], wb[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    wa[x] = widen8<FA>((uint32_t)fa[x][2 * j], (uint32_t)fa[x][2 * j + 1], power(ea[x]));
                    wb[x] = widen8<FB>((uint32_t)fb[x][2 * j], (uint32_t)fb[x][2 * j + 1], power(eb[x]));
                }
#pragma unroll
                for (int x = 0; x < 4; ++x)
#pragma unroll
                    for (int y = 0; y < 4; ++y)
                        acc[x][y] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wb[y], wa[x], acc[x][y], 0, 0, 0);
            }
        }
    }
#pragma unroll
    for (int x = 0; x < 4; ++x) {
        const int64_t m = m0 + wm + 16 * x + (lane & 15);
        if (m >= p.a.rows) continue;
        D* row = static_cast<D*>(p.d) + m * p.ldd;
#pragma unroll
        for (int y = 0; y < 4; ++y)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int64_t n = n0 + wn + 16 * y + 4 * (lane >> 4) + r;
                if (n < p.b.rows) row[n] = narrow<D>(acc[x][y][r]);
            }
    }
}

template <int FA, int FB>
void launch(const F8Product& p, hipStream_t s)
{
    const int64_t grid = (p.a.rows + kTileRows - 1) / kTileRows * ((p.b.rows + kTileRows - 1) / kTileRows);
    if (p.f32) product_kernel<FA, FB, float><<<dim3((uint32_t)grid), kThreads, 0, s>>>(p);
    else product_kernel<FA, FB, __bf16><<<dim3((uint32_t)grid), kThreads, 0, s>>>(p);
}

}  // namespace

hipError_t launch_f8_product(const F8Product& p, hipStream_t s)
{
    if (p.a.e5m2) { if (p.b.e5m2) launch<1, 1>(p, s); else launch<1, 0>(p, s); }
    else          { if (p.b.e5m2) launch<0, 1>(p, s); else launch<0, 0>(p, s); }
    return hipGetLastError();
}

}  // namespace z1
