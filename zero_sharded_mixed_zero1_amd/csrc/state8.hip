// state8.hip -- moments in 8 bits (state8.h) from and to fp32 or bf16: what a
// program that resumes from, or writes, a checkpoint of wider moments calls.
//
// encode: per block of 256, the exponent byte from the largest magnitude and the
// codes to the nearest, ties to even (counts start at zero); of v the codes hold
// the root.  decode: the product of code and scale, which fp32 holds exactly;
// squared for v.
//
// HBM-bound: 5 bytes an element.  A wave takes a block, lane l its elements 4 l to
// 4 l + 3 where x allows vector access, and l, l + 64, ... where it does not and in
// a short last block.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "internal.h"
#include "state8.h"

#pragma clang fp contract(off)

namespace z1 {
namespace {

using namespace dev8;

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint16_t u16x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ float widen(float x) { return x; }
__device__ __forceinline__ float widen(uint16_t h) { return __uint_as_float((uint32_t)h << 16); }

__device__ __forceinline__ void narrow(float x, float& o) { o = x; }
__device__ __forceinline__ void narrow(float x, uint16_t& o)   // to the nearest bf16, ties to even; NaN stays NaN
{
    const uint32_t u = __float_as_uint(x);
    o = (uint16_t)(abs_bits(x) > kInfBits ? (u >> 16) | 0x40u : (u + 0x7fffu + ((u >> 16) & 1u)) >> 16);
}

// Code to the nearest, ties to even.
__device__ __forceinline__ uint32_t code_near(float y) { return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(y, y, 0, false) & 0xffu; }

template <typename T, bool VEC, bool V>
__global__ __launch_bounds__(kThreads) void encode_kernel(const T* __restrict__ x, int64_t n, uint8_t* __restrict__ codes,
                                                          uint32_t* __restrict__ words)
{
    typedef T T4 __attribute__((ext_vector_type(4)));
    const int lane = threadIdx.x & 63;
    const int64_t blocks = state8_blocks(n), step = (int64_t)gridDim.x * (kThreads / 64);
    for (int64_t k = (int64_t)blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6); k < blocks; k += step) {
        const int64_t at = k * kBlock8;
        const bool whole = VEC && at + kBlock8 <= n;
        float y[4];
        if (whole) {
            const T4 q = *reinterpret_cast<const T4*>(x + at + 4 * lane);
#pragma unroll
            for (int i = 0; i < 4; ++i) y[i] = widen(q[i]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t e = at + lane + 64 * i;
                y[i] = e < n ? widen(x[e]) : 0.0f;
            }
        }
        if constexpr (V) {
#pragma unroll
            for (int i = 0; i < 4; ++i) y[i] = sqrtf(y[i]);
        }
        const Top8 t = top8<V>(y);
        const float inv = inverse8(t.b);
        uint32_t c[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            c[i] = code_near(y[i] * inv);
            if constexpr (V) c[i] = max(c[i] & 0x7fu, y[i] > 0.0f ? 1u : 0u);   // (the root of -0 is -0)
            if (t.special) c[i] = held8<V>(y[i], c[i], t);
        }
        if (whole) {
            *reinterpret_cast<uint32_t*>(codes + at + 4 * lane) = c[0] | c[1] << 8 | c[2] << 16 | c[3] << 24;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t e = at + lane + 64 * i;
                if (e < n) codes[e] = (uint8_t)c[i];
            }
        }
        if (lane == 0) words[k] = t.b;
    }
}

template <typename T, bool VEC, bool V>
__global__ __launch_bounds__(kThreads) void decode_kernel(const uint8_t* __restrict__ codes,
                                                          const uint32_t* __restrict__ words, int64_t n,
                                                          T* __restrict__ x)
{
    typedef T T4 __attribute__((ext_vector_type(4)));
    const int lane = threadIdx.x & 63;
    const int64_t blocks = state8_blocks(n), step = (int64_t)gridDim.x * (kThreads / 64);
    for (int64_t k = (int64_t)blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6); k < blocks; k += step) {
        const int64_t at = k * kBlock8;
        const float scale = scale8(words[k]);
        if (VEC && at + kBlock8 <= n) {
            float y[4];
            decode4(*reinterpret_cast<const uint32_t*>(codes + at + 4 * lane), scale, y);
            T4 q;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                T o;
                narrow(V ? y[i] * y[i] : y[i], o);
                q[i] = o;
            }
            *reinterpret_cast<T4*>(x + at + 4 * lane) = q;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t e = at + lane + 64 * i;
                if (e < n) {
                    const float y = __builtin_amdgcn_cvt_f32_fp8(codes[e], 0) * scale;
                    narrow(V ? y * y : y, x[e]);
                }
            }
        }
    }
}

}  // namespace

hipError_t launch_state8_encode(const void* x, int64_t n, bool bf16, bool v, void* state, int nblocks, hipStream_t s)
{
    uint8_t* codes = static_cast<uint8_t*>(state);
    uint32_t* words = reinterpret_cast<uint32_t*>(codes + state8_words_at(n));
    const bool vec = reinterpret_cast<uintptr_t>(x) % (bf16 ? 8 : 16) == 0;
#define Z1_ENC(T, VEC, V) encode_kernel<T, VEC, V><<<nblocks, kThreads, 0, s>>>(static_cast<const T*>(x), n, codes, words)
#define Z1_ENC_T(T)                                                                   \
    do {                                                                              \
        if (vec) { if (v) Z1_ENC(T, true, true); else Z1_ENC(T, true, false); }       \
        else     { if (v) Z1_ENC(T, false, true); else Z1_ENC(T, false, false); }     \
    } while (0)
    if (bf16) Z1_ENC_T(uint16_t);
    else Z1_ENC_T(float);
#undef Z1_ENC_T
#undef Z1_ENC
    return hipGetLastError();
}

hipError_t launch_state8_decode(const void* state, int64_t n, bool bf16, bool v, void* x, int nblocks, hipStream_t s)
{
    const uint8_t* codes = static_cast<const uint8_t*>(state);
    const uint32_t* words = reinterpret_cast<const uint32_t*>(codes + state8_words_at(n));
    const bool vec = reinterpret_cast<uintptr_t>(x) % (bf16 ? 8 : 16) == 0;
#define Z1_DEC(T, VEC, V) decode_kernel<T, VEC, V><<<nblocks, kThreads, 0, s>>>(codes, words, n, static_cast<T*>(x))
#define Z1_DEC_T(T)                                                                   \
    do {                                                                              \
        if (vec) { if (v) Z1_DEC(T, true, true); else Z1_DEC(T, true, false); }       \
        else     { if (v) Z1_DEC(T, false, true); else Z1_DEC(T, false, false); }     \
    } while (0)
    if (bf16) Z1_DEC_T(uint16_t);
    else Z1_DEC_T(float);
#undef Z1_DEC_T
#undef Z1_DEC
    return hipGetLastError();
}

}  // namespace z1
