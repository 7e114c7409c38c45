// state8.hip -- moments in 8 bits (state8.h) from and to fp32 or bf16: what a
// program that resumes from, or writes, a checkpoint of wider moments calls.
//
// encode: per block of 256, the exponent byte from the largest magnitude and the
// codes to the nearest, ties to even (counts start at zero); of v the codes hold
// the root.  decode: the product of code and scale, which fp32 holds exactly;
// squared for v.
//
// HBM-bound: 5 bytes an element (fp32); 45 M elements decoded 32 us (7.0 TB/s, the MALL
// takes what is written), 100 003 encoded 3.1 us of latency.  A workgroup takes a tile of 2048, a wave two
// blocks of it, a lane a quad of each: whole quads at any alignment of x (gfx950's
// vector accesses need no more than the elements'), the one that the end cuts
// element by element.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "internal.h"
#include "state8.h"

#pragma clang fp contract(off)

namespace z1 {
namespace {

using namespace dev8;

template <typename T>
struct Quad {
    typedef T Plain __attribute__((ext_vector_type(4)));
    typedef Plain Any __attribute__((aligned(sizeof(T))));
};

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

// Where the lane's quad h of tile blockIdx.x begins, and how many of its elements
// there are.
__device__ __forceinline__ int64_t quad_at(int h)
{
    return (int64_t)blockIdx.x * kTile + 512 * (int)(threadIdx.x >> 6) + 256 * h + 4 * (int)(threadIdx.x & 63);
}

__device__ __forceinline__ int present(int64_t at, int64_t n) { return n - at > 4 ? 4 : (int)(n - at); }

template <typename T, bool V>
__global__ __launch_bounds__(kThreads) void encode_kernel(const T* __restrict__ x, int64_t n, uint8_t* __restrict__ codes,
                                                          uint32_t* __restrict__ words)
{
    float y[2][4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int64_t at = quad_at(h);
        const int c = present(at, n);
        typename Quad<T>::Plain q = {0, 0, 0, 0};
        if (c == 4) {
            q = *reinterpret_cast<const typename Quad<T>::Any*>(x + at);
        } else {
#pragma unroll
            for (int j = 0; j < 3; ++j)
                if (j < c) q[j] = x[at + j];
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) y[h][j] = widen((T)q[j]);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if constexpr (V) {
#pragma unroll
            for (int j = 0; j < 4; ++j) y[h][j] = sqrtf(y[h][j]);
        }
        const Top8 t = top8<V>(y[h]);
        const float inv = inverse8(t.b);
        uint32_t word = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint32_t c = code_near(y[h][j] * inv);
            if constexpr (V) c = max(c & 0x7fu, y[h][j] > 0.0f ? 1u : 0u);   // (the root of -0 is -0)
            if (t.special) c = held8<V>(y[h][j], c, t);
            word |= c << (8 * j);
        }
        const int64_t at = quad_at(h);
        const int c = present(at, n);
        if (c == 4) {
            *reinterpret_cast<uint32_t*>(codes + at) = word;
        } else {
#pragma unroll
            for (int j = 0; j < 3; ++j)
                if (j < c) codes[at + j] = (uint8_t)(word >> (8 * j));
        }
        if ((threadIdx.x & 63) == 0 && c > 0) words[at >> 8] = t.b;
    }
}

template <typename T, bool V>
__global__ __launch_bounds__(kThreads) void decode_kernel(const uint8_t* __restrict__ codes,
                                                          const uint32_t* __restrict__ words, int64_t n,
                                                          T* __restrict__ x)
{
    uint32_t w[2] = {0, 0}, b[2] = {0, 0};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int64_t at = quad_at(h);
        const int c = present(at, n);
        if (c > 0) b[h] = words[at >> 8];
        if (c == 4) {
            w[h] = *reinterpret_cast<const uint32_t*>(codes + at);
        } else {
#pragma unroll
            for (int j = 0; j < 3; ++j)
                if (j < c) w[h] |= (uint32_t)codes[at + j] << (8 * j);
        }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int64_t at = quad_at(h);
        const int c = present(at, n);
        float y[4];
        decode4(w[h], scale8(b[h]), y);
        typename Quad<T>::Plain q;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            T o;
            narrow(V ? y[j] * y[j] : y[j], o);
            q[j] = o;
        }
        if (c == 4) {
            __builtin_nontemporal_store((typename Quad<T>::Any)q, reinterpret_cast<typename Quad<T>::Any*>(x + at));
        } else {
#pragma unroll
            for (int j = 0; j < 3; ++j)
                if (j < c) x[at + j] = q[j];
        }
    }
}

}  // namespace

hipError_t launch_state8_encode(const void* x, int64_t n, bool bf16, bool v, void* state, hipStream_t s)
{
    uint8_t* codes = static_cast<uint8_t*>(state);
    uint32_t* words = reinterpret_cast<uint32_t*>(codes + state8_words_at(n));
    const dim3 grid((uint32_t)((n + kTile - 1) / kTile));
    if (bf16) {
        const uint16_t* h = static_cast<const uint16_t*>(x);
        if (v) encode_kernel<uint16_t, true><<<grid, kThreads, 0, s>>>(h, n, codes, words);
        else encode_kernel<uint16_t, false><<<grid, kThreads, 0, s>>>(h, n, codes, words);
    } else {
        const float* f = static_cast<const float*>(x);
        if (v) encode_kernel<float, true><<<grid, kThreads, 0, s>>>(f, n, codes, words);
        else encode_kernel<float, false><<<grid, kThreads, 0, s>>>(f, n, codes, words);
    }
    return hipGetLastError();
}

hipError_t launch_state8_decode(const void* state, int64_t n, bool bf16, bool v, void* x, hipStream_t s)
{
    const uint8_t* codes = static_cast<const uint8_t*>(state);
    const uint32_t* words = reinterpret_cast<const uint32_t*>(codes + state8_words_at(n));
    const dim3 grid((uint32_t)((n + kTile - 1) / kTile));
    if (bf16) {
        uint16_t* h = static_cast<uint16_t*>(x);
        if (v) decode_kernel<uint16_t, true><<<grid, kThreads, 0, s>>>(codes, words, n, h);
        else decode_kernel<uint16_t, false><<<grid, kThreads, 0, s>>>(codes, words, n, h);
    } else {
        float* f = static_cast<float*>(x);
        if (v) decode_kernel<float, true><<<grid, kThreads, 0, s>>>(codes, words, n, f);
        else decode_kernel<float, false><<<grid, kThreads, 0, s>>>(codes, words, n, f);
    }
    return hipGetLastError();
}

}  // namespace z1
