// state8.h -- moments in 8 bits: the layout shared by host and device, and the
// device code that reads and writes one block of 256 elements a wave.
//
// A moment of n elements is a buffer of state8_bytes(n) bytes: n codes, then, from
// the next multiple of 16 on, one 32-bit word for each block of 256 consecutive
// elements (the last may be short).  Bits 0-7 of a word are an exponent byte b,
// bits 8-31 count how often the block has been rounded.  A code is e4m3 (sign, four
// bits of exponent, three of mantissa) and stands for e4m3(code) * 2^(b-127): for m
// that is the value, for v its square root r (v = r * r).
//
// Why the root: a code spans 2^17 between its smallest step and the block's largest
// value, so v spans 2^34, and the update needs r anyway.  Why powers of two: scaling is
// exact, so a block whose values did not change keeps its codes.  Why 256: a
// wave's load of four codes a lane is one block, so its largest value is found
// without LDS.  The words cost 1/64 byte an element.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace z1 {

constexpr int kBlock8 = 256;      // elements of a block

inline __host__ __device__ size_t state8_words_at(int64_t n) { return ((size_t)n + 15) / 16 * 16; }
inline __host__ __device__ int64_t state8_blocks(int64_t n) { return (n + kBlock8 - 1) / kBlock8; }
inline __host__ __device__ size_t state8_size(int64_t n) { return n > 0 ? state8_words_at(n) + 4 * (size_t)state8_blocks(n) : 0; }

namespace dev8 {

// The block's largest value lies in [2^7, 2^8) of its scale, so that rounding up
// stays inside the format (448 ends it) and NaN's code is never reached.
constexpr int kTop8 = 7;
constexpr uint32_t kNan8 = 0x7f, kLast8 = 0x77, kInfBits = 0x7f800000u;
// The last binade of m, and of r (where r * r still is finite), and its exponent byte.
constexpr uint32_t kHugeBits[2] = {0x7f000000u, 0x5f000000u}, kLastB[2] = {247, 183};

// Largest of the wave's 64 values, in every lane (as a scalar).
__device__ __forceinline__ uint32_t wave_max(uint32_t x)
{
    auto step = [](uint32_t a, uint32_t b) { return a > b ? a : b; };
    x = step(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x111, 0xf, 0xf, false));   // row_shr:1
    x = step(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x112, 0xf, 0xf, false));   // row_shr:2
    x = step(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x114, 0xf, 0xf, false));   // row_shr:4
    x = step(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x118, 0xf, 0xf, false));   // row_shr:8
    x = step(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x142, 0xa, 0xf, false));   // row_bcast:15
    x = step(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x143, 0xc, 0xf, false));   // row_bcast:31
    return (uint32_t)__builtin_amdgcn_readlane((int)x, 63);
}

__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// 2^(b-127) of an exponent byte; 0 for b = 0 (a block that was never written).
__device__ __forceinline__ float scale8(uint32_t word) { return __uint_as_float((word & 255u) << 23); }

// Four codes, times the block's scale.
__device__ __forceinline__ void decode4(uint32_t codes, float scale, float (&x)[4])
{
    const auto a = __builtin_amdgcn_cvt_pk_f32_fp8((int)codes, false);
    const auto b = __builtin_amdgcn_cvt_pk_f32_fp8((int)codes, true);
    x[0] = a[0] * scale; x[1] = a[1] * scale; x[2] = b[0] * scale; x[3] = b[1] * scale;
}

__device__ __forceinline__ float inverse8(uint32_t b) { return __uint_as_float((254u - b) << 23); }

// The exponent byte of a block from the largest of its values' abs_bits, and
// whether any of them is infinite, NaN or in the last binade.  Infinite ones and NaN
// leave the others' scale alone (the largest finite one sets it) and get NaN's
// code; in the last binade rounding up to what stands for infinity is held back
// (kLast8).  x: the lane's values, zero where it has none.  V: roots.
struct Top8 {
    uint32_t b;
    bool special;
};

template <bool V, int N>
__device__ __forceinline__ Top8 top8(const float (&x)[N])
{
    float f = 0.0f;   // (the maximum that NaN goes through: three operands, magnitudes for free)
#pragma unroll
    for (int i = 0; i < N; ++i) f = __builtin_elementwise_maximum(f, fabsf(x[i]));
    uint32_t t = wave_max(abs_bits(f));
    const bool special = t >= kHugeBits[V];
    if (t >= kInfBits) {
        t = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) t = max(t, abs_bits(x[i]) >= kInfBits ? 0u : abs_bits(x[i]));
        t = wave_max(t);
    }
    const int b = (int)(t >> 23) - kTop8;
    return Top8{(uint32_t)(b > 1 ? b : 1), special};
}

// 32 mixed bits of 32 (the multipliers are the fractions of the square roots of 2
// and 3): every input bit reaches every output bit.
__device__ __forceinline__ uint32_t mix32(uint32_t x)
{
    x = (x ^ (x >> 16)) * 0x6A09E667u;
    x = (x ^ (x >> 15)) * 0xBB67AE85u;
    return x ^ (x >> 16);
}

// Rounding of a step's result.  With b2 = 0.999 a step changes v by a thousandth, far
// below half a code's distance, so rounding to the nearest would hold v still
// for ever: a value is rounded up with the probability of what lies below it, by 16
// random bits, so the mean over steps is right.  The bits are a hash of the
// block's place in the shard, the count in its word and the element's place in it:
// the same state and gradients give the same bits, in a replayed graph too.
__device__ __forceinline__ uint32_t key8(uint32_t first, uint32_t count) { return mix32(mix32(first) + count); }

// x's code, rounded by 16 bits, into byte J of `old`.  The instruction divides by the
// scale (a power of two) and adds the upper 20 of its 32 random bits below the last
// bit kept: floor(|x| / step + u / 65536) steps, over the whole range of codes.
template <int J>
__device__ __forceinline__ uint32_t put_random(uint32_t old, float x, float scale, uint32_t bits16_high)
{
    return (uint32_t)__builtin_amdgcn_cvt_scalef32_sr_fp8_f32((int)old, x, bits16_high, scale, J);
}

// A code in a block with special values (see top8).
template <bool V>
__device__ __forceinline__ uint32_t held8(float x, uint32_t code, const Top8& t)
{
    uint32_t c = code & 0x7fu;
    if (t.b == kLastB[V]) c = min(c, kLast8);
    return abs_bits(x) >= kInfBits ? kNan8 : c | (code & 0x80u);
}

// m's code, and r's: a root that is not zero does not become zero (m / (0 + eps)
// would throw the parameter off), it stays at the smallest step.
__device__ __forceinline__ uint32_t code_m(float m, uint32_t bits, const Top8& t)
{
    const uint32_t c = put_random<0>(0, m, scale8(t.b), bits << 16) & 0xffu;
    return t.special ? held8<false>(m, c, t) : c;
}

__device__ __forceinline__ uint32_t code_r(float r, uint32_t bits, const Top8& t)
{
    uint32_t c = put_random<0>(0, r, scale8(t.b), bits & 0xffff0000u) & 0xffu;
    c = max(c, r > 0.0f ? 1u : 0u);
    return t.special ? held8<true>(r, c & 0x7fu, t) : c;
}

// Four codes of m and of r from their elements' bits: an instruction a code, but in
// blocks with special values and, of r, where a lane has a code of zero (which may
// stand for a root that is not zero).
__device__ __forceinline__ void codes4(const float (&m)[4], const float (&r)[4], const uint32_t (&bits)[4],
                                       const Top8& tm, const Top8& tr, uint32_t& cm, uint32_t& cr)
{
    const float sm = scale8(tm.b), sr = scale8(tr.b);
    cm = put_random<0>(0, m[0], sm, bits[0] << 16);
    cm = put_random<1>(cm, m[1], sm, bits[1] << 16);
    cm = put_random<2>(cm, m[2], sm, bits[2] << 16);
    cm = put_random<3>(cm, m[3], sm, bits[3] << 16);
    cr = put_random<0>(0, r[0], sr, bits[0] & 0xffff0000u);
    cr = put_random<1>(cr, r[1], sr, bits[1] & 0xffff0000u);
    cr = put_random<2>(cr, r[2], sr, bits[2] & 0xffff0000u);
    cr = put_random<3>(cr, r[3], sr, bits[3] & 0xffff0000u);
    if (tm.special) {
        cm = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) cm |= code_m(m[j], bits[j], tm) << (8 * j);
    }
    if (tr.special || __any(((cr - 0x01010101u) & ~cr & 0x80808080u) != 0)) {
        cr = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) cr |= code_r(r[j], bits[j], tr) << (8 * j);
    }
}

__device__ __forceinline__ uint32_t next_word(uint32_t word, uint32_t b) { return ((word & ~255u) + 256u) | b; }

}  // namespace dev8
}  // namespace z1
