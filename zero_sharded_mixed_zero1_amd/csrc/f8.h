// f8.h -- matrices in 8-bit floating point with a scale for each block of 128:
// what the host side (f8_api.cpp) and the kernels (f8_quantize.hip,
// f8_product.hip) share.
//
// A matrix of rows x cols is rows of codes (e4m3 or e5m2, OCP), padded with zeros
// to whole blocks of 128 columns, and one byte b for each block of 128 columns of
// one row or of 128 rows: a code stands for itself times 2^(b-127).  Why powers of
// two: the matrix cores take such a scale with each operand, so a block's scale
// costs the product nothing; and a floating point code loses no precision to it,
// only up to one binade of the 17 that e4m3 has.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace z1 {

constexpr int kF8Block = 128;

// A matrix as the kernels see it.
struct F8 {
    uint8_t* codes;        // NULL: absent (quantize)
    uint8_t* scales;
    int64_t rows, cols, ld, ld_scales;
    int shift;             // row >> shift is the row of its scales: 0 or 7
    int e5m2;
};

// Quantizes src (rows x cols, bf16 or fp32) into q, its transpose into qt.
hipError_t launch_f8_quantize(const void* src, bool f32, int64_t rows, int64_t cols, int64_t ld, const F8& q,
                              const F8& qt, hipStream_t s);

// Which kernel a product takes (f8_product.hip): few rows of A, or tiles of 64 x 64,
// 128 x 128 or 256 x 256 of D (the last into bf16 only).
enum F8Kind : int { kF8Thin, kF8Tile64, kF8Tile128, kF8Tile256 };

// D[i][j] = sum over k of a(i, k) b(j, k).
struct F8Product {
    F8 a, b;
    void* d;
    int64_t ldd;
    int f32;               // D is fp32, else bf16
    int vec;               // D and its rows begin at multiples of 16 bytes
    int kind;              // F8Kind
    int parts, part_steps; // the summed axis in parts of so many blocks of 128
    int64_t whole;         // 256: tiles of a workgroup each; the others' workgroups take
    int bands;             // 256 / bands rows
    float* sums;           // parts > 1: their sums, rows of ld_sums, part_elems a part
    int64_t ld_sums, part_elems;
};
hipError_t launch_f8_product(const F8Product& p, hipStream_t s);

}  // namespace z1
