// muon.h -- declarations shared by the Muon entry points' host code
// (muon_api.cpp) and kernels (muon.hip, newton_schulz.hip).  Not part of the
// public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "internal.h"

namespace z1 {

// Streaming kernels (momentum, update, sum of squares): a workgroup's tile is
// 512 quads, a quad being up to four neighbouring elements of one row.
constexpr int kQuadsPerTile = 512;
constexpr int kSumsqTiles = 4;     // tiles that a workgroup of the sum of squares takes at once
// Side of the square blocks that X, A and B are laid out in and padded to.
constexpr int kPad = 64;
// Power of two that X, A and B carry in fp16 (see newton_schulz.hip).
constexpr float kNsScale = 4096.0f;

// One matrix.  "x" is the matrix the iteration works on: u, or u transposed
// when u is tall, so that k = min(rows, cols) rows of n = max(rows, cols).
struct MatDesc {
    int64_t rows, cols, ld, shard_offset, ldu, ldo;
    uint16_t* param;
    float* master;
    void* m;
    void* u;
    uint16_t* o;
    float scale;
    int32_t tall;
    int32_t k, n, kp, np;          // kp, np: k, n rounded up to kPad
    // the streaming kernels' view: vrows rows of vcols elements, qpr quads each
    // (one row when the matrix and its u and o are contiguous)
    int64_t vcols, qpr;
    int32_t vrows;
    int32_t tile0, n_tiles;        // its streaming tiles
    int32_t split, n_parts;        // thin: columns a part of the gram sum, parts
    int32_t reserved;
    // byte offsets inside the workspace's group area: of a thin matrix fp32 X, the
    // parts' exponents, the parts, P; of others X (twice), its low halves, A and B,
    // which the kernels form from x[0] (Buffers): the plans' test reads them here
    int64_t x[2], lo, a, b;
};
static_assert(sizeof(MatDesc) == 192, "matrix descriptor layout");

// A streaming tile: quads [512 idx, +512) of matrix `mat`, the first of them
// quad q0 of row row0.
struct StreamTile {
    int32_t mat, idx, row0, q0;
};

// A tile of one matrix's product: its first block row i and block column j.
// With what of the matrix the products need beside it (`at`: d.x[0]; kb, nb:
// blocks of kp and np), so that a workgroup knows its addresses after one load
// from memory, not two in a row: 0.4 us of the 13.8 that a gram of 768 x 768 took.
struct ProdTile {
    int64_t at;
    int32_t mat, i, j, kb, nb, reserved;
};
static_assert(sizeof(ProdTile) == 32, "tile layout");

// Matrices with k up to this take the kernels of ns_thin.hip.
constexpr int kThin = 128;
constexpr int kThinMaxParts = 32;
constexpr int kThinOne = 256;      // n up to this: one workgroup does all of a matrix of k <= 64
// The iteration's buffers of a matrix that is not thin: byte offsets of X (two
// copies), its low halves, A and B.
struct Buffers {
    int64_t x0, x1, lo, a, b, end;
};

inline __host__ __device__ Buffers buffers(int64_t at, uint32_t kb, uint32_t nb)
{   // (numbers of blocks fit 32 bits, and 32-bit products stay in scalar registers)
    const int64_t x = (int64_t)(kb * nb) * (2 * kPad * kPad), a = (int64_t)(kb * kb) * (2 * kPad * kPad);
    return Buffers{at, at + x, at + 2 * x, at + 3 * x, at + 3 * x + a, at + 3 * x + 2 * a};
}

// How much a segment's steps before its last may grow small singular values
// (ns_thin.hip).
constexpr double kThinGrowth = 160.0;

// Matrices of at most this many streaming tiles: every workgroup of prepare forms
// its matrix's norm from their partial sums; for larger ones a launch before it
// does.  Prepare alone and both: 288 tiles 9.2 and 10.4 us, 1357 tiles 11.3 and
// 13.1, 2048 tiles 9.2 and 12.2, 4096 tiles 12.0 and 12.2.
constexpr int kNormTiles = 2048;

// A = X X^T of few block rows and a long inner dimension (blocks): each 64 x 64
// block is a workgroup's, whose four waves take every fourth inner block.  By the
// matrix alone, so that its sums are in one order whatever else is in the plan.
// Against 128 x 128 tiles: 2 of 4050 x 209 13.6 us and 33.1, 1 of 512 x 4096 13.6
// and 33.6, 6 of 500 x 2000 9.8 and 19.4, 12 of 512 x 2048 17.6 and 20.4; where
// such tiles fill the chip it is even or behind: 24 of 384 x 1152 13.9 and 13.6,
// 64 of 320 x 2048 39.0 and 37.3, 40 of 512 x 2048 62 and 43 (a step takes 158).
constexpr int kSplitRows = 8, kSplitInner = 16;

// Shapes of the products' tiles.
enum TileShape : int { kTile128 = 0, kTile192 = 1, kTile256 = 2 };

// Norm of one matrix's u as the iteration uses it: S / (norm + eps) = 2^e r
// with r in [1, 2); r is NaN when the quotient is not finite.
struct NormRec {
    float r;
    int32_t e;
};

// Per-step scalars (zero1_muon_scalars).
struct MuonScal {
    float lr, mu, delta, reserved;
    double max_norm;
};

struct MuonArgs {
    float lr, mu, delta;
    const MuonScal* dev;           // non-null: read lr, mu, delta, max_norm from here
    int decay_first;
};

// Clip prologue; rank_sumsq null: no clipping.
struct MuonClip {
    const double* rank_sumsq;
    int n_ranks;
    double max_norm;
    int clip_eps;
    NormInfo* info_out;
};

struct NsArgs {
    const MatDesc* mats;
    const ProdTile* sym;           // tiles of A and B; of thin matrices the parts of the gram sum
                                   // (i: the part, j: its first 64 columns)
    const ProdTile* full;          // tiles of X; of thin matrices X's columns in 64s (j)
    const ProdTile* blocks;        // blocks of X; of thin matrices none
    const ProdTile* gram;          // blocks of A, where the gram is split (kSplitRows)
    int first;                     // the group's first matrix
    char* area;                    // the workspace's group area
    const NormRec* norms;
    float a, b, c;
};

enum NsLast : int { kNsMid = 0, kNsWriteO = 1, kNsUpdate = 2 };

hipError_t launch_momentum(const Reduce& r, const MatDesc* mats, const StreamTile* tiles, int n_tiles, bool m_bf16,
                           bool u_f32, bool nesterov, const MuonArgs& ma, const MuonClip& mc, double* partials,
                           int nblocks, int split, hipStream_t s);
hipError_t launch_u_sumsq(const MatDesc* mats, const StreamTile* tiles, int n_tiles, bool u_f32, double* partials,
                          int nblocks, int split, hipStream_t s);
hipError_t launch_ns_norms(const MatDesc* mats, int n_mats, const double* partials, double eps, NormRec* norms,
                           hipStream_t s);
hipError_t launch_muon_update(const MatDesc* mats, const StreamTile* tiles, int n_tiles, const MuonArgs& ma,
                              int nblocks, int split, hipStream_t s);

// partials: the norms are formed here too (else launch_ns_norms has).
hipError_t launch_ns_prepare(const NsArgs& g, bool u_f32, const double* partials, double eps, NormRec* norms, int grid,
                             hipStream_t s);
hipError_t launch_ns_gram(const NsArgs& g, int it, TileShape tile, int grid, hipStream_t s);
hipError_t launch_ns_gram_split(const NsArgs& g, int it, int grid, hipStream_t s);
hipError_t launch_ns_poly(const NsArgs& g, TileShape tile, int grid, hipStream_t s);
hipError_t launch_ns_apply(const NsArgs& g, int it, bool u_f32, NsLast last, const MuonArgs& ma, TileShape tile,
                           int grid, hipStream_t s);

// Thin matrices padded to kp (32, 64 or 128) rows; f32: X is read as fp32; mid:
// from the workspace.
hipError_t launch_thin_gram(const NsArgs& g, int kp, bool f32, int mid, int grid, hipStream_t s);
hipError_t launch_thin_poly(const NsArgs& g, int kp, int mid, int steps, double eps, NormRec* norms, int grid,
                            hipStream_t s);
// The parts' sum, where there is more than one.
hipError_t launch_thin_sum(const NsArgs& g, int kp, int n_mats, hipStream_t s);
// A group of matrices of one part and k <= 64, in one launch (from u, all
// steps in one segment).
hipError_t launch_thin_one(const NsArgs& g, int kp, bool f32, int steps, double eps, NormRec* norms, NsLast last,
                           const MuonArgs& ma, int n_mats, hipStream_t s);
hipError_t launch_thin_apply(const NsArgs& g, int kp, bool f32, int mid, NsLast last, const MuonArgs& ma, int grid,
                             hipStream_t s);

#ifdef __HIPCC__
// ------------------------------------------------------------------ device
namespace dev {

template <typename T>
using gptr = __attribute__((address_space(1))) T*;

// Vectors of four elements at any element's address: rows of an odd stride
// start anywhere, and gfx950 loads and stores them whole all the same.
typedef uint16_t u16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef u16x4 u16x4u __attribute__((aligned(2)));
typedef f32x4 f32x4u __attribute__((aligned(4)));

template <bool KEEP = false>
__device__ __forceinline__ u16x4 ld4(const uint16_t* p)
{
    if constexpr (KEEP) return *(gptr<const u16x4u>)p;
    else return __builtin_nontemporal_load((gptr<const u16x4u>)p);
}
template <bool KEEP = false>
__device__ __forceinline__ f32x4 ld4(const float* p)
{
    if constexpr (KEEP) return *(gptr<const f32x4u>)p;
    else return __builtin_nontemporal_load((gptr<const f32x4u>)p);
}
__device__ __forceinline__ void st4(uint16_t* p, u16x4 v) { __builtin_nontemporal_store(v, (gptr<u16x4u>)p); }
__device__ __forceinline__ void st4(float* p, f32x4 v) { __builtin_nontemporal_store(v, (gptr<f32x4u>)p); }

// What the iteration starts with, from the sum of squares of u.  A zero matrix
// stays one at any scale, but for eps = 0: then, and when the norm is infinite or
// NaN, u / (norm + eps) holds a NaN and the iteration spreads it over the whole
// matrix.  (No other norm leaves the exponents: the least is 2^-149.)
__device__ __forceinline__ NormRec norm_rec(double sumsq, double eps)
{
    if (sumsq == 0.0 && eps > 0.0) return NormRec{1.0f, 0};
    const double f = (double)kNsScale / (sqrt(sumsq) + eps);
    if (!(f > 0.0) || isinf(f)) return NormRec{__builtin_nanf(""), 0};
    const int e = ilogb(f);
    return NormRec{(float)ldexp(f, -e), e};
}

// x plus the x of another lane, as the data-parallel primitive CTRL picks it
// (zero where it picks none or the row is masked out).
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_add(double x)
{
    const long long b = __double_as_longlong(x);
    const int lo = __builtin_amdgcn_update_dpp(0, (int)b, CTRL, ROWS, 0xf, true);
    const int hi = __builtin_amdgcn_update_dpp(0, (int)(b >> 32), CTRL, ROWS, 0xf, true);
    return x + __longlong_as_double(((long long)hi << 32) | (unsigned)lo);
}

// The sum over a wave, in lane 63, in a fixed order: within rows of 16 lanes,
// then across the rows.  (Six exchanges through LDS take twelve of its
// instructions a tile and bound a pass over bf16.)
__device__ __forceinline__ double wave_sum(double x)
{
    x = dpp_add<0x111, 0xf>(x);   // row_shr 1, 2, 4, 8
    x = dpp_add<0x112, 0xf>(x);
    x = dpp_add<0x114, 0xf>(x);
    x = dpp_add<0x118, 0xf>(x);
    x = dpp_add<0x142, 0xa>(x);   // row_bcast 15: rows 0, 2 into 1, 3
    x = dpp_add<0x143, 0xc>(x);   // row_bcast 31: rows 0-1 into 2-3
    return x;
}

// Fixed-order workgroup sums of N tiles at once, one number a wave in `sh` at
// the end.  `sh` alternates between two buffers, so one barrier a round is
// enough.
template <int N>
__device__ __forceinline__ void tile_sums(double (&x)[N], double (*sh)[kThreads / 64])
{
#pragma unroll
    for (int k = 0; k < N; ++k) {
        x[k] = wave_sum(x[k]);
        if ((threadIdx.x & 63) == 63) sh[k][threadIdx.x >> 6] = x[k];
    }
    __syncthreads();
}

__device__ __forceinline__ double four(const double (&s)[kThreads / 64]) { return ((s[0] + s[1]) + s[2]) + s[3]; }

// The start of a matrix's iteration from its streaming tiles' partial sums, added
// in a fixed order by a workgroup of kThreads; all of it gets the result.
__device__ __forceinline__ NormRec matrix_norm(const MatDesc& d, const double* __restrict__ partials, double eps,
                                               double (*sums)[kThreads / 64])
{
    double a = 0.0;
    for (int i0 = threadIdx.x; i0 < d.n_tiles; i0 += 16 * kThreads) {   // 16 loads in flight
        double x[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) x[k] = i0 + k * kThreads < d.n_tiles ? partials[d.tile0 + i0 + k * kThreads] : 0.0;
#pragma unroll
        for (int k = 0; k < 16; ++k) a = a + x[k];
    }
    double x[1] = {a};
    tile_sums<1>(x, sums);
    return norm_rec(four(sums[0]), eps);
}

__device__ __forceinline__ float widen(uint16_t h) { return __uint_as_float((uint32_t)h << 16); }

// Nearest-even bf16; NaNs stay quiet NaNs with their sign.
__device__ __forceinline__ uint16_t bf16_rne(float x)
{
    const uint32_t u = __float_as_uint(x);
    const uint32_t r = (u + 0x7fffu + ((u >> 16) & 1u)) >> 16;
    return (uint16_t)(((u & 0x7fffffffu) > 0x7f800000u) ? ((u >> 16) | 0x40u) : r);
}

__device__ __forceinline__ void use_device_scalars(MuonArgs& a, double* max_norm)
{
    if (a.dev) {
        const MuonScal d = *a.dev;
        a.lr = d.lr;
        a.mu = d.mu;
        a.delta = d.delta;
        if (max_norm) *max_norm = d.max_norm;
    }
}

// p moves by eta*o and is multiplied by the decay factor (decay_first swaps
// the two); eta = lr * the matrix's scale.
__device__ __forceinline__ float muon_elem(float p, float o, float eta, const MuonArgs& a)
{
#pragma clang fp contract(off)
    if (a.decay_first) return p * a.delta - eta * o;
    return (p - eta * o) * a.delta;
}

// A quad: four neighbouring elements of a row, loaded and stored whole.  The
// last quad of a row that is no multiple of four long begins `skip` elements
// early, so that it too can be loaded whole; those elements belong to the quad
// before, and are not stored.  skip = 4: nothing of it is the lane's (it loads
// from wherever the caller points it).  Rows shorter than four elements have
// one quad with `skip` negative: -skip elements, one by one.
__device__ __forceinline__ void widen4(u16x4 v, float (&x)[4])
{
    x[0] = widen(v.x); x[1] = widen(v.y); x[2] = widen(v.z); x[3] = widen(v.w);
}

template <bool SHORT, bool KEEP = false>
__device__ __forceinline__ void load_quad(const uint16_t* p, int skip, float (&x)[4])
{
    if constexpr (SHORT) {
#pragma unroll
        for (int j = 0; j < 3; ++j) x[j] = j < -skip ? widen(p[j]) : 0.0f;
        x[3] = 0.0f;
    } else {
        widen4(ld4<KEEP>(p), x);
    }
}

template <bool SHORT, bool KEEP = false>
__device__ __forceinline__ void load_quad(const float* p, int skip, float (&x)[4])
{
    if constexpr (SHORT) {
#pragma unroll
        for (int j = 0; j < 3; ++j) x[j] = j < -skip ? p[j] : 0.0f;
        x[3] = 0.0f;
    } else {
        const f32x4 v = ld4<KEEP>(p);
        x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
    }
}

// Whether element j of a quad is the lane's.
template <bool SHORT>
__device__ __forceinline__ bool owns(int skip, int j)
{
    return SHORT ? j < -skip : j >= skip;
}

// Stores the lane's elements in the array's type; x becomes what was stored.
template <bool SHORT>
__device__ __forceinline__ void store_quad(uint16_t* p, int skip, float (&x)[4])
{
    const u16x4 v = {bf16_rne(x[0]), bf16_rne(x[1]), bf16_rne(x[2]), bf16_rne(x[3])};
    widen4(v, x);
    if (!SHORT && skip == 0) {
        st4(p, v);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (owns<SHORT>(skip, j)) p[j] = v[j];
    }
}

template <bool SHORT>
__device__ __forceinline__ void store_quad(float* p, int skip, float (&x)[4])
{
    if (!SHORT && skip == 0) {
        st4(p, f32x4{x[0], x[1], x[2], x[3]});
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (owns<SHORT>(skip, j)) p[j] = x[j];
    }
}

// The quad of columns [c, c + 4) of a row of `cols`: where it begins and its
// skip; nothing of it is the lane's unless `in`.
struct Span4 {
    int64_t col;
    int skip;
};

template <bool SHORT>
__device__ __forceinline__ Span4 span4(int64_t c, int64_t cols, bool in)
{
    if constexpr (SHORT) return Span4{0, in && c == 0 ? -(int)cols : 0};
    const int64_t left = cols - c;
    if (!in || left <= 0) return Span4{0, 4};
    if (left >= 4) return Span4{c, 0};
    return Span4{cols - 4, 4 - (int)left};
}

// Elements c .. c + 3 of a row of `cols` in x, zeros past its end.
template <bool SHORT, typename T>
__device__ __forceinline__ void load_padded(const T* row, int64_t c, int64_t cols, bool in, float (&x)[4])
{
    const Span4 s = span4<SHORT>(c, cols, in);
    float v[4];
    load_quad<SHORT, true>(row + s.col, s.skip, v);
    if constexpr (SHORT) {
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = v[j];
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float y = v[j];
#pragma unroll
            for (int k = 1; k <= 4; ++k) y = s.skip == k ? (j + k < 4 ? v[(j + k) & 3] : 0.0f) : y;
            x[j] = y;
        }
    }
}

}  // namespace dev
#endif

}  // namespace z1
