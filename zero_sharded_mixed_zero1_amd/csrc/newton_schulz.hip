// newton_schulz.hip -- orthogonalisation by Newton-Schulz products on gfx950.
//
// One step of the iteration on X (k x n, k <= n; a tall u enters transposed):
//   A = X X^T,  B = b A + c A A,  X <- a X + B X.
// Three grouped products a step over the matrices of a group, each a launch:
// gram (A, upper triangle of tiles and their mirror images), poly (B,
// likewise: A is symmetric, so A A is), apply (X).
//
// Number format.  The matrix cores multiply fp16 (11 bits, the same rate as
// bf16's 8) and add in fp32.  X, A and B are stored times S = 2^12: their
// entries are bounded by the singular values (X by at most 3, A by 9, B by 12,
// checked on the host for the given coefficients), so nothing overflows, and
// entries down to 2^-26 keep all their bits.  X is held as two fp16 halves,
// hi + lo (22 bits): a X is formed from both, the products from hi alone.
// With hi alone every rounding of X is a new direction of full rank that the
// iteration multiplies by up to a^steps: on matrices with a few strong
// directions the result is off by 2-3 % (25 % with bf16), with both halves by
// 0.04-0.2 % in five steps before its own rounding to bf16 (0.17 %); the worst
// spectrum found, equal singular values, by 0.35 %.  A and B need one half: their
// roundings are multiplied by X, not added to it.
//
// What bounds it: the matrix cores at the clock that the chip's power allows (about
// 1.8 GHz with all of them busy) and, near them, the LDS reads that feed them; for
// small matrices what a launch costs beside its products (2 us, then 1.8 us until
// the first tiles have come from memory, and an epilogue of about 1 us).  Measured:
// 4096 x 11008 (192 x 192 tiles for A and B, 256 x 256 for X) gram 204 us, poly 83,
// apply 352: 905, 830 and 1050 TFLOP/s of what A's symmetry leaves; twelve 768 x 768
// gram 12.3 us, poly 13.1, apply 20.1.
//
// The norm enters as a power of two 2^e, exact on the way into fp16, and a
// factor r in [1, 2) folded into the first step: X = r Xs / S.
//
// Layout: X, A and B lie in blocks of 64 x 64 (8 KiB), block rows one after the
// other, rows of 128 bytes inside a block with their 16-byte slots permuted
// (slot_key).  A block is what the products stage: eight loads of 1 KiB go from
// memory to LDS as they lie, and from there both directions read without bank
// conflicts: along rows (ds_read_b128) and, for X in B X, down columns
// (ds_read_b64_tr_b16).  The padding up to 64 is zero and stays zero.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "muon.h"

namespace z1 {
namespace {

using namespace dev;

typedef _Float16 half_t;
typedef half_t h4 __attribute__((ext_vector_type(4)));
typedef half_t h8 __attribute__((ext_vector_type(8)));
typedef short s4 __attribute__((ext_vector_type(4)));

constexpr int kB = kPad;                 // block side
constexpr int kBlock = kB * kB;          // elements of a block

// What the 16-byte slots of row r are XORed with, so that what sixteen lanes
// read at once falls into different banks (64 banks: 256 bytes, two rows).
// Along rows they read one slot of 16 neighbouring rows: the key takes each
// value once over (r >> 1) & 7.  Down columns they read 32 bytes of 4
// neighbouring rows, the four groups of a wave rows 8 apart: bits 0 and 2 of
// r >> 1 select the 32-byte unit.  (A key over r & 7 costs the second kind 19 %
// more LDS cycles.)
__device__ __forceinline__ int slot_key(int r)
{
    const int v = r >> 1;
    return ((v >> 1) & 1) | ((v & 1) << 1) | (v & 4);
}

// ------------------------------------------------------------- prepare
// Xs = 2^e u as hi (and lo where u is fp32: a bf16 u fits hi exactly), u
// transposed if tall, zeros in the padding.  One workgroup a block.
// Given `partials`, each workgroup forms its matrix's norm from them itself, and
// the first one stores it for the products.
template <typename U>
__global__ __launch_bounds__(kThreads) void ns_prepare_kernel(NsArgs g, const double* partials, double eps,
                                                              NormRec* norms)
{
    constexpr bool LO = sizeof(U) == 4;
    __shared__ float sh[kB][kB + 1];
    __shared__ double sums[1][kThreads / 64];
    const ProdTile pt = g.blocks[blockIdx.x];
    const MatDesc& d = g.mats[pt.mat];
    const U* u = static_cast<const U*>(d.u);
    const int i0 = pt.i * kB, j0 = pt.j * kB;
    // rows of u are rows of X, or columns when u is tall
    const int a0 = d.tall ? j0 : i0, b0 = d.tall ? i0 : j0;
    float v[4][4];
    const int c = 4 * (threadIdx.x & 15), r0 = threadIdx.x >> 4;
#pragma unroll
    for (int h = 0; h < 4; ++h) {   // (rows and columns are more than kThin here)
        const int64_t row = a0 + r0 + 16 * h;
        const bool in = row < d.rows;
        load_padded<false>(u + (in ? row : 0) * d.ldu, b0 + c, d.cols, in, v[h]);
    }
    int e;
    if (partials) {
        const NormRec n = matrix_norm(d, partials, eps, sums);
        e = n.e;
        if (pt.i == 0 && pt.j == 0 && threadIdx.x == 0) norms[pt.mat] = n;
    } else {
        e = norms[pt.mat].e;
    }
#pragma unroll
    for (int h = 0; h < 4; ++h)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const float x = ldexpf(v[h][q], e);
            if (d.tall) sh[c + q][r0 + 16 * h] = x;
            else sh[r0 + 16 * h][c + q] = x;
        }
    __syncthreads();
    const Buffers buf = buffers(pt.at, pt.kb, pt.nb);
    const int64_t at = ((int64_t)pt.i * pt.nb + pt.j) * kBlock;
    half_t* hi = reinterpret_cast<half_t*>(g.area + buf.x0) + at;
    half_t* lo = reinterpret_cast<half_t*>(g.area + buf.lo) + at;
#pragma unroll
    for (int h = 0; h < kBlock / 8 / kThreads; ++h) {
        const int slot = threadIdx.x + h * kThreads, r = slot >> 3, j = ((slot & 7) ^ slot_key(r)) << 3;
        h8 vh, vl;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            vh[q] = (half_t)sh[r][j + q];
            vl[q] = (half_t)(sh[r][j + q] - (float)vh[q]);
        }
        *reinterpret_cast<h8*>(hi + slot * 8) = vh;
        if constexpr (LO) *reinterpret_cast<h8*>(lo + slot * 8) = vl;
    }
}

// ------------------------------------------------------------- products
// C = P Q^T of a tile of (64 MB WR) x (64 WC): WR x WC waves, each of 64 MB
// rows and 64 columns in MFMAs of 16 x 16 x 32.  The operands of the MFMA are
// swapped, so that a lane holds four neighbouring columns of C:
// acc[x][y][r] = C[16 x + (lane & 15)][16 y + 4 (lane >> 4) + r].
//
// S stages of 64 of the inner dimension lie in LDS: while one is multiplied,
// the loads of the next S - 1 are under way.
template <int WR, int WC, int MB, int S>
struct Tile {
    static constexpr int kWaves = WR * WC, kThr = 64 * kWaves;
    static constexpr int kRowBlocks = WR * MB, kColBlocks = WC, kBlocks = kRowBlocks + kColBlocks;
    static constexpr int kStage = kBlocks * kBlock;            // elements of a stage
    static constexpr int kLoads = (kBlocks * 8 + kWaves - 1) / kWaves;   // 1 KiB loads a wave issues a stage
    static constexpr bool kEven = kBlocks * 8 % kWaves == 0;
    static constexpr size_t kStages = (size_t)S * kStage * 2, kOuts = (size_t)kWaves * kBlock * 4;
    static constexpr size_t kLds = kStages > kOuts ? kStages : kOuts;
    static_assert(kLds <= 160 * 1024, "LDS of a CU");
    // Waves a SIMD that registers are left for (not what LDS allows: with half of
    // LDS to itself a kernel of four waves would be given 512 registers, half of
    // them behind copies).  LDS is dynamic for the same reason.
    static constexpr int kMinBlocks = kThr == 256 ? 2 : 1;
    // registers left for the epilogue's operands while the product runs (256 a
    // lane at two waves a SIMD; three leave 168)
    static constexpr bool kAhead = MB == 1 && kWaves <= 4;
};

// One wave copies 1 KiB from memory to LDS: lane l its 16 bytes at base +
// 16 l, to lds + 16 l.  No register receives the data; whoever reads it waits
// (stage_wait) first.  The compiler does not know that m0 is written (it reserves
// m0 and takes no such clobber), so nothing else in this file's kernels may use it:
// a test reads their assembly for that.
__device__ __forceinline__ void load_1k(const half_t* base, uint32_t lane_off, uint32_t lds)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
                 :
                 : "s"(lds), "v"(lane_off), "s"(base)
                 : "memory");
}

// All of this wave's loads but the N youngest have reached LDS.
template <int N>
__device__ __forceinline__ void stage_wait()
{
    static_assert(N >= 0 && N < 64, "vmcnt is six bits");
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// Reads a block in LDS down its columns: a lane gets column c0 + (lane & 15), rows
// r0 + 8 (lane >> 4) and the next seven.  (It gives the address of 8 bytes: of row
// ((lane & 15) >> 2) of a group of four, a quarter of the 16 columns.)
__device__ __forceinline__ h8 columns(const half_t* block, int r0, int c0)
{
    typedef __attribute__((address_space(3))) s4 lds_s4;
    const int lane = threadIdx.x & 63;
    union { s4 s[2]; h8 v; } both;
#pragma unroll
    for (int z = 0; z < 2; ++z) {
        const int r = r0 + 8 * (lane >> 4) + ((lane & 15) >> 2) + 4 * z, c = c0 + 4 * (lane & 3);
        const half_t* a = block + r * kB + (((c >> 3) ^ slot_key(r)) << 3) + (c & 7);
        both.s[z] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4*)a);
    }
    return both.v;
}

// P: block row p0 of a matrix of `pc` blocks a row and `pr` block rows, read
// along its rows; Q: block row q0 of one of `qr` by `qc` likewise, or, with QT,
// block column q0, read down its columns.  `steps` blocks of the inner
// dimension.  Tiles past the last block row or column repeat it (their results
// are not stored).  `ahead` runs when the last stage has arrived: the loads that
// it issues delay none of the product's.
template <typename T, int WR, int WC, int MB, int S, bool QT, typename F>
__device__ __forceinline__ void product(const half_t* P, int p0, int pr, int pc, const half_t* Q, int q0, int qr,
                                        int qc, int steps, half_t* sh, f32x4 (&acc)[4 * MB][4], F ahead)
{
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int wi = wave / WC, wj = wave % WC;
    const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) half_t*)sh;
    const half_t* src[T::kLoads];
    int64_t adv[T::kLoads];
    uint32_t dst[T::kLoads];
#pragma unroll
    for (int l = 0; l < T::kLoads; ++l) {
        // (where the loads do not divide evenly, the last waves repeat the last)
        const int idx = T::kEven ? wave * T::kLoads + l : min(wave * T::kLoads + l, T::kBlocks * 8 - 1);
        const int blk = idx >> 3, part = idx & 7;
        if (blk < T::kRowBlocks) {
            const int b = p0 + blk < pr ? p0 + blk : pr - 1;
            src[l] = P + (int64_t)b * pc * kBlock + part * 512;
            adv[l] = kBlock;
        } else if (!QT) {
            const int b = q0 + blk - T::kRowBlocks < qr ? q0 + blk - T::kRowBlocks : qr - 1;
            src[l] = Q + (int64_t)b * qc * kBlock + part * 512;
            adv[l] = kBlock;
        } else {
            const int b = q0 + blk - T::kRowBlocks < qc ? q0 + blk - T::kRowBlocks : qc - 1;
            src[l] = Q + (int64_t)b * kBlock + part * 512;
            adv[l] = (int64_t)qc * kBlock;
        }
        dst[l] = lds0 + idx * 1024;
    }
    auto issue = [&](int buf) {
#pragma unroll
        for (int l = 0; l < T::kLoads; ++l) {
            load_1k(src[l], lane * 16, dst[l] + buf * (T::kStage * 2));
            src[l] += adv[l];
        }
    };
#pragma unroll
    for (int x = 0; x < 4 * MB; ++x)
#pragma unroll
        for (int y = 0; y < 4; ++y) acc[x][y] = f32x4{0, 0, 0, 0};
    // lane's place in a block: row lane & 15 (of 16), slot lane >> 4 (+ 4 for
    // the second half of the inner block); rows 16 apart have the same key
    const int row = lane & 15, key = slot_key(row);
    const int off[2] = {row * kB + (((lane >> 4) ^ key) << 3), row * kB + (((4 + (lane >> 4)) ^ key) << 3)};
    struct Frag {
        h8 p[4 * MB], q[4];
    };
    // the wave's operands for half h of the stage in buffer `buf`
    auto read = [&](Frag& f, int buf, int h) {
        const half_t* sp = sh + buf * T::kStage + wi * MB * kBlock;
        const half_t* sq = sh + buf * T::kStage + (T::kRowBlocks + wj) * kBlock;
#pragma unroll
        for (int y = 0; y < 4; ++y) {
            if constexpr (!QT) {
                f.q[y] = *reinterpret_cast<const h8*>(sq + y * 16 * kB + off[h]);
            } else {
                f.q[y] = columns(sq, 32 * h, 16 * y);
            }
        }
#pragma unroll
        for (int x = 0; x < 4 * MB; ++x) f.p[x] = *reinterpret_cast<const h8*>(sp + x * 16 * kB + off[h]);
    };
    auto multiply = [&](const Frag& f) {
#pragma unroll
        for (int x = 0; x < 4 * MB; ++x)
#pragma unroll
            for (int y = 0; y < 4; ++y)
                acc[x][y] = __builtin_amdgcn_mfma_f32_16x16x32_f16(f.q[y], f.p[x], acc[x][y], 0, 0, 0);
    };
    // the order that a half is scheduled in: its MFMAs with the LDS reads of the
    // next spread between them
    auto spread = [] {
        constexpr int kMfma = 16 * MB, kReads = 4 * MB + (QT ? 8 : 4), kEach = kMfma / kReads;
#pragma unroll
        for (int i = 0; i < kReads; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x008, kEach, 0);
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        }
        __builtin_amdgcn_sched_group_barrier(0x008, kMfma - kReads * kEach, 0);
    };
    // each half's operands are read from LDS while the half before is
    // multiplied; the barrier lies between the halves, when this wave's reads
    // of stage t are done and its loads of stage t + 1 have arrived
    int put = 0, get = 0;   // buffers: the next one to load into, the one to read
    auto next = [](int b) { return b + 1 == S ? 0 : b + 1; };
#pragma unroll
    for (int k = 0; k < S; ++k)
        if (k < steps) {
            issue(put);
            put = next(put);
        }
    Frag f0, f1;
    if (steps > S - 1) stage_wait<(S - 1) * T::kLoads>();
    else stage_wait<0>();
    __syncthreads();
    read(f0, get, 0);
    for (int t = 0; t < steps; ++t) {
        read(f1, get, 1);
        multiply(f0);
        spread();
        if (t + 1 < steps) {
            if (t + S - 1 < steps) stage_wait<(S - 2) * T::kLoads>();   // stages t + 2 .. t + S - 1 may be under way
            else stage_wait<0>();
            __syncthreads();
            if (t + S < steps) {
                issue(put);
                put = next(put);
            }
            if (t + 2 == steps) ahead();
            get = next(get);
        }
        // (the last round reads the last stage again: the loop stays one block)
        read(f0, get, 0);
        multiply(f1);
        spread();
    }
    __syncthreads();   // the stages are free for the epilogue
}

// LDS accesses of one wave execute in order; this keeps the compiler from
// moving them past each other.
__device__ __forceinline__ void wave_sync()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Where a wave's fp32 copy of a block in LDS holds (row, col): its quads of four
// columns are XORed with a key that takes 16 values over 16 rows (a wave writes
// quads of 16 rows at once), other ones in the next rows (it reads quads of four
// rows), and pairs over columns (for a tall u): the first two meet in no bank,
// the third in two.
__device__ __forceinline__ int spot(int row, int col)
{
    const int key = (((row ^ (row >> 3)) & 7) << 1) | (row & 1);
    return row * kB + (((col >> 2) ^ key) << 2) + (col & 3);
}

// Where a block holds the quads of a lane's accumulators: row 16 x + (lane & 15),
// columns 16 y + 4 (lane >> 4).
__device__ __forceinline__ int quad(int x, int y)
{
    const int lane = threadIdx.x & 63, row = lane & 15;   // (rows 16 apart have the same key)
    return (16 * x + row) * kB + (((2 * y + (lane >> 5)) ^ slot_key(row)) << 3) + ((lane >> 4) & 1) * 4;
}

// All of a lane's quads of a block, in flight.
__device__ __forceinline__ void load_quads(const half_t* block, h4 (&v)[4][4])
{
#pragma unroll
    for (int x = 0; x < 4; ++x)
#pragma unroll
        for (int y = 0; y < 4; ++y) v[x][y] = *reinterpret_cast<const h4*>(block + quad(x, y));
}

// A block that the wave has put together in LDS to memory, whole slots.
__device__ __forceinline__ void store_block(half_t* block, const half_t* lds)
{
#pragma unroll
    for (int h = 0; h < 8; ++h) {
        const int at = ((threadIdx.x & 63) + 64 * h) * 8;
        *reinterpret_cast<h8*>(block + at) = *reinterpret_cast<const h8*>(lds + at);
    }
}

// One 64 x 64 block of the wave's accumulators into its part of LDS, in fp32.
__device__ __forceinline__ void stage_block(const f32x4 (*acc)[4], float* out)
{
    const int lane = threadIdx.x & 63;
    wave_sync();
#pragma unroll
    for (int x = 0; x < 4; ++x)
#pragma unroll
        for (int y = 0; y < 4; ++y)
            *reinterpret_cast<f32x4*>(out + spot(16 * x + (lane & 15), 16 * y + 4 * (lane >> 4))) = acc[x][y];
    wave_sync();
}

// A lane's slots of a block, all in flight.
__device__ __forceinline__ void load_slots(const half_t* block, h8 (&v)[8])
{
#pragma unroll
    for (int h = 0; h < 8; ++h) v[h] = *reinterpret_cast<const h8*>(block + ((threadIdx.x & 63) + 64 * h) * 8);
}

enum Op : int { kGram = 0, kPoly = 1 };

// A = X X^T or B = b A + c A A: the blocks of the upper triangle, each stored
// with its mirror image.
template <int OP, int WR, int WC, int MB, int S>
__global__ __launch_bounds__(64 * WR * WC, (Tile<WR, WC, MB, S>::kMinBlocks))
void ns_sym_kernel(NsArgs g, int it)
{
    using T = Tile<WR, WC, MB, S>;
    extern __shared__ __attribute__((aligned(1024))) char lds[];
    const ProdTile pt = g.sym[blockIdx.x];
    const Buffers buf = buffers(pt.at, pt.kb, pt.nb);
    const half_t* src = reinterpret_cast<const half_t*>(g.area + (OP == kGram ? (it & 1 ? buf.x1 : buf.x0) : buf.a));
    half_t* dst = reinterpret_cast<half_t*>(g.area + (OP == kGram ? buf.a : buf.b));
    const int kb = pt.kb, inner = OP == kGram ? pt.nb : kb;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int bj = pt.j + wave % WC;
    const float r = it == 0 ? g.norms[pt.mat].r : 1.0f;
    const int lane_row = lane & 15, key = slot_key(lane_row);   // (rows 16 apart have the same key)
    h4 av[4][4];
    auto operands = [&](int bi) {   // A of the epilogue's block (bi, bj)
        if (OP == kPoly && bi <= bj && bj < kb) {
            const half_t* a = src + ((int64_t)bi * kb + bj) * kBlock;
            load_quads(a, av);
        }
    };
    f32x4 acc[4 * MB][4];
    product<T, WR, WC, MB, S, false>(src, pt.i, kb, inner, src, pt.j, kb, inner, inner, reinterpret_cast<half_t*>(lds),
                                     acc, [&] { if constexpr (T::kAhead) operands(pt.i + wave / WC); });
    half_t* out = reinterpret_cast<half_t*>(lds) + wave * kBlock;
    const float f = OP == kGram ? r * r / kNsScale : g.c / kNsScale;
#pragma unroll
    for (int m = 0; m < MB; ++m) {
        const int bi = pt.i + (wave / WC) * MB + m;
        if (bi > bj || bi >= kb || bj >= kb) continue;   // below the diagonal, or past the end
        if constexpr (!T::kAhead) operands(bi);
        half_t* at = dst + ((int64_t)bi * kb + bj) * kBlock;
        half_t* mirror = dst + ((int64_t)bj * kb + bi) * kBlock;
        wave_sync();
#pragma unroll
        for (int x = 0; x < 4; ++x)
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                f32x4 z = f * acc[4 * m + x][y];
                if constexpr (OP == kPoly) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) z[q] = fmaf(g.b, (float)av[x][y][q], z[q]);
                }
                *reinterpret_cast<h4*>(out + quad(x, y)) = __builtin_convertvector(z, h4);
            }
        wave_sync();
        store_block(at, out);
        if (bi == bj) continue;
        // the mirror image: a lane gets column 16 y + lane_row, rows 32 h + 8 (lane >> 4)
        // and the next seven, as one slot (A is its own transpose bit for bit, so
        // b A needs no other block)
#pragma unroll
        for (int y = 0; y < 4; ++y)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                *reinterpret_cast<h8*>(mirror + (16 * y + lane_row) * kB + (((4 * h + (lane >> 4)) ^ key) << 3)) =
                    columns(out, 32 * h, 16 * y);
    }
}

// A = X X^T of matrices of few block rows: a 64 x 64 block a workgroup, each wave
// every fourth inner block through two stages of its own (nothing to wait for but
// its own loads), the four sums joined in LDS in a fixed order.  A tile's workgroup
// walks the inner dimension at 0.5 us a block however few there are, here it walks
// a quarter: 2 of 4050 x 209 take 13.6 us (6 tiles of 128 x 128: 33.1).
constexpr size_t kSplitLds = (size_t)4 * 2 * 2 * kBlock * 2;

__global__ __launch_bounds__(256, 2) void ns_gram_split_kernel(NsArgs g, int it)
{
    extern __shared__ __attribute__((aligned(1024))) char lds[];
    constexpr int kLoads = 16;
    const ProdTile pt = g.gram[blockIdx.x];
    const Buffers buf = buffers(pt.at, pt.kb, pt.nb);
    const half_t* src = reinterpret_cast<const half_t*>(g.area + (it & 1 ? buf.x1 : buf.x0));
    half_t* dst = reinterpret_cast<half_t*>(g.area + buf.a);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const float r = it == 0 ? g.norms[pt.mat].r : 1.0f;
    half_t* sh = reinterpret_cast<half_t*>(lds) + wave * (4 * kBlock);
    const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) half_t*)sh;
    const half_t* row[2] = {src + ((int64_t)pt.i * pt.nb + wave) * kBlock, src + ((int64_t)pt.j * pt.nb + wave) * kBlock};
    const int count = (pt.nb - wave + 3) / 4;
    auto issue = [&](int b) {
#pragma unroll
        for (int l = 0; l < kLoads; ++l)
            load_1k(row[l >> 3] + (l & 7) * 512, lane * 16, lds0 + (b * 2 * kBlock + l * 512) * 2);
        row[0] += 4 * kBlock;
        row[1] += 4 * kBlock;
    };
    f32x4 acc[4][4];
#pragma unroll
    for (int x = 0; x < 4; ++x)
#pragma unroll
        for (int y = 0; y < 4; ++y) acc[x][y] = f32x4{0, 0, 0, 0};
    const int lane_row = lane & 15, key = slot_key(lane_row);
    const int off[2] = {lane_row * kB + (((lane >> 4) ^ key) << 3), lane_row * kB + (((4 + (lane >> 4)) ^ key) << 3)};
    if (count > 0) issue(0);
    if (count > 1) issue(1);
    for (int t = 0; t < count; ++t) {
        if (t + 1 < count) stage_wait<kLoads>();   // the next stage may be under way
        else stage_wait<0>();
        const half_t* s = sh + (t & 1) * (2 * kBlock);
        h8 p[2][4], q[2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                p[h][x] = *reinterpret_cast<const h8*>(s + x * 16 * kB + off[h]);
                q[h][x] = *reinterpret_cast<const h8*>(s + kBlock + x * 16 * kB + off[h]);
            }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // read before it is loaded over
        if (t + 2 < count) issue(t & 1);
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int x = 0; x < 4; ++x)
#pragma unroll
                for (int y = 0; y < 4; ++y)
                    acc[x][y] = __builtin_amdgcn_mfma_f32_16x16x32_f16(q[h][y], p[h][x], acc[x][y], 0, 0, 0);
    }
    __syncthreads();
    f32x4* join = reinterpret_cast<f32x4*>(lds);
#pragma unroll
    for (int x = 0; x < 4; ++x)
#pragma unroll
        for (int y = 0; y < 4; ++y) join[((wave * 4 + x) * 4 + y) * 64 + lane] = acc[x][y];
    __syncthreads();
    // each wave finishes rows 16 wave .. 16 wave + 15
    half_t* out = reinterpret_cast<half_t*>(lds) + 4 * 2 * kBlock;   // behind the four sums
    const float f = r * r / kNsScale;
#pragma unroll
    for (int y = 0; y < 4; ++y) {
        f32x4 z = join[((0 * 4 + wave) * 4 + y) * 64 + lane];
#pragma unroll
        for (int w = 1; w < 4; ++w) z += join[((w * 4 + wave) * 4 + y) * 64 + lane];
        *reinterpret_cast<h4*>(out + quad(wave, y)) = __builtin_convertvector(f * z, h4);
    }
    __syncthreads();
    half_t* at = dst + ((int64_t)pt.i * pt.kb + pt.j) * kBlock;
    half_t* mirror = dst + ((int64_t)pt.j * pt.kb + pt.i) * kBlock;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int slot = (threadIdx.x + 256 * h) * 8;
        *reinterpret_cast<h8*>(at + slot) = *reinterpret_cast<const h8*>(out + slot);
    }
    if (pt.i != pt.j) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
            *reinterpret_cast<h8*>(mirror + (16 * wave + lane_row) * kB + (((4 * h + (lane >> 4)) ^ key) << 3)) =
                columns(out, 32 * h, 16 * wave);
    }
}

// The end of the last step for one block of o, staged in `out`: o as bf16, or
// the update of the master and the parameter with it.  Rows of o are the
// block's rows, or its columns when u is tall; four elements a lane, the loads
// of eight quads in flight.
template <int LAST>
__device__ __forceinline__ void finish_block(const MatDesc& d, const float* out, int bi, int bj, const MuonArgs& ma)
{
    const int lane = threadIdx.x & 63;
    const int64_t r0 = (int64_t)(d.tall ? bj : bi) * kB, c0 = (int64_t)(d.tall ? bi : bj) * kB;
    const float eta = ma.lr * d.scale;
    const int c = 4 * (lane & 15), rl = lane >> 4;
    const Span4 s = span4<false>(c0 + c, d.cols, true);
#pragma unroll
    for (int h0 = 0; h0 < 16; h0 += 8) {
        auto row_of = [&](int h) { return r0 + 4 * (h0 + h) + rl; };
        float v[8][4];
        if constexpr (LAST == kNsUpdate) {
#pragma unroll
            for (int h = 0; h < 8; ++h) {
                const int64_t r = row_of(h);
                load_quad<false>(d.master + (r < d.rows ? r : 0) * d.ld + s.col, 0, v[h]);
            }
        }
#pragma unroll
        for (int h = 0; h < 8; ++h) {
            const int rr = 4 * (h0 + h) + rl;
            const int64_t row = row_of(h);
            if (row >= d.rows) continue;
            // columns c .. c + 3 of o; a quad that begins `skip` elements early holds
            // column c there
            float w[4], o[4];
            if (d.tall) {
#pragma unroll
                for (int q = 0; q < 4; ++q) w[q] = out[spot(c + q, rr)];
            } else {
                const f32x4 x = *reinterpret_cast<const f32x4*>(out + spot(rr, c));
#pragma unroll
                for (int q = 0; q < 4; ++q) w[q] = x[q];
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                o[q] = w[q];
#pragma unroll
                for (int k = 1; k <= q; ++k) o[q] = s.skip == k ? w[q - k] : o[q];
            }
            if constexpr (LAST == kNsWriteO) {
                store_quad<false>(d.o + row * d.ldo + s.col, s.skip, o);
            } else {
#pragma unroll
                for (int q = 0; q < 4; ++q) v[h][q] = muon_elem(v[h][q], o[q], eta, ma);
                store_quad<false>(d.master + row * d.ld + s.col, s.skip, v[h]);
                store_quad<false>(d.param + row * d.ld + s.col, s.skip, v[h]);
            }
        }
    }
}

// X <- a X + B X; the last step writes o as bf16, or updates the master and
// the parameter with it, instead of X.
template <int LAST, int WR, int WC, int MB, int S>
__global__ __launch_bounds__(64 * WR * WC, (Tile<WR, WC, MB, S>::kMinBlocks))
void ns_apply_kernel(NsArgs g, int it, int has_lo, MuonArgs ma)
{
    using T = Tile<WR, WC, MB, S>;
    extern __shared__ __attribute__((aligned(1024))) char lds[];
    const ProdTile pt = g.full[blockIdx.x];
    const Buffers buf = buffers(pt.at, pt.kb, pt.nb);
    const half_t* xi = reinterpret_cast<const half_t*>(g.area + (it & 1 ? buf.x1 : buf.x0));
    half_t* xo = reinterpret_cast<half_t*>(g.area + (it & 1 ? buf.x0 : buf.x1));
    half_t* lo = reinterpret_cast<half_t*>(g.area + buf.lo);
    const half_t* bm = reinterpret_cast<const half_t*>(g.area + buf.b);
    const int kb = pt.kb, nb = pt.nb;
    MatDesc d;
    if constexpr (LAST != kNsMid) d = g.mats[pt.mat];
    if constexpr (LAST == kNsUpdate) use_device_scalars(ma, nullptr);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int bj = pt.j + wave % WC;
    const float r = it == 0 ? g.norms[pt.mat].r : 1.0f;
    h8 xh[8], xl[8] = {};
    auto operands = [&](int bi) {   // of the epilogue's block (bi, bj)
        if (bi < kb && bj < nb) {
            const int64_t at = ((int64_t)bi * nb + bj) * kBlock;
            load_slots(xi + at, xh);
            if (has_lo) load_slots(lo + at, xl);
        }
    };
    f32x4 acc[4 * MB][4];
    product<T, WR, WC, MB, S, true>(bm, pt.i, kb, kb, xi, pt.j, kb, nb, kb, reinterpret_cast<half_t*>(lds), acc,
                                    [&] { if constexpr (T::kAhead) operands(pt.i + wave / WC); });
    float* out = reinterpret_cast<float*>(lds) + wave * kBlock;
    const float scale = LAST == kNsMid ? 1.0f : 1.0f / kNsScale;
    const float fa = g.a * r * scale, fb = r / kNsScale * scale;
#pragma unroll
    for (int m = 0; m < MB; ++m) {
        const int bi = pt.i + (wave / WC) * MB + m;
        if (bi >= kb || bj >= nb) continue;
        const int64_t at = ((int64_t)bi * nb + bj) * kBlock;
        if constexpr (!T::kAhead) operands(bi);
        stage_block(acc + 4 * m, out);
#pragma unroll
        for (int h = 0; h < 8; ++h) {
            const int slot = lane + 64 * h, row = slot >> 3, j = ((slot & 7) ^ slot_key(row)) << 3;
            f32x4* const x[2] = {reinterpret_cast<f32x4*>(out + spot(row, j)), reinterpret_cast<f32x4*>(out + spot(row, j + 4))};
            h8 vh, vl;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                f32x4 z = *x[e];
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    z[q] = fmaf(fb, z[q], fmaf(fa, (float)xh[h][4 * e + q], fa * (float)xl[h][4 * e + q]));
                if constexpr (LAST == kNsMid) {
                    const h4 hi = __builtin_convertvector(z, h4);
#pragma unroll
                    for (int q = 0; q < 4; ++q) z[q] = fmaf(-1.0f, (float)hi[q], z[q]);
                    const h4 rest = __builtin_convertvector(z, h4);
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        vh[4 * e + q] = hi[q];
                        vl[4 * e + q] = rest[q];
                    }
                } else {
                    *x[e] = z;
                }
            }
            if constexpr (LAST == kNsMid) {
                *reinterpret_cast<h8*>(xo + at + slot * 8) = vh;
                *reinterpret_cast<h8*>(lo + at + slot * 8) = vl;
            }
        }
        if constexpr (LAST != kNsMid) {
            wave_sync();
            finish_block<LAST>(d, out, bi, bj, ma);
        }
    }
}

}  // namespace

// ------------------------------------------------------------------ launchers
hipError_t launch_ns_prepare(const NsArgs& g, bool u_f32, const double* partials, double eps, NormRec* norms, int grid,
                             hipStream_t s)
{
    if (u_f32) ns_prepare_kernel<float><<<dim3(grid), dim3(kThreads), 0, s>>>(g, partials, eps, norms);
    else ns_prepare_kernel<uint16_t><<<dim3(grid), dim3(kThreads), 0, s>>>(g, partials, eps, norms);
    return hipGetLastError();
}

constexpr int kFewTiles = 256;   // as many as the whole chip has CUs

#define Z1_TILES(tile, CALL)                              \
    do {                                                  \
        if ((tile) == kTile256) CALL(2, 4, 2, 2);         \
        else if ((tile) == kTile192) CALL(3, 3, 1, 3);    \
        else CALL(2, 2, 1, 2);                            \
    } while (0)

hipError_t launch_ns_gram(const NsArgs& g, int it, TileShape tile, int grid, hipStream_t s)
{
#define Z1_CALL(WR, WC, MB, S) ns_sym_kernel<kGram, WR, WC, MB, S><<<dim3(grid), dim3(64 * WR * WC), Tile<WR, WC, MB, S>::kLds, s>>>(g, it)
    // Where no CU has two tiles, LDS has room for two stages more, whose loads
    // then cover the first touch of X by the chip.  Two against four: 3 of 1111 x
    // 2501 27.2 and 24.8 us, 1000 x 1000 12.3 and 11.7, 12 of 768 x 768 12.3 both,
    // 192 x 192 4.2 and 4.4; poly and apply, whose operands are smaller, lose by it
    // (13.1 and 13.4; 13.9 and 14.3).
    if (tile == kTile128 && grid <= kFewTiles) Z1_CALL(2, 2, 1, 4);
    else Z1_TILES(tile, Z1_CALL);
#undef Z1_CALL
    return hipGetLastError();
}

hipError_t launch_ns_gram_split(const NsArgs& g, int it, int grid, hipStream_t s)
{
    ns_gram_split_kernel<<<dim3(grid), dim3(256), kSplitLds, s>>>(g, it);
    return hipGetLastError();
}

hipError_t launch_ns_poly(const NsArgs& g, TileShape tile, int grid, hipStream_t s)
{
#define Z1_CALL(WR, WC, MB, S) ns_sym_kernel<kPoly, WR, WC, MB, S><<<dim3(grid), dim3(64 * WR * WC), Tile<WR, WC, MB, S>::kLds, s>>>(g, 1)
    Z1_TILES(tile, Z1_CALL);
#undef Z1_CALL
    return hipGetLastError();
}

hipError_t launch_ns_apply(const NsArgs& g, int it, bool u_f32, NsLast last, const MuonArgs& ma, TileShape tile,
                           int grid, hipStream_t s)
{
    const int has_lo = it > 0 || u_f32 ? 1 : 0;
#define Z1_APPLY(LAST, WR, WC, MB, S) \
    ns_apply_kernel<LAST, WR, WC, MB, S><<<dim3(grid), dim3(64 * WR * WC), Tile<WR, WC, MB, S>::kLds, s>>>(g, it, has_lo, ma)
#define Z1_MID(WR, WC, MB, S) Z1_APPLY(kNsMid, WR, WC, MB, S)
#define Z1_O(WR, WC, MB, S) Z1_APPLY(kNsWriteO, WR, WC, MB, S)
#define Z1_UPD(WR, WC, MB, S) Z1_APPLY(kNsUpdate, WR, WC, MB, S)
    if (last == kNsMid) Z1_TILES(tile, Z1_MID);
    else if (last == kNsWriteO) Z1_TILES(tile, Z1_O);
    else Z1_TILES(tile, Z1_UPD);
#undef Z1_UPD
#undef Z1_O
#undef Z1_MID
#undef Z1_APPLY
    return hipGetLastError();
}
#undef Z1_TILES

}  // namespace z1
