// f8_product.hip -- D = A B^T of matrices in 8-bit floating point with a power of
// two for each block of 128 (f8.h) on gfx950's matrix cores.
//
// Into bf16: v_mfma_scale_f32_32x32x64_f8f6f4 multiplies 32 x 64 codes by 32 x 64 and
// takes a scale for each operand's row, so two instructions are one block of 128,
// scales included.  It adds groups of eight neighbouring products, each cut toward
// zero to a multiple of 2^(E - 13), E the largest sum of two codes' exponents in the
// group (one below the smallest normal code counts as that; zeros do not count; found by
// adding powers of two and products of 15 by 15; beyond the groups sums keep
// fp32's 24 bits).  On random operands that takes 1e-5 to 8e-5 of the result, a
// hundredth of bf16's own rounding; at worst 7 * 2^-13 of each group's largest product,
// whatever the result is, so a sum that cancels may lose most of what is left.  Taken
// all the same, because the way without it costs: 8192 x 11008 x 4096 takes 610 us by
// the bf16 instructions and 310 so, 2048 x 4096 x 4096 63 and 39, 1 x 1024 x 8192 8.6
// and 6.1, 1 x 11008 x 4096 12.4 and 11.5.
// Into fp32 the cuts would be the largest error there is, so codes are widened to bf16
// with their scales (each exactly) and multiplied as bf16, which adds to
// 24 bits (7e-8), at half the rate: the way for sums that cancel.
//
// The operands are swapped (B's rows first), so that a lane holds four neighbouring
// columns of D: acc[x][y][r] = D[32 x + (lane & 31)][32 y + 8 (r >> 2) + 4 (lane >>
// 5) + (r & 3)].
//
// What bounds it: at 8192 x 11008 x 4096 (321 us among other passes, 2.3 PFLOP/s; by
// itself under the profiler 332) the clock that power leaves (1.8 GHz, the matrix cores busy 63 % of it; operands that lie in L2 gain 5 to
// 10 %); between 512 and 2048 rows whole rounds of the chip and the first stages' latency
// (2048 x 4096 x 4096 34.9 us, 2.0 PFLOP/s; into fp32 60, 1.1); up to 32 rows memory (1 x
// 11008 x 4096 10.2 us, 4.4 TB/s).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "f8.h"
#include "internal.h"

namespace z1 {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kLine = kF8Block;    // bytes of a row of a stage in LDS

// What the 16-byte slots of row r are XORed with: what a few neighbouring lanes read
// at once is one slot of as many rows, 128 bytes apart (64 banks: two rows), and the
// key takes each value once over eight pairs of rows.
__device__ __forceinline__ int slot_key(int r) { return (r >> 1) & 7; }

// Loads from memory to LDS: lane l its 16 (or 4) bytes at base + off to lds + 16 l (4
// l).  No register receives the data; whoever reads it waits (stage_wait) first.
// The compiler does not know that m0 is written (it reserves m0 and takes no such
// clobber), so nothing else in this file's kernels may use it: a test reads their
// assembly for that.
__device__ __forceinline__ void load_1k(const uint8_t* base, uint32_t off, uint32_t lds)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" : : "s"(lds), "v"(off), "s"(base) : "memory");
}

__device__ __forceinline__ void load_256(const uint8_t* base, uint32_t off, uint32_t lds)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, %2" : : "s"(lds), "v"(off), "s"(base) : "memory");
}

// All of this wave's loads but the N youngest have reached LDS.
template <int N>
__device__ __forceinline__ void stage_wait()
{
    static_assert(N >= 0 && N < 64, "vmcnt is six bits");
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// LDS accesses of one wave execute in order; this keeps the compiler from
// moving them past each other.
__device__ __forceinline__ void wave_sync()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
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

__device__ __forceinline__ void narrow4(f32x4 v, float* o) { *reinterpret_cast<f32x4*>(o) = v; }
__device__ __forceinline__ void narrow4(f32x4 v, __bf16* o) { *reinterpret_cast<bf16x4*>(o) = __builtin_convertvector(v, bf16x4); }

// A tile of D: WR x WC waves, each of 32 PX rows and 32 QY columns.  S stages of one
// block of 128 of the summed axis lie in LDS: while one is multiplied, the loads
// of the next S - 1 are under way.
template <int WR, int WC, int PX, int QY, int S>
struct Tile {
    static constexpr int kWaves = WR * WC, kThr = 64 * kWaves;
    static constexpr int kRows = 32 * PX * WR, kCols = 32 * QY * WC, kLines = kRows + kCols;
    static constexpr int kLoads = kLines / 8 / kWaves;                       // of 1 KiB, a wave a stage
    static constexpr int kScaleLoads = (kLines / 64 + kWaves - 1) / kWaves;  // of 64 rows' scales
    static constexpr int kInFlight = kLoads + kScaleLoads;
    static constexpr int kStage = kLines * kLine + kLines * 4;
    static constexpr int kPitch = 32 * QY * 4 + 16;                          // of a wave's 32 rows on their way out
    static constexpr int kOut = kWaves * 32 * kPitch;
    static constexpr int kLds = S * kStage > kOut ? S * kStage : kOut;
    static_assert(kLds <= 160 * 1024 && kRows % 64 == 0 && kCols % 64 == 0 && kLines / 8 % kWaves == 0, "tile");
};

struct Yes { static constexpr bool value = true; };
struct No { static constexpr bool value = false; };

// Workgroup b of n runs on XCD b % 8: each XCD takes one contiguous eighth.
__device__ __forceinline__ int64_t xcd_part(int64_t b, int64_t n)
{
    const int64_t x = b % 8, q = n / 8, rest = n % 8;
    return x * q + (x < rest ? x : rest) + b / 8;
}

// Tile t of D, in an order that keeps what an XCD works on at once close to a square:
// in bands of 8 tile rows, down a band's columns first.
__device__ __forceinline__ void tile_at(int64_t t, int64_t tiles_m, int64_t tiles_n, int64_t& i, int64_t& j)
{
    const int64_t band = t / (8 * tiles_n), high = tiles_m - band * 8 < 8 ? tiles_m - band * 8 : 8, in = t - band * 8 * tiles_n;
    i = band * 8 + in % high;
    j = in / high;
}

// EXACT: widened to bf16.  Each of p.parts workgroups of a tile adds up p.part_steps
// blocks of the summed axis; where there are more than one, they leave their sums
// in fp32 for join_kernel.
template <int WR, int WC, int PX, int QY, int S, int FA, int FB, bool EXACT, typename D>
__device__ __forceinline__ void tile(const F8Product& p, uint8_t* lds, int64_t m0, int64_t n0, int64_t part)
{
    using T = Tile<WR, WC, PX, QY, S>;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int wi = wave / WC, wj = wave % WC;
    const int from = (int)part * p.part_steps;
    const int steps = min(p.part_steps, (int)((p.a.cols + kF8Block - 1) / kF8Block) - from);

    // what this wave loads: lines of 128 bytes (A's rows, then B's), eight a load,
    // their 16-byte slots permuted on the way; then 64 rows' scales of four blocks.
    // Rows past the end repeat the last one.
    const uint8_t* const ca = p.a.codes + m0 * p.a.ld + (int64_t)from * kF8Block;
    const uint8_t* const cb = p.b.codes + n0 * p.b.ld + (int64_t)from * kF8Block;
    const uint8_t* const sa = p.a.scales + (m0 >> p.a.shift) * p.a.ld_scales;
    const uint8_t* const sb = p.b.scales + (n0 >> p.b.shift) * p.b.ld_scales;
    const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds;
    const int last_a = (int)(p.a.rows - 1 - m0 < T::kRows ? p.a.rows - 1 - m0 : T::kRows - 1);
    const int last_b = (int)(p.b.rows - 1 - n0 < T::kCols ? p.b.rows - 1 - n0 : T::kCols - 1);
    uint32_t off[T::kLoads], soff[T::kScaleLoads];
#pragma unroll
    for (int l = 0; l < T::kLoads; ++l) {
        const int first = (wave * T::kLoads + l) * 8, line = first + (lane >> 3);
        const uint32_t slot = 16 * ((lane & 7) ^ slot_key(line));
        if (first < T::kRows) off[l] = (uint32_t)min(line, last_a) * (uint32_t)p.a.ld + slot;
        else off[l] = (uint32_t)min(line - T::kRows, last_b) * (uint32_t)p.b.ld + slot;
    }
#pragma unroll
    for (int l = 0; l < T::kScaleLoads; ++l) {
        const int first = min(wave * T::kScaleLoads + l, T::kLines / 64 - 1) * 64, line = first + lane;
        if (first < T::kRows) soff[l] = (uint32_t)(((m0 + min(line, last_a)) >> p.a.shift) - (m0 >> p.a.shift)) * (uint32_t)p.a.ld_scales;
        else soff[l] = (uint32_t)(((n0 + min(line - T::kRows, last_b)) >> p.b.shift) - (n0 >> p.b.shift)) * (uint32_t)p.b.ld_scales;
    }
    auto issue_scales = [&](int t, uint32_t at) {
#pragma unroll
        for (int l = 0; l < T::kScaleLoads; ++l) {
            const int first = min(wave * T::kScaleLoads + l, T::kLines / 64 - 1) * 64;
            load_256((first < T::kRows ? sa : sb) + ((from + t) & ~3), soff[l], at + T::kLines * kLine + first * 4);
        }
    };
    auto issue = [&](int t, int buf) {
        const uint32_t at = lds0 + buf * T::kStage;
        const uint8_t *la = ca + (int64_t)t * kF8Block, *lb = cb + (int64_t)t * kF8Block;
#pragma unroll
        for (int l = 0; l < T::kLoads; ++l) {
            const int first = (wave * T::kLoads + l) * 8;
            load_1k(first < T::kRows ? la : lb, off[l], at + first * kLine);
        }
        issue_scales(t, at);
    };

    f32x16 acc[PX][QY];
#pragma unroll
    for (int x = 0; x < PX; ++x)
#pragma unroll
        for (int y = 0; y < QY; ++y)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[x][y][r] = 0.0f;

    // the lane's place in 32 lines: half h of a block is slots 4 h + (lane >> 5) and
    // two further (which bytes is the same for both operands, so the sum is over the
    // whole block either way)
    const int key = slot_key(lane & 31);
    int place[2][2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int c = 0; c < 2; ++c) place[h][c] = (lane & 31) * kLine + 16 * ((4 * h + 2 * c + (lane >> 5)) ^ key);
    union Codes {
        u32x4 v[2];
        i32x8 f;
    };
    const uint8_t* const lds_p = lds + wi * 32 * PX * kLine;
    const uint8_t* const lds_q = lds + (T::kRows + wj * 32 * QY) * kLine;
    auto read_p = [&](Codes& v, int buf, int x, int h) {
#pragma unroll
        for (int c = 0; c < 2; ++c) v.v[c] = *reinterpret_cast<const u32x4*>(lds_p + buf * T::kStage + x * 32 * kLine + place[h][c]);
    };
    auto read_q = [&](Codes (&v)[QY], int buf, int h) {
#pragma unroll
        for (int y = 0; y < QY; ++y)
#pragma unroll
            for (int c = 0; c < 2; ++c) v[y].v[c] = *reinterpret_cast<const u32x4*>(lds_q + buf * T::kStage + y * 32 * kLine + place[h][c]);
    };
    auto read_scales = [&](int (&ep)[PX], int (&eq)[QY], int buf, int t) {
        const uint8_t* e = lds + buf * T::kStage + T::kLines * kLine + ((from + t) & 3) + 4 * (lane & 31);
#pragma unroll
        for (int x = 0; x < PX; ++x) ep[x] = e[4 * (wi * 32 * PX + 32 * x)];
#pragma unroll
        for (int y = 0; y < QY; ++y) eq[y] = e[4 * (T::kRows + wj * 32 * QY + 32 * y)];
    };

    int put = 0, get = 0;   // buffers: the next one to load into, the one to read
    auto next = [](int b) { return b + 1 == S ? 0 : b + 1; };
#pragma unroll
    for (int k = 0; k < S; ++k)
        if (k < steps) {
            issue(k, put);
            put = next(put);
        }
    // A stage is 2 PX turns, each of the QY MFMAs of 32 rows and one half of the
    // block.  A turn's operands are read from LDS in the turn before; at the last turn
    // this wave's reads of the stage are done, so there lies the barrier after
    // which the next stage is read and the stage after the following loaded.  (All
    // of a half's operands read ahead instead takes 40 registers more and 4 % more
    // time at 8192 x 11008 x 4096.)  EXACT: a turn is a half of the block, so that
    // each code is widened once.
    int ep[PX], eq[QY], np[PX], nq[QY];
    constexpr int kTurns = EXACT ? 2 : 2 * PX;
    Codes rp[EXACT ? 2 * PX : 2], rq[2][QY];
    auto stage = [&](int t, auto more_, auto last_) {
        constexpr bool more = decltype(more_)::value, last = decltype(last_)::value;
#pragma unroll
        for (int i = 0; i < kTurns; ++i) {
            if (i == kTurns - 1) {
                if constexpr (!last) {
                    if constexpr (more) stage_wait<(S - 2) * T::kInFlight>();   // stages t + 2 .. t + S - 1 may be under way
                    else stage_wait<0>();
                    __syncthreads();
                    get = next(get);
                }
                // (the last round reads the last stage again)
                read_q(rq[0], get, 0);
                read_scales(np, nq, get, last ? t : t + 1);
            }
            if (EXACT ? i == 0 : i == PX - 1) read_q(rq[1], get, 1);
            if constexpr (EXACT) {
#pragma unroll
                for (int x = 0; x < PX; ++x) read_p(rp[(1 - i) * PX + x], get, x, 1 - i);
            } else {
                read_p(rp[(i + 1) & 1], get, (i + 1) % PX, (i + 1) % kTurns / PX);
            }
            if constexpr (more) {
                if (i == kTurns - 1) issue(t + S, put);
            }
            if constexpr (EXACT) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    bf16x8 wp[PX], wq[QY];
#pragma unroll
                    for (int x = 0; x < PX; ++x)
                        wp[x] = widen8<FA>((uint32_t)rp[i * PX + x].f[2 * j], (uint32_t)rp[i * PX + x].f[2 * j + 1], power(ep[x]));
#pragma unroll
                    for (int y = 0; y < QY; ++y)
                        wq[y] = widen8<FB>((uint32_t)rq[i][y].f[2 * j], (uint32_t)rq[i][y].f[2 * j + 1], power(eq[y]));
#pragma unroll
                    for (int x = 0; x < PX; ++x)
#pragma unroll
                        for (int y = 0; y < QY; ++y) acc[x][y] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(wq[y], wp[x], acc[x][y], 0, 0, 0);
                }
            } else {
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int y = 0; y < QY; ++y)
                    acc[i % PX][y] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(rq[i / PX][y].f, rp[i & 1].f, acc[i % PX][y], FB, FA, 0,
                                                                                     eq[y], 0, ep[i % PX]);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        if constexpr (more) put = next(put);
#pragma unroll
        for (int x = 0; x < PX; ++x) ep[x] = np[x];
#pragma unroll
        for (int y = 0; y < QY; ++y) eq[y] = nq[y];
    };
    if (steps > 0) {
        if (steps > S - 1) stage_wait<(S - 1) * T::kInFlight>();
        else stage_wait<0>();
        __syncthreads();
        read_q(rq[0], get, 0);
        read_scales(ep, eq, get, 0);
#pragma unroll
        for (int x = 0; x < (EXACT ? PX : 1); ++x) read_p(rp[x], get, x, 0);
        int t = 0;
        for (; t + S < steps; ++t) stage(t, Yes{}, No{});
        for (; t + 1 < steps; ++t) stage(t, No{}, No{});
        stage(t, No{}, Yes{});
    }
    __syncthreads();   // the stages are free for the way out

    // 32 rows of the wave at a time through LDS, to leave as whole rows
    constexpr int kVec = 16 / (int)sizeof(D), kRowVecs = 32 * QY / kVec, kPitch = T::kPitch / 4 * (int)sizeof(D) + (sizeof(D) == 2 ? 8 : 0);
    static_assert(kPitch % 16 == 0, "rows in LDS begin at 16 bytes");
    uint8_t* out = lds + wave * 32 * T::kPitch;
    D* const d = static_cast<D*>(p.d) + part * p.part_elems;
    const bool vec = p.vec != 0;
#pragma unroll
    for (int x = 0; x < PX; ++x) {
        wave_sync();
#pragma unroll
        for (int y = 0; y < QY; ++y)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const f32x4 v = {acc[x][y][4 * g], acc[x][y][4 * g + 1], acc[x][y][4 * g + 2], acc[x][y][4 * g + 3]};
                narrow4(v, reinterpret_cast<D*>(out + (lane & 31) * kPitch) + 32 * y + 8 * g + 4 * (lane >> 5));
            }
        wave_sync();
#pragma unroll
        for (int h = 0; h < 32 * kRowVecs / 64; ++h) {
            const int at = lane + 64 * h, row = at / kRowVecs, col = at % kRowVecs * kVec;
            const int64_t m = m0 + (wi * PX + x) * 32 + row, n = n0 + wj * 32 * QY + col;
            if (m >= p.a.rows || n >= p.b.rows) continue;
            const u32x4 v = *reinterpret_cast<const u32x4*>(out + row * kPitch + col * (int)sizeof(D));
            D* o = d + m * p.ldd + n;
            if (vec && n + kVec <= p.b.rows) {
                *reinterpret_cast<u32x4*>(o) = v;
            } else {
                union { u32x4 v; D e[kVec]; } u;
                u.v = v;
#pragma unroll
                for (int e = 0; e < kVec; ++e)
                    if (n + e < p.b.rows) o[e] = u.e[e];
            }
        }
    }
}

template <int WR, int WC, int PX, int QY, int S, int FA, int FB, bool EXACT, typename D>
__global__ __launch_bounds__(64 * WR * WC) void tile_kernel(F8Product p)
{
    using T = Tile<WR, WC, PX, QY, S>;
    extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
    const int64_t tiles_m = (p.a.rows + T::kRows - 1) / T::kRows, tiles_n = (p.b.rows + T::kCols - 1) / T::kCols;
    const int64_t part = blockIdx.x / (tiles_m * tiles_n);
    int64_t i, j;
    tile_at(xcd_part(blockIdx.x - part * (tiles_m * tiles_n), tiles_m * tiles_n), tiles_m, tiles_n, i, j);
    tile<WR, WC, PX, QY, S, FA, FB, EXACT, D>(p, lds, i * T::kRows, j * T::kCols, part);
}

// Tiles of 256 x 256, the first p.whole of them by one workgroup each; the others,
// which would leave CUs without one in the last round, by p.bands (2 or 4) workgroups
// of 128 or 64 rows.
template <int FA, int FB, typename D>
__global__ __launch_bounds__(512) void big_kernel(F8Product p)
{
    extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
    const int64_t tiles_m = (p.a.rows + 255) / 256, tiles_n = (p.b.rows + 255) / 256;
    int64_t i, j;
    if (blockIdx.x < p.whole) {
        tile_at(xcd_part(blockIdx.x, p.whole), tiles_m, tiles_n, i, j);
        tile<2, 4, 4, 2, 2, FA, FB, false, D>(p, lds, i * 256, j * 256, 0);
        return;
    }
    const int64_t u = xcd_part(blockIdx.x - p.whole, (tiles_m * tiles_n - p.whole) * p.bands);
    tile_at(p.whole + u / p.bands, tiles_m, tiles_n, i, j);
    const int64_t m0 = i * 256 + u % p.bands * (256 / p.bands);
    if (m0 >= p.a.rows) return;
    if (p.bands == 2) tile<2, 4, 2, 2, 3, FA, FB, false, D>(p, lds, m0, j * 256, 0);
    else tile<2, 4, 1, 2, 3, FA, FB, false, D>(p, lds, m0, j * 256, 0);
}

// D from the parts' sums, added in the parts' order: four columns a lane.
template <typename D>
__global__ __launch_bounds__(kThreads) void join_kernel(const float* __restrict__ sums, int parts, int64_t part_elems,
                                                        int64_t lds, int64_t rows, int64_t cols, D* __restrict__ d,
                                                        int64_t ldd, int vec)
{
    const int64_t per = (cols + 3) / 4, at = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (at >= rows * per) return;
    const int64_t m = at / per, n = at % per * 4;
    const float* s = sums + m * lds + n;   // (rows of sums are padded to whole quads)
    f32x4 v = *reinterpret_cast<const f32x4*>(s);
    for (int k = 1; k < parts; ++k) v += *reinterpret_cast<const f32x4*>(s + k * part_elems);
    D* o = d + m * ldd + n;
    if (vec && n + 4 <= cols) {
        narrow4(v, o);
    } else {
        D e[4];
        narrow4(v, e);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (n + j < cols) o[j] = e[j];
    }
}

// Few rows of A (at most AR): what counts is reading B once, at the rate of memory.  A
// workgroup takes 32 rows of B; its waves take the blocks of the summed axis in
// turn, each with a ring of R blocks in LDS of its own, so that nothing waits for
// another wave until they add up their sums at the end.
template <int NW, int R, int AR>
struct Thin {
    static constexpr int kBytesB = 32 * kLine, kBytesA = AR * kLine, kSlot = kBytesB + kBytesA + 256;
    static constexpr int kLoads = (32 + AR) / 8 + 1;
    static constexpr int kPitch = 36;                                  // floats of a row of sums in LDS
    static constexpr int kRing = NW * R * kSlot, kSums = NW * 32 * kPitch * 4;
    static constexpr int kLds = kRing > kSums ? kRing : kSums;
    static_assert(kLds <= 160 * 1024, "LDS of a CU");
};

__device__ __forceinline__ void load_256_at(const uint8_t* lane_base, uint32_t lds)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" : : "s"(lds), "v"(lane_base) : "memory");
}

template <typename T, int NW, int R, int AR, int FA, int FB, typename D>
__global__ __launch_bounds__(64 * NW) void thin_kernel(F8Product p)
{
    constexpr bool EXACT = sizeof(D) == 4;
    extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int64_t n0 = (int64_t)blockIdx.x * 32;
    const int last_a = (int)p.a.rows - 1, last_b = (int)(p.b.rows - 1 - n0 < 31 ? p.b.rows - 1 - n0 : 31);
    const int blocks = (int)((p.a.cols + kF8Block - 1) / kF8Block), mine = (blocks - wave + NW - 1) / NW;
    const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds + wave * R * T::kSlot;
    const uint8_t* const cb = p.b.codes + n0 * p.b.ld;
    uint32_t off_b[4], off_a[AR / 8];
#pragma unroll
    for (int l = 0; l < 4; ++l) {
        const int line = 8 * l + (lane >> 3);
        off_b[l] = (uint32_t)min(line, last_b) * (uint32_t)p.b.ld + 16 * ((lane & 7) ^ slot_key(line));
    }
#pragma unroll
    for (int l = 0; l < AR / 8; ++l) {
        const int line = 8 * l + (lane >> 3);
        off_a[l] = (uint32_t)min(line, last_a) * (uint32_t)p.a.ld + 16 * ((lane & 7) ^ slot_key(line));
    }
    // lanes 0-31: the scales of B's rows, 32-63: of A's
    const uint8_t* const scales = lane < 32
        ? p.b.scales + ((n0 + min(lane, last_b)) >> p.b.shift) * p.b.ld_scales
        : p.a.scales + ((int64_t)min(lane - 32, last_a) >> p.a.shift) * p.a.ld_scales;
    auto issue = [&](int i, int slot) {
        const int kb = wave + i * NW;
        const uint32_t at = lds0 + slot * T::kSlot;
#pragma unroll
        for (int l = 0; l < 4; ++l) load_1k(cb + (int64_t)kb * kF8Block, off_b[l], at + 1024 * l);
#pragma unroll
        for (int l = 0; l < AR / 8; ++l) load_1k(p.a.codes + (int64_t)kb * kF8Block, off_a[l], at + T::kBytesB + 1024 * l);
        load_256_at(scales + (kb & ~3), at + T::kBytesB + T::kBytesA);
    };
    f32x16 acc;
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[r] = 0.0f;
#pragma unroll
    for (int k = 0; k < R; ++k)
        if (k < mine) issue(k, k);
    const int row_a = (lane & 31) & (AR - 1);
    int slot = 0;
    for (int i = 0; i < mine; ++i) {
        if (i + R <= mine) stage_wait<(R - 1) * T::kLoads>();
        else stage_wait<0>();
        const uint8_t* b = lds + (wave * R + slot) * T::kSlot;
        const uint8_t* a = b + T::kBytesB;
        union Codes {
            u32x4 v[2];
            i32x8 f;
        } q[2], u[2];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int s = 4 * h + 2 * c + (lane >> 5);
                q[h].v[c] = *reinterpret_cast<const u32x4*>(b + (lane & 31) * kLine + 16 * (s ^ slot_key(lane & 31)));
                u[h].v[c] = *reinterpret_cast<const u32x4*>(a + row_a * kLine + 16 * (s ^ slot_key(row_a)));
            }
        const uint8_t* e = a + T::kBytesA + ((wave + i * NW) & 3);
        const int eq = e[4 * (lane & 31)], ep = e[4 * (32 + (lane & 31))];
        // the slot has been read: its next block may come
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        if (i + R < mine) issue(i + R, slot);
        slot = slot + 1 == R ? 0 : slot + 1;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if constexpr (EXACT) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const bf16x8 wq = widen8<FB>((uint32_t)q[h].f[2 * j], (uint32_t)q[h].f[2 * j + 1], power(eq));
                    const bf16x8 wp = widen8<FA>((uint32_t)u[h].f[2 * j], (uint32_t)u[h].f[2 * j + 1], power(ep));
                    acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(wq, wp, acc, 0, 0, 0);
                }
            } else {
                acc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(q[h].f, u[h].f, acc, FB, FA, 0, eq, 0, ep);
            }
        }
    }
    __syncthreads();   // the rings are free for the sums
    float* const sums = reinterpret_cast<float*>(lds);
    if ((lane & 31) <= last_a) {
#pragma unroll
        for (int g = 0; g < 4; ++g)
            *reinterpret_cast<f32x4*>(sums + (wave * 32 + (lane & 31)) * T::kPitch + 8 * g + 4 * (lane >> 5)) =
                f32x4{acc[4 * g], acc[4 * g + 1], acc[4 * g + 2], acc[4 * g + 3]};
    }
    __syncthreads();
    for (int at = threadIdx.x; at < 32 * (last_a + 1); at += 64 * NW) {
        const int m = at >> 5, n = at & 31;
        if (n > last_b) continue;
        float v = sums[m * T::kPitch + n];
#pragma unroll
        for (int w = 1; w < NW; ++w) v += sums[(w * 32 + m) * T::kPitch + n];
        static_cast<D*>(p.d)[m * p.ldd + n0 + n] = (D)v;
    }
}

// ------------------------------------------------------------------ launchers
template <int FA, int FB, bool EXACT, typename D, int WR, int WC, int PX, int QY, int S>
void launch_tile(const F8Product& p, hipStream_t s)
{
    using T = Tile<WR, WC, PX, QY, S>;
    const int64_t tiles = (p.a.rows + T::kRows - 1) / T::kRows * ((p.b.rows + T::kCols - 1) / T::kCols);
    const dim3 grid((uint32_t)(tiles * p.parts));
    if (p.parts == 1) {
        tile_kernel<WR, WC, PX, QY, S, FA, FB, EXACT, D><<<grid, dim3(T::kThr), T::kLds, s>>>(p);
        return;
    }
    F8Product q = p;
    q.d = p.sums;
    q.ldd = p.ld_sums;
    q.vec = 1;
    tile_kernel<WR, WC, PX, QY, S, FA, FB, EXACT, float><<<grid, dim3(T::kThr), T::kLds, s>>>(q);
    const int64_t quads = p.a.rows * ((p.b.rows + 3) / 4);
    join_kernel<D><<<dim3((uint32_t)((quads + kThreads - 1) / kThreads)), kThreads, 0, s>>>(
        p.sums, p.parts, p.part_elems, p.ld_sums, p.a.rows, p.b.rows, static_cast<D*>(p.d), p.ldd, p.vec);
}

template <int FA, int FB, typename D>
void launch_big(const F8Product& p, hipStream_t s)
{
    const int64_t n = (p.a.rows + 255) / 256 * ((p.b.rows + 255) / 256);
    constexpr int lds = Tile<2, 4, 2, 2, 3>::kLds;
    static_assert(lds >= Tile<2, 4, 4, 2, 2>::kLds && lds >= Tile<2, 4, 1, 2, 3>::kLds, "LDS of the largest of the three");
    big_kernel<FA, FB, D><<<dim3((uint32_t)(p.whole + (n - p.whole) * p.bands)), dim3(512), lds, s>>>(p);
}

template <int FA, int FB, typename D, int NW, int AR>
void launch_thin(const F8Product& p, hipStream_t s)
{
    constexpr int R = AR == 32 ? 2 : 3;   // two workgroups a CU
    using T = Thin<NW, R, AR>;
    thin_kernel<T, NW, R, AR, FA, FB, D><<<dim3((uint32_t)((p.b.rows + 31) / 32)), dim3(64 * NW), T::kLds, s>>>(p);
}

template <int FA, int FB, typename D>
void launch_kind(const F8Product& p, hipStream_t s)
{
    constexpr bool EXACT = sizeof(D) == 4;
    switch (p.kind) {
    case kF8Thin:
        if (p.a.rows <= 8) launch_thin<FA, FB, D, 4, 8>(p, s);
        else if (p.a.rows <= 16) launch_thin<FA, FB, D, 4, 16>(p, s);
        else launch_thin<FA, FB, D, 4, 32>(p, s);
        break;
    case kF8Tile64: launch_tile<FA, FB, EXACT, D, 2, 2, 1, 1, 4>(p, s); break;
    case kF8Tile128: launch_tile<FA, FB, EXACT, D, 2, 2, 2, 2, 2>(p, s); break;
    default:
        if constexpr (!EXACT) launch_big<FA, FB, D>(p, s);
    }
}

template <int FA, int FB>
void launch(const F8Product& p, hipStream_t s)
{
    if (p.f32) launch_kind<FA, FB, float>(p, s);
    else launch_kind<FA, FB, __bf16>(p, s);
}

}  // namespace

hipError_t launch_f8_product(const F8Product& p, hipStream_t s)
{
    if (p.a.e5m2) { if (p.b.e5m2) launch<1, 1>(p, s); else launch<1, 0>(p, s); }
    else          { if (p.b.e5m2) launch<0, 1>(p, s); else launch<0, 0>(p, s); }
    return hipGetLastError();
}

}  // namespace z1
