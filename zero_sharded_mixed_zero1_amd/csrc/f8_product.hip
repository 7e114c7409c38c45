// f8_product.hip -- D = A B^T of matrices in 8-bit floating point with a power of
// two for each block of 128 (f8.h) on gfx950's matrix cores.
//
// Into bf16: v_mfma_scale_f32_32x32x64_f8f6f4 multiplies 32 x 64 codes by 32 x 64 and
// takes a scale for each operand's row, so two instructions are one block of 128,
// scales included.  It adds groups of eight products after aligning them to the
// group's largest, and what lies below 2^-13 of that is dropped (found by adding
// powers of two; beyond the groups sums keep fp32's 24 bits): 1e-5 to 6e-5 of the
// result on random operands, a hundredth of bf16's own rounding.
// Into fp32 that would be the largest error there is, so codes are widened to bf16
// with their scales (each exactly) and multiplied as bf16, which adds to
// 24 bits (7e-8), at half the rate.
//
// The operands are swapped (B's rows first), so that a lane holds four neighbouring
// columns of D: acc[x][y][r] = D[32 x + (lane & 31)][32 y + 8 (r >> 2) + 4 (lane >>
// 5) + (r & 3)].
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

// Tiles of D in an order that keeps what an XCD works on at once (workgroup b runs on
// XCD b % 8) close to a square: each XCD takes one contiguous eighth of the tiles
// in bands of 8 tile rows, down a band's columns first.
__device__ __forceinline__ void tile_at(int64_t b, int64_t tiles_m, int64_t tiles_n, int64_t& i, int64_t& j)
{
    const int64_t n = tiles_m * tiles_n, q = n / 8, rest = n % 8, x = b % 8;
    const int64_t t = x * q + (x < rest ? x : rest) + b / 8;
    const int64_t band = t / (8 * tiles_n), high = tiles_m - band * 8 < 8 ? tiles_m - band * 8 : 8, in = t - band * 8 * tiles_n;
    i = band * 8 + in % high;
    j = in / high;
}

// EXACT: widened to bf16 (D fp32).
template <typename T, int WR, int WC, int PX, int QY, int S, int FA, int FB, typename D>
__global__ __launch_bounds__(64 * WR * WC) void tile_kernel(F8Product p)
{
    constexpr bool EXACT = sizeof(D) == 4;
    extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int wi = wave / WC, wj = wave % WC;
    int64_t ti, tj;
    tile_at(blockIdx.x, (p.a.rows + T::kRows - 1) / T::kRows, (p.b.rows + T::kCols - 1) / T::kCols, ti, tj);
    const int64_t m0 = ti * T::kRows, n0 = tj * T::kCols;
    const int steps = (int)((p.a.cols + kF8Block - 1) / kF8Block);

    // what this wave loads: lines of 128 bytes (A's rows, then B's), eight a load,
    // their 16-byte slots permuted on the way; then 64 rows' scales of four blocks.
    // Rows past the end repeat the last one.
    const uint8_t* const ca = p.a.codes + m0 * p.a.ld;
    const uint8_t* const cb = p.b.codes + n0 * p.b.ld;
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
    auto issue = [&](int kb, int buf) {
        const uint32_t at = lds0 + buf * T::kStage;
#pragma unroll
        for (int l = 0; l < T::kLoads; ++l) {
            const int first = (wave * T::kLoads + l) * 8;
            load_1k((first < T::kRows ? ca : cb) + (int64_t)kb * kF8Block, off[l], at + first * kLine);
        }
#pragma unroll
        for (int l = 0; l < T::kScaleLoads; ++l) {
            const int first = min(wave * T::kScaleLoads + l, T::kLines / 64 - 1) * 64;
            load_256((first < T::kRows ? sa : sb) + (kb & ~3), soff[l], at + T::kLines * kLine + first * 4);
        }
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
    struct Frag {
        Codes p[PX], q[QY];
    };
    int ep[PX], eq[QY];
    auto read = [&](Frag& f, int buf, int h) {
        const uint8_t* a = lds + buf * T::kStage + wi * 32 * PX * kLine;
        const uint8_t* b = lds + buf * T::kStage + (T::kRows + wj * 32 * QY) * kLine;
#pragma unroll
        for (int y = 0; y < QY; ++y)
#pragma unroll
            for (int c = 0; c < 2; ++c) f.q[y].v[c] = *reinterpret_cast<const u32x4*>(b + y * 32 * kLine + place[h][c]);
#pragma unroll
        for (int x = 0; x < PX; ++x)
#pragma unroll
            for (int c = 0; c < 2; ++c) f.p[x].v[c] = *reinterpret_cast<const u32x4*>(a + x * 32 * kLine + place[h][c]);
    };
    auto read_scales = [&](int buf, int kb) {
        const uint8_t* e = lds + buf * T::kStage + T::kLines * kLine + (kb & 3) + 4 * (lane & 31);
#pragma unroll
        for (int x = 0; x < PX; ++x) ep[x] = e[4 * (wi * 32 * PX + 32 * x)];
#pragma unroll
        for (int y = 0; y < QY; ++y) eq[y] = e[4 * (T::kRows + wj * 32 * QY + 32 * y)];
    };
    auto multiply = [&](const Frag& f) {
        if constexpr (!EXACT) {
#pragma unroll
            for (int x = 0; x < PX; ++x)
#pragma unroll
                for (int y = 0; y < QY; ++y)
                    acc[x][y] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(f.q[y].f, f.p[x].f, acc[x][y], FB, FA, 0, eq[y], 0, ep[x]);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                bf16x8 wp[PX], wq[QY];
#pragma unroll
                for (int x = 0; x < PX; ++x) wp[x] = widen8<FA>((uint32_t)f.p[x].f[2 * j], (uint32_t)f.p[x].f[2 * j + 1], power(ep[x]));
#pragma unroll
                for (int y = 0; y < QY; ++y) wq[y] = widen8<FB>((uint32_t)f.q[y].f[2 * j], (uint32_t)f.q[y].f[2 * j + 1], power(eq[y]));
#pragma unroll
                for (int x = 0; x < PX; ++x)
#pragma unroll
                    for (int y = 0; y < QY; ++y) acc[x][y] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(wq[y], wp[x], acc[x][y], 0, 0, 0);
            }
        }
    };
    // the order that a half is scheduled in: its MFMAs with the LDS reads of the
    // next spread between them
    auto spread = [] {
        if constexpr (!EXACT) {
            constexpr int kMfma = PX * QY, kReads = 2 * (PX + QY), kEach = (kReads + kMfma - 1) / kMfma;
#pragma unroll
            for (int i = 0; i < kMfma; ++i) {
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x100, kEach, 0);
            }
        }
    };

    // each half's operands are read from LDS while the half before is multiplied;
    // the barrier lies between the halves, when this wave's reads of stage t are
    // done and its loads of stage t + 1 have arrived
    int put = 0, get = 0;   // buffers: the next one to load into, the one to read
    auto next = [](int b) { return b + 1 == S ? 0 : b + 1; };
#pragma unroll
    for (int k = 0; k < S; ++k)
        if (k < steps) {
            issue(k, put);
            put = next(put);
        }
    if (steps > 0) {
        Frag f0, f1;
        if (steps > S - 1) stage_wait<(S - 1) * T::kInFlight>();
        else stage_wait<0>();
        __syncthreads();
        read(f0, get, 0);
        read_scales(get, 0);
        for (int t = 0; t < steps; ++t) {
            read(f1, get, 1);
            multiply(f0);
            spread();
            if (t + 1 < steps) {
                if (t + S - 1 < steps) stage_wait<(S - 2) * T::kInFlight>();   // stages t + 2 .. t + S - 1 may be under way
                else stage_wait<0>();
                __syncthreads();
                if (t + S < steps) {
                    issue(t + S, put);
                    put = next(put);
                }
                get = next(get);
            }
            // (the last round reads the last stage again: the loop stays one block)
            read(f0, get, 0);
            multiply(f1);
            spread();
            read_scales(get, t + 1 < steps ? t + 1 : t);
        }
    }
    __syncthreads();   // the stages are free for the way out

    // 32 rows of the wave at a time through LDS, to leave as whole rows
    constexpr int kVec = 16 / (int)sizeof(D), kRowVecs = 32 * QY / kVec, kPitch = T::kPitch / 4 * (int)sizeof(D) + (sizeof(D) == 2 ? 8 : 0);
    static_assert(kPitch % 16 == 0, "rows in LDS begin at 16 bytes");
    uint8_t* out = lds + wave * 32 * T::kPitch;
    D* const d = static_cast<D*>(p.d);
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

template <int FA, int FB, typename D, int WR, int WC, int PX, int QY, int S>
void launch_tile(const F8Product& p, hipStream_t s)
{
    using T = Tile<WR, WC, PX, QY, S>;
    const int64_t grid = (p.a.rows + T::kRows - 1) / T::kRows * ((p.b.rows + T::kCols - 1) / T::kCols);
    tile_kernel<T, WR, WC, PX, QY, S, FA, FB, D><<<dim3((uint32_t)grid), dim3(T::kThr), T::kLds, s>>>(p);
}

template <int FA, int FB>
void launch(const F8Product& p, hipStream_t s)
{
    if (p.f32) launch_tile<FA, FB, float, 2, 2, 2, 2, 2>(p, s);
    else if (p.a.rows > 1024) launch_tile<FA, FB, __bf16, 2, 2, 4, 4, 2>(p, s);
    else launch_tile<FA, FB, __bf16, 2, 2, 2, 2, 2>(p, s);
}

}  // namespace

hipError_t launch_f8_product(const F8Product& p, hipStream_t s)
{
    if (p.a.e5m2) { if (p.b.e5m2) launch<1, 1>(p, s); else launch<1, 0>(p, s); }
    else          { if (p.b.e5m2) launch<0, 1>(p, s); else launch<0, 0>(p, s); }
    return hipGetLastError();
}

}  // namespace z1
