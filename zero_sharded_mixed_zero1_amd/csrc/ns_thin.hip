// ns_thin.hip -- orthogonalisation of thin matrices (k = min(rows, cols) up to
// 128) on gfx950, in one to four launches a segment of steps (five default ones).
//
// A step multiplies X from the left by Q = a I + b A + c A A, a polynomial of
// A = X X^T, and A becomes Q A Q.  So the steps need X only through A, which is
// k x k: gram forms A once, poly runs all steps in one workgroup a matrix and
// keeps the product P = Q_m ... Q_1, apply forms P X.  X is read twice and
// written once, where the tiles of newton_schulz.hip read and write it every
// step (and would leave most of the chip idle: k <= 128 is one tile of A).
//
// Precision: A, B = b A + c A A, T = A Q and P are held in fp32 and multiplied
// as two fp16 halves (22 bits; hi hi, hi lo and lo hi).  What A is off from the
// true P X X^T P^T is multiplied by Q on both sides, so on directions that X
// hardly has it grows by a^2 a step, from 2^-22 of the largest eigenvalue to
// 5e-3 of it in the four steps before the fifth, where b A stands beside a.  So
// steps are taken in segments whose A has grown by at most 160^2 (five default
// steps), with X in fp32 between them and A formed anew.  (All steps at once: a
// sixth step is off by 0.1 to 0.7 %, an eighth by more.)  The products keep the
// order of their factors: taking Q A Q as Q Q A, or reading P or T transposed,
// is the same only for factors that commute exactly, and is off by up to 9e-3
// after five steps, where this is off by up to 2e-4 (2-norm, singular values 1/i);
// the worst spectrum found, five decades of them, by 9e-4, in eight steps by 2e-3.
//
// Measured, five steps: 64 x 64 20.5 us (one launch); 24 of 100 x 1000 79 us: gram
// 14, the parts' sum 5, poly 51, apply 13.
//
// Powers of two carried in fp16: X and A 2^12, B 2^10, P 2^3 (|A| <= 9,
// |B| <= 12, |P| <= 160 * 27, checked on the host).
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

constexpr float kQScale = 1024.0f, kPScale = 8.0f;

// Where a segment finds X: u, or (mid) the workspace's fp32 X, which carries S
// and is zero in its padding.
template <typename U>
struct Source {
    const U* p;
    int64_t ld, rows, cols;
    int tall;
};

template <typename U>
__device__ __forceinline__ Source<U> source(const NsArgs& g, const MatDesc& d, int mid)
{
    if (mid) return Source<U>{reinterpret_cast<const U*>(g.area + d.x[0]), d.np, d.k, d.np, 0};
    return Source<U>{static_cast<const U*>(d.u), d.ldu, d.rows, d.cols, d.tall};
}

// A workgroup's share of KP x C of X, columns [j0, j0 + C): a quad a lane and
// round, along j (wide) or along i (tall), zeros outside X.
template <int KP, int C>
struct Chunk {
    static constexpr int kRounds = KP * C / 4 / kThreads;
    float v[kRounds][4];

    static __device__ __forceinline__ int at_i(int tall, int h)
    {
        const int t = threadIdx.x + h * kThreads;
        return tall ? (t % (KP / 4)) * 4 : t / (C / 4);
    }
    static __device__ __forceinline__ int at_j(int tall, int h)
    {
        const int t = threadIdx.x + h * kThreads;
        return tall ? t / (KP / 4) : (t % (C / 4)) * 4;
    }

    template <bool SHORT, typename U>
    __device__ __forceinline__ void load_rows(const Source<U>& s, int64_t j0)
    {
#pragma unroll
        for (int h = 0; h < kRounds; ++h) {
            const int64_t i = at_i(s.tall, h), j = j0 + at_j(s.tall, h);
            const int64_t row = s.tall ? j : i, col = s.tall ? i : j;
            const bool in = row < s.rows;
            load_padded<SHORT>(s.p + (in ? row : 0) * s.ld, col, s.cols, in, v[h]);
        }
    }

    // (no quad of these columns crosses the end of a row; a lane's quads are of one
    // column and of rows a constant apart)
    template <typename U>
    __device__ __forceinline__ void load_whole(const Source<U>& s, int64_t j0)
    {
        const int64_t i = at_i(s.tall, 0), j = j0 + at_j(s.tall, 0);
        const int64_t row = s.tall ? j : i, col = s.tall ? i : j;
        const int64_t step = s.tall ? kThreads / (KP / 4) : kThreads / (C / 4);
        const int64_t left = col < s.cols ? s.rows - row : 0;   // rows from the lane's first on
        const U* p = s.p + row * s.ld + col;
        const int64_t apart = step * s.ld;
#pragma unroll
        for (int h = 0; h < kRounds; ++h) {
            const bool in = h * step < left;
            float x[4];
            load_quad<false>(in ? p : s.p, 0, x);
            p += apart;
#pragma unroll
            for (int q = 0; q < 4; ++q) v[h][q] = in ? x[q] : 0.0f;
        }
    }

    template <typename U>
    __device__ __forceinline__ void load(const Source<U>& s, int64_t j0)
    {
        if (s.cols < 4) load_rows<true>(s, j0);
        else if ((s.cols & 3) == 0 || (!s.tall && j0 + C <= s.cols)) load_whole(s, j0);
        else load_rows<false>(s, j0);
    }
};

struct HiLo {
    half_t hi, lo;
};

__device__ __forceinline__ HiLo split(float x)
{
    const half_t h = (half_t)x;
    return HiLo{h, (half_t)(x - (float)h)};
}

// ------------------------------------------------------------- gram
// The exponent of a sum of nothing but zeros: above every other, so that the least
// of several parts' exponents is that of a part which holds something (zeros are
// zeros at any exponent).
constexpr int kZeros = 1000;

// Partial sums of X X^T over `split` columns of X each, one workgroup a part,
// 64 columns at a time: G times 2^2e, with the power of two 2^e that brings the
// largest element so far to 2^13..2^14 (exact, so that neither squares of tiny
// u underflow nor those of huge u overflow); when a larger one comes, the sum
// is scaled down to it.  The next 64 columns are loaded while these are
// multiplied.
//
// The matrix cores round the sum after every 8 products, each time by up to 2^-24
// of it and, where all are alike, to the same side: a norm of 2^26 equal elements
// was off by 1.1e-3 when each part was one chain of fp32 additions.  So the
// registers go into the part's sum in memory every kRun times 64 columns (2^-14 of
// the sum in a run, 2^-24 a run); a part of up to 8192 columns does so at its end
// only.  What one chain takes: 1 of 64 x 200000 in bf16 225 us (230), 128 x 200000
// 393 (384), 400 of 64 x 1000 142 (141).
constexpr int kRun = 128;

template <typename U, int KP>
__device__ __forceinline__ void thin_gram(const NsArgs& g, const MatDesc& d, int part, int64_t c0, int mid)
{
    constexpr bool LO = sizeof(U) == 4;
    constexpr int N = KP / 32, ROW = 64 + 8;   // 16 x 16 tiles a wave and side; LDS row
    typedef Chunk<KP, 64> C;
    __shared__ half_t hi[KP][ROW], lo[LO ? KP : 1][ROW];
    __shared__ uint32_t top;
    const Source<U> src = source<U>(g, d, mid);
    const int64_t c1 = min((int64_t)d.n, c0 + d.split);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int wi = (wave >> 1) * (KP / 2), wj = (wave & 1) * (KP / 2);
    f32x4 acc[N][N];
#pragma unroll
    for (int x = 0; x < N; ++x)
#pragma unroll
        for (int y = 0; y < N; ++y) acc[x][y] = f32x4{0, 0, 0, 0};
    if (threadIdx.x == 0) top = 0;
    int e = mid ? 0 : kZeros, kept = kZeros;   // kept: the exponent of the sum in memory, of the runs before
    float* out = reinterpret_cast<float*>(g.area + d.a) + (int64_t)part * KP * KP;
    C x;
    x.load(src, c0);
    int left = kRun;     // of 64 columns, until the registers go to memory
    bool more = false;
    for (int64_t j0 = c0; j0 < c1; j0 += 64) {
        __syncthreads();   // top is set; hi and lo have been read
        if (!mid) {
            uint32_t m = 0;
#pragma unroll
            for (int h = 0; h < C::kRounds; ++h)
#pragma unroll
                for (int q = 0; q < 4; ++q) m = max(m, __float_as_uint(x.v[h][q]) & 0x7fffffffu);
#pragma unroll
            for (int off = 32; off > 0; off >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, off, 64));
            if (lane == 0) atomicMax(&top, m);   // a maximum of integers: any order
            __syncthreads();
            const uint32_t t = top;
            // (an infinity or a NaN makes the sum one, at any scale)
            const int en = t == 0 ? kZeros : t < 0x7f800000u ? 13 - ilogbf(__uint_as_float(t)) : min(e, 0);
            if (en != e && e != kZeros) {
                const float f = ldexpf(1.0f, max(2 * (en - e), -200));
#pragma unroll
                for (int a = 0; a < N; ++a)
#pragma unroll
                    for (int b = 0; b < N; ++b) acc[a][b] *= f;
            }
            e = en;
        }
        const int ex = e == kZeros ? 0 : e;
#pragma unroll
        for (int h = 0; h < C::kRounds; ++h) {
            const int i = C::at_i(src.tall, h), j = C::at_j(src.tall, h);
            HiLo s[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) s[q] = split(ldexpf(x.v[h][q], ex));
            if (!src.tall) {
                *reinterpret_cast<h4*>(&hi[i][j]) = h4{s[0].hi, s[1].hi, s[2].hi, s[3].hi};
                if constexpr (LO) *reinterpret_cast<h4*>(&lo[i][j]) = h4{s[0].lo, s[1].lo, s[2].lo, s[3].lo};
            } else {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    hi[i + q][j] = s[q].hi;
                    if constexpr (LO) lo[i + q][j] = s[q].lo;
                }
            }
        }
        __syncthreads();
        if (j0 + 64 < c1) x.load(src, j0 + 64);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int c = 32 * h + 8 * (lane >> 4), r = lane & 15;
            h8 ph[N], qh[N], pl[N], ql[N];
#pragma unroll
            for (int a = 0; a < N; ++a) {
                ph[a] = *reinterpret_cast<const h8*>(&hi[wi + 16 * a + r][c]);
                qh[a] = *reinterpret_cast<const h8*>(&hi[wj + 16 * a + r][c]);
                if constexpr (LO) {
                    pl[a] = *reinterpret_cast<const h8*>(&lo[wi + 16 * a + r][c]);
                    ql[a] = *reinterpret_cast<const h8*>(&lo[wj + 16 * a + r][c]);
                }
            }
#pragma unroll
            for (int a = 0; a < N; ++a)
#pragma unroll
                for (int b = 0; b < N; ++b) {
                    acc[a][b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(qh[b], ph[a], acc[a][b], 0, 0, 0);
                    if constexpr (LO) {
                        acc[a][b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(ql[b], ph[a], acc[a][b], 0, 0, 0);
                        acc[a][b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(qh[b], pl[a], acc[a][b], 0, 0, 0);
                    }
                }
        }
        if (__builtin_expect(j0 + 64 >= c1 || --left == 0, 0)) {
            // (one of several parts: the tiles on and above the diagonal, thin_sum mirrors
            // the sum; writing them all took 1.3 us more of 24 matrices of 100 x 1000)
            const float f = ldexpf(1.0f, max(2 * (e - kept), -200));
#pragma unroll
            for (int a = 0; a < N; ++a)
#pragma unroll
                for (int b = 0; b < N; ++b)
                    if (d.n_parts == 1 || wi + 16 * a <= wj + 16 * b) {
                        f32x4* at = reinterpret_cast<f32x4*>(out + (wi + 16 * a + (lane & 15)) * KP + wj + 16 * b +
                                                             4 * (lane >> 4));
                        if (more) acc[a][b] += f * *at;
                        *at = acc[a][b];
                        acc[a][b] = f32x4{0, 0, 0, 0};
                    }
            kept = e;
            left = kRun;
            more = true;
        }
    }
    if (threadIdx.x == 0) reinterpret_cast<int32_t*>(g.area + d.lo)[part] = e;
}

// (two waves a SIMD, which leaves 256 registers: without it the sums go back and
// forth between a lane's two kinds of them, 1 of 64 x 200000, fp32 u, 341 us, 303 with)
template <typename U, int KP>
__global__ __launch_bounds__(kThreads, 2) void thin_gram_kernel(NsArgs g, int mid)
{
    const ProdTile pt = g.sym[blockIdx.x];
    thin_gram<U, KP>(g, g.mats[pt.mat], pt.i, (int64_t)pt.j * 64, mid);
}

// Slot of the sum's exponent among the parts'.
constexpr int kSumExp = kThinMaxParts;

// The parts' sum into part 0, with the least of their exponents: a quad a lane,
// KP * KP / 4 lanes a matrix (one workgroup alone would read 64 KiB a part at
// k = 128: 2 to 3 us each).  Tiles of 16 x 16 above the diagonal are stored with
// their mirror images.
template <int KP>
__global__ __launch_bounds__(kThreads) void thin_sum_kernel(NsArgs g)
{
    constexpr int kPer = KP * KP / 4 / kThreads;   // workgroups a matrix
    const MatDesc& d = g.mats[g.first + (int)blockIdx.x / kPer];
    const int quad = ((int)blockIdx.x % kPer) * kThreads + threadIdx.x, i = quad / (KP / 4), j = quad % (KP / 4) * 4;
    if (d.n_parts == 1 || i / 16 > j / 16) return;
    f32x4* part = reinterpret_cast<f32x4*>(g.area + d.a) + quad;
    int32_t* exps = reinterpret_cast<int32_t*>(g.area + d.lo);
    int least = exps[0];
    for (int n = 1; n < d.n_parts; ++n) least = min(least, exps[n]);
    f32x4 sum = f32x4{0, 0, 0, 0};
#pragma unroll 8
    for (int n = 0; n < d.n_parts; ++n)
        sum += ldexpf(1.0f, max(2 * (least - exps[n]), -200)) * part[(int64_t)n * (KP * KP / 4)];
    *part = sum;
    if (i / 16 < j / 16) {
        float* mirror = reinterpret_cast<float*>(g.area + d.a) + j * KP + i;
#pragma unroll
        for (int q = 0; q < 4; ++q) mirror[q * KP] = sum[q];
    }
    if (quad == 0) exps[kSumExp] = least;
}

// ------------------------------------------------------------- poly
// The waves of the poly kernel: RW x CW of them, MI x NI tiles of 16 x 16 each.
// kOwnP: P has LDS of its own.
template <int KP>
struct Poly {
    static constexpr int RW = KP == 128 ? 4 : 2, CW = 2, MI = KP / 16 / RW, NI = KP / 16 / CW;
    // rows are 32 bytes more than a multiple of 128: neither eight lanes along
    // eight rows nor sixteen down four rows meet in a bank
    static constexpr int kThr = 64 * RW * CW, ROW = KP + 16;
    static constexpr bool kOwnP = KP < 128;
    typedef f32x4 Acc[MI][NI];
    typedef half_t Mat[2][KP][ROW];   // high and low halves
};

// acc = M N, or M N^T (NT), without the product of the low halves.  N is read
// along its rows for M N^T and down its columns for M N.  The operands of the
// next 32 of the inner dimension are read while these are multiplied.
template <int KP, bool NT>
__device__ __forceinline__ void multiply(const typename Poly<KP>::Mat& M, const typename Poly<KP>::Mat& N,
                                         typename Poly<KP>::Acc& acc)
{
    using T = Poly<KP>;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15;
    const int wi = (wave / T::CW) * 16 * T::MI, wj = (wave % T::CW) * 16 * T::NI;
#pragma unroll
    for (int x = 0; x < T::MI; ++x)
#pragma unroll
        for (int y = 0; y < T::NI; ++y) acc[x][y] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int k0 = 0; k0 < KP; k0 += 32) {
        const int c = k0 + 8 * (lane >> 4);
        h8 p[2][T::MI], q[2][T::NI];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int x = 0; x < T::MI; ++x) p[h][x] = *reinterpret_cast<const h8*>(&M[h][wi + 16 * x + r][c]);
#pragma unroll
            for (int y = 0; y < T::NI; ++y) {
                if constexpr (NT) {
                    q[h][y] = *reinterpret_cast<const h8*>(&N[h][wj + 16 * y + r][c]);
                } else {
                    typedef __attribute__((address_space(3))) s4 lds_s4;
                    union { s4 s[2]; h8 v; } both;
#pragma unroll
                    for (int z = 0; z < 2; ++z)
                        both.s[z] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                            (lds_s4*)&N[h][c + 4 * z + (r >> 2)][wj + 16 * y + 4 * (r & 3)]);
                    q[h][y] = both.v;
                }
            }
        }
#pragma unroll
        for (int ab = 0; ab < 3; ++ab)   // hi hi, hi lo, lo hi
#pragma unroll
            for (int x = 0; x < T::MI; ++x)
#pragma unroll
                for (int y = 0; y < T::NI; ++y)
                    acc[x][y] = __builtin_amdgcn_mfma_f32_16x16x32_f16(q[ab & 1][y], p[ab >> 1][x], acc[x][y], 0, 0, 0);
    }
    constexpr int kReads = 2 * (T::MI + (NT ? 1 : 2) * T::NI), kMfma = 3 * T::MI * T::NI;
    constexpr int kEach = kMfma / kReads > 0 ? kMfma / kReads : 1;
    __builtin_amdgcn_sched_group_barrier(0x100, kReads, 0);
#pragma unroll
    for (int k0 = 32; k0 < KP; k0 += 32)
#pragma unroll
        for (int i = 0; i < kReads; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x008, kEach, 0);
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        }
}

// f(x, y, i, j) for the lane's quads of an accumulator: [x][y] is row i,
// columns j..j+3.
template <int KP, typename F>
__device__ __forceinline__ void for_quads(F f)
{
    using T = Poly<KP>;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int wi = (wave / T::CW) * 16 * T::MI + (lane & 15), wj = (wave % T::CW) * 16 * T::NI + 4 * (lane >> 4);
#pragma unroll
    for (int x = 0; x < T::MI; ++x)
#pragma unroll
        for (int y = 0; y < T::NI; ++y) f(x, y, wi + 16 * x, wj + 16 * y);
}

// a x + b y.
__device__ __forceinline__ f32x4 axby(float a, const f32x4& x, float b, const f32x4& y)
{
    f32x4 z;
#pragma unroll
    for (int q = 0; q < 4; ++q) z[q] = fmaf(a, x[q], b * y[q]);
    return z;
}

// A quad as two halves to M[..][i][j..j+3].
template <int KP>
__device__ __forceinline__ void put(typename Poly<KP>::Mat& M, int i, int j, const f32x4& v)
{
    const h4 hi = __builtin_convertvector(v, h4);
    f32x4 rest;
#pragma unroll
    for (int q = 0; q < 4; ++q) rest[q] = fmaf(-1.0f, (float)hi[q], v[q]);   // (one instruction an element)
    *reinterpret_cast<h4*>(&M[0][i][j]) = hi;
    *reinterpret_cast<h4*>(&M[1][i][j]) = __builtin_convertvector(rest, h4);
}

// One workgroup a matrix: the norm (the trace of the sum is |u|^2), A from the
// sum, `steps` steps, and P as two fp16 halves.  The norm goes to
// `norms` for apply: S / (norm + eps) = 2^e r.
//
// A step multiplies by Q = a I + B: T = A Q = a A + A B, A <- Q T = a T + B T,
// P <- Q P = a P + B P, with A, T and P in registers (fp32) for the a-terms and
// in LDS as two halves for the products.
// Bound by the chain of products: at k = 128 each takes 3100 cycles of MFMA and as
// many of LDS reads on its one CU (9 us a step), at 64 mostly latency (2.5 us).
template <int KP>
__device__ __forceinline__ NormRec thin_poly(const NsArgs& g, const MatDesc& d, int mat, int mid, int steps, double eps,
                                             NormRec* norms)
{
    using T = Poly<KP>;
    __shared__ typename T::Mat A, B;
    __shared__ typename Poly<T::kOwnP ? KP : 16>::Mat own_p;   // (unused, and left out, where P shares A's)
    __shared__ double diag[KP];
    __shared__ NormRec nr;
    const float* part = reinterpret_cast<const float*>(g.area + d.a);
    const int ex = -2 * reinterpret_cast<const int32_t*>(g.area + d.lo)[d.n_parts > 1 ? kSumExp : 0];
    half_t* pm = reinterpret_cast<half_t*>(g.area + d.b);
    double f2;   // A is f2 times the sum, divided by its power of two
    if (!mid) {
        for (int t = threadIdx.x; t < KP; t += T::kThr) diag[t] = ldexp((double)part[t * KP + t], ex);
        __syncthreads();
        double tr = 0.0;
#pragma unroll 8
        for (int t = 0; t < KP; ++t) tr = tr + diag[t];
        const double f = (double)kNsScale / (sqrt(tr) + eps);
        if (threadIdx.x == 0) norms[mat] = nr = norm_rec(tr, eps);
        __syncthreads();
        f2 = tr > 0.0 ? f * f / kNsScale : 0.0;
    } else {
        if (threadIdx.x == 0) norms[mat] = nr = NormRec{1.0f, 0};
        __syncthreads();
        f2 = 1.0 / kNsScale;   // the parts carry S^2, A carries S
    }
    if (nr.r != nr.r) {   // u / (norm + eps) holds a NaN: so does all of o, by apply's factor
        for (int t = threadIdx.x; t < 2 * KP * KP; t += T::kThr) pm[t] = (half_t)0.0f;
        return nr;
    }
    typename T::Acc acc, a, t, p;
    const float w = (float)ldexp(f2, ex);
    for_quads<KP>([&](int x, int y, int i, int j) { a[x][y] = w * *reinterpret_cast<const f32x4*>(part + i * KP + j); });
    for_quads<KP>([&](int x, int y, int i, int j) { put<KP>(A, i, j, a[x][y]); });
    __syncthreads();
    const float qb = g.b * (kQScale / kNsScale), qc = g.c * (kQScale / (kNsScale * kNsScale)), inv = 1.0f / kQScale;
    for (int it = 0; it < steps; ++it) {
        const bool last = it + 1 == steps;
        multiply<KP, true>(A, A, acc);
        for_quads<KP>([&](int x, int y, int i, int j) {
            const f32x4 v = axby(qc, acc[x][y], qb, a[x][y]);
            put<KP>(B, i, j, v);
            if (it == 0) {   // P = a I + B
                p[x][y] = (kPScale * inv) * v;
#pragma unroll
                for (int q = 0; q < 4; ++q) p[x][y][q] += i == j + q ? g.a * kPScale : 0.0f;
            }
        });
        __syncthreads();
        if (!last) {
            multiply<KP, true>(A, B, acc);
            for_quads<KP>([&](int x, int y, int, int) { t[x][y] = axby(g.a, a[x][y], inv, acc[x][y]); });
        }
        if constexpr (T::kOwnP) {
            if (it > 0) {
                multiply<KP, false>(B, own_p, acc);
                for_quads<KP>([&](int x, int y, int, int) { p[x][y] = axby(g.a, p[x][y], inv, acc[x][y]); });
            }
            if (!last) {
                __syncthreads();
                for_quads<KP>([&](int x, int y, int i, int j) { put<KP>(own_p, i, j, p[x][y]); });
            }
        } else {
            if (it > 0) {
                __syncthreads();
                for_quads<KP>([&](int x, int y, int i, int j) { put<KP>(A, i, j, p[x][y]); });
                __syncthreads();
                multiply<KP, false>(B, A, acc);
                for_quads<KP>([&](int x, int y, int, int) { p[x][y] = axby(g.a, p[x][y], inv, acc[x][y]); });
            }
            if (!last) __syncthreads();
        }
        if (!last) {
            for_quads<KP>([&](int x, int y, int i, int j) { put<KP>(A, i, j, t[x][y]); });
            __syncthreads();
            multiply<KP, false>(B, A, acc);
            for_quads<KP>([&](int x, int y, int, int) { a[x][y] = axby(g.a, t[x][y], inv, acc[x][y]); });
            __syncthreads();
            for_quads<KP>([&](int x, int y, int i, int j) { put<KP>(A, i, j, a[x][y]); });
            __syncthreads();
        }
    }
    for_quads<KP>([&](int x, int y, int i, int j) {
        h4 h, l;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const HiLo s = split(p[x][y][q]);
            h[q] = s.hi;
            l[q] = s.lo;
        }
        *reinterpret_cast<h4*>(pm + i * KP + j) = h;
        *reinterpret_cast<h4*>(pm + KP * KP + i * KP + j) = l;
    });
    return nr;
}

template <int KP>
__global__ __launch_bounds__(Poly<KP>::kThr) void thin_poly_kernel(NsArgs g, int mid, int steps, double eps,
                                                                   NormRec* norms)
{
    const int mat = g.first + (int)blockIdx.x;
    thin_poly<KP>(g, g.mats[mat], mat, mid, steps, eps, norms);
}

// ------------------------------------------------------------- apply
// o, or the update with it, from a wave's accumulators: rows i0.. and columns
// j0.. of X; a lane holds four neighbouring columns, or rows (along_i).
template <int LAST, bool SHORT, int MI, int NI>
__device__ __forceinline__ void thin_finish(const MatDesc& d, const f32x4 (&acc)[MI][NI], float f, int i0, int64_t j0,
                                            bool along_i, const MuonArgs& ma)
{
    const int lane = threadIdx.x & 63, r = lane & 15, four = 4 * (lane >> 4);
    const float eta = ma.lr * d.scale;
    float v[MI][NI][4];
    int64_t row[MI][NI], col[MI][NI];
    int skip[MI][NI], shift[MI][NI];
#pragma unroll
    for (int x = 0; x < MI; ++x)
#pragma unroll
        for (int y = 0; y < NI; ++y) {
            const int64_t i = i0 + 16 * x + (along_i ? four : r), j = j0 + 16 * y + (along_i ? r : four);
            const int64_t rr = along_i ? j : i, cc = along_i ? i : j;
            const bool in = rr < d.rows;
            row[x][y] = in ? rr : 0;
            // the lane's elements are columns cc .. cc + 3 of o; those past its
            // end are dropped one by one (no lane holds the ones before cc)
            const int64_t left = d.cols - cc;
            skip[x][y] = !in || left <= 0 ? 0 : left >= 4 ? 4 : (int)left;
            col[x][y] = skip[x][y] == 4 ? cc : SHORT ? 0 : (skip[x][y] ? d.cols - 4 : 0);
            shift[x][y] = (int)(cc - col[x][y]);
            if constexpr (LAST == kNsUpdate)
                load_quad<SHORT>(d.master + row[x][y] * d.ld + col[x][y], SHORT ? -skip[x][y] : 0, v[x][y]);
        }
#pragma unroll
    for (int x = 0; x < MI; ++x)
#pragma unroll
        for (int y = 0; y < NI; ++y) {
            const int n = skip[x][y];
            float o[4], p[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) o[q] = acc[x][y][q] * f;
            if constexpr (LAST == kNsUpdate) {
#pragma unroll
                for (int q = 0; q < 4; ++q) {   // the master's element for o[q]
                    float y4 = v[x][y][q];
#pragma unroll
                    for (int k = 1; k < 4; ++k) y4 = shift[x][y] == k ? v[x][y][(q + k) & 3] : y4;
                    p[q] = muon_elem(y4, o[q], eta, ma);
                }
            }
            const int64_t at = row[x][y] * (LAST == kNsUpdate ? d.ld : d.ldo) + col[x][y] + (n < 4 ? shift[x][y] : 0);
            if constexpr (LAST == kNsUpdate) {
                if (n == 4) {
                    store_quad<false>(d.master + at, 0, p);
                    store_quad<false>(d.param + at, 0, p);
                } else if (n > 0) {
                    store_quad<true>(d.master + at, -n, p);
                    store_quad<true>(d.param + at, -n, p);
                }
            } else {
                if (n == 4) store_quad<false>(d.o + at, 0, o);
                else if (n > 0) store_quad<true>(d.o + at, -n, o);
            }
        }
}

// 64 columns of P X a workgroup.  P comes straight from memory (L2) into the
// MFMA's registers, X through LDS with its inner dimension (k) along rows.
template <typename U, int KP, int LAST>
__device__ __forceinline__ void thin_apply(const NsArgs& g, const MatDesc& d, NormRec nr, int64_t j0, int mid,
                                           const MuonArgs& ma)
{
    constexpr bool LO = sizeof(U) == 4;
    constexpr int RW = KP == 32 ? 2 : 4, CW = 4 / RW, MI = KP / 16 / RW, NI = 4 / CW, ROW = KP + 8;
    __shared__ half_t hi[64][ROW], lo[LO ? 64 : 1][ROW];
    const Source<U> src = source<U>(g, d, mid);
    Chunk<KP, 64> xs;
    xs.load(src, j0);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15;
    const int wi = (wave / CW) * 16 * MI, wj = (wave % CW) * 16 * NI;
    const half_t* pm = reinterpret_cast<const half_t*>(g.area + d.b);
    h8 ph[KP / 32][MI], pl[KP / 32][MI];
#pragma unroll
    for (int k = 0; k < KP / 32; ++k)
#pragma unroll
        for (int x = 0; x < MI; ++x) {
            const half_t* at = pm + (wi + 16 * x + r) * KP + 32 * k + 8 * (lane >> 4);
            ph[k][x] = *reinterpret_cast<const h8*>(at);
            pl[k][x] = *reinterpret_cast<const h8*>(at + KP * KP);
        }
#pragma unroll
    for (int h = 0; h < Chunk<KP, 64>::kRounds; ++h) {
        const int i = Chunk<KP, 64>::at_i(src.tall, h), j = Chunk<KP, 64>::at_j(src.tall, h);
        HiLo s[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) s[q] = split(ldexpf(xs.v[h][q], nr.e));
        if (src.tall) {
            *reinterpret_cast<h4*>(&hi[j][i]) = h4{s[0].hi, s[1].hi, s[2].hi, s[3].hi};
            if constexpr (LO) *reinterpret_cast<h4*>(&lo[j][i]) = h4{s[0].lo, s[1].lo, s[2].lo, s[3].lo};
        } else {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                hi[j + q][i] = s[q].hi;
                if constexpr (LO) lo[j + q][i] = s[q].lo;
            }
        }
    }
    __syncthreads();
    // o's rows are X's columns when u is tall: then the lane's four elements
    // are to be four neighbouring rows of X
    const bool along_i = LAST != kNsMid && d.tall;
    f32x4 acc[MI][NI];
#pragma unroll
    for (int x = 0; x < MI; ++x)
#pragma unroll
        for (int y = 0; y < NI; ++y) acc[x][y] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int k = 0; k < KP / 32; ++k) {
        const int c = 32 * k + 8 * (lane >> 4);
        h8 xh[NI], xl[NI];
#pragma unroll
        for (int y = 0; y < NI; ++y) {
            xh[y] = *reinterpret_cast<const h8*>(&hi[wj + 16 * y + r][c]);
            if constexpr (LO) xl[y] = *reinterpret_cast<const h8*>(&lo[wj + 16 * y + r][c]);
        }
        auto add = [&](f32x4& a, h8 p, h8 v) {
            a = along_i ? __builtin_amdgcn_mfma_f32_16x16x32_f16(p, v, a, 0, 0, 0)
                        : __builtin_amdgcn_mfma_f32_16x16x32_f16(v, p, a, 0, 0, 0);
        };
#pragma unroll
        for (int x = 0; x < MI; ++x)
#pragma unroll
            for (int y = 0; y < NI; ++y) {
                add(acc[x][y], ph[k][x], xh[y]);
                add(acc[x][y], pl[k][x], xh[y]);
                if constexpr (LO) add(acc[x][y], ph[k][x], xl[y]);
            }
    }
    const float f = nr.r * (LAST == kNsMid ? 1.0f / kPScale : 1.0f / (kPScale * kNsScale));
    if constexpr (LAST == kNsMid) {
#pragma unroll
        for (int x = 0; x < MI; ++x)
#pragma unroll
            for (int y = 0; y < NI; ++y) {
                // (np is a multiple of 64: the row has room, its padding gets zeros)
                const int i = wi + 16 * x + r;
                const int64_t j = j0 + wj + 16 * y + 4 * (lane >> 4);
                if (i < d.k) st4(reinterpret_cast<float*>(g.area + d.x[0]) + i * (int64_t)d.np + j, acc[x][y] * f);
            }
    } else {
        if (d.cols >= 4) thin_finish<LAST, false>(d, acc, f, wi, j0 + wj, along_i, ma);
        else thin_finish<LAST, true>(d, acc, f, wi, j0 + wj, along_i, ma);
    }
}

template <typename U, int KP, int LAST>
__global__ __launch_bounds__(kThreads) void thin_apply_kernel(NsArgs g, int mid, MuonArgs ma)
{
    if constexpr (LAST == kNsUpdate) use_device_scalars(ma, nullptr);
    const ProdTile pt = g.full[blockIdx.x];
    thin_apply<U, KP, LAST>(g, g.mats[pt.mat], g.norms[pt.mat], (int64_t)pt.j * 64, mid, ma);
}

// All three for a matrix of one part, where a launch costs more than the work:
// 64 x 64 takes 20.5 us this way and 25 in three launches.  What passes between them goes
// through memory as it does there (the workgroup's own L1).
template <typename U, int KP, int LAST>
__global__ __launch_bounds__(kThreads) void thin_one_kernel(NsArgs g, int steps, double eps, NormRec* norms, MuonArgs ma)
{
    static_assert(Poly<KP>::kThr == kThreads, "one workgroup shape");
    if constexpr (LAST == kNsUpdate) use_device_scalars(ma, nullptr);
    const int mat = g.first + (int)blockIdx.x;
    const MatDesc& d = g.mats[mat];
    thin_gram<U, KP>(g, d, 0, 0, 0);
    __syncthreads();
    const NormRec nr = thin_poly<KP>(g, d, mat, 0, steps, eps, norms);
    __syncthreads();
    for (int64_t j0 = 0; j0 < d.n; j0 += 64) {
        thin_apply<U, KP, LAST>(g, d, nr, j0, 0, ma);
        __syncthreads();
    }
}

}  // namespace

// ------------------------------------------------------------------ launchers
#define Z1_KP(kp, CALL)           \
    do {                          \
        if ((kp) == 32) CALL(32);  \
        else if ((kp) == 64) CALL(64); \
        else CALL(128);           \
    } while (0)

hipError_t launch_thin_gram(const NsArgs& g, int kp, bool f32, int mid, int grid, hipStream_t s)
{
#define Z1_CALL(KP)                                                                                     \
    do {                                                                                                \
        if (f32) thin_gram_kernel<float, KP><<<dim3(grid), dim3(kThreads), 0, s>>>(g, mid);             \
        else thin_gram_kernel<uint16_t, KP><<<dim3(grid), dim3(kThreads), 0, s>>>(g, mid);              \
    } while (0)
    Z1_KP(kp, Z1_CALL);
#undef Z1_CALL
    return hipGetLastError();
}

hipError_t launch_thin_poly(const NsArgs& g, int kp, int mid, int steps, double eps, NormRec* norms, int grid,
                            hipStream_t s)
{
#define Z1_CALL(KP) thin_poly_kernel<KP><<<dim3(grid), dim3(Poly<KP>::kThr), 0, s>>>(g, mid, steps, eps, norms)
    Z1_KP(kp, Z1_CALL);
#undef Z1_CALL
    return hipGetLastError();
}

hipError_t launch_thin_sum(const NsArgs& g, int kp, int n_mats, hipStream_t s)
{
#define Z1_CALL(KP) thin_sum_kernel<KP><<<dim3(n_mats * (KP * KP / 4 / kThreads)), dim3(kThreads), 0, s>>>(g)
    Z1_KP(kp, Z1_CALL);
#undef Z1_CALL
    return hipGetLastError();
}

hipError_t launch_thin_one(const NsArgs& g, int kp, bool f32, int steps, double eps, NormRec* norms, NsLast last,
                           const MuonArgs& ma, int n_mats, hipStream_t s)
{
#define Z1_ONE(U, KP, LAST) thin_one_kernel<U, KP, LAST><<<dim3(n_mats), dim3(kThreads), 0, s>>>(g, steps, eps, norms, ma)
#define Z1_TYPE(KP, LAST)                      \
    do {                                       \
        if (f32) Z1_ONE(float, KP, LAST);      \
        else Z1_ONE(uint16_t, KP, LAST);       \
    } while (0)
    if (kp == 32) {
        if (last == kNsWriteO) Z1_TYPE(32, kNsWriteO);
        else Z1_TYPE(32, kNsUpdate);
    } else {
        if (last == kNsWriteO) Z1_TYPE(64, kNsWriteO);
        else Z1_TYPE(64, kNsUpdate);
    }
#undef Z1_TYPE
#undef Z1_ONE
    return hipGetLastError();
}

hipError_t launch_thin_apply(const NsArgs& g, int kp, bool f32, int mid, NsLast last, const MuonArgs& ma, int grid,
                             hipStream_t s)
{
#define Z1_LAST(U, KP)                                                                                          \
    do {                                                                                                        \
        const dim3 gr(grid), bl(kThreads);                                                                      \
        if (last == kNsMid) thin_apply_kernel<U, KP, kNsMid><<<gr, bl, 0, s>>>(g, mid, ma);                     \
        else if (last == kNsWriteO) thin_apply_kernel<U, KP, kNsWriteO><<<gr, bl, 0, s>>>(g, mid, ma);          \
        else thin_apply_kernel<U, KP, kNsUpdate><<<gr, bl, 0, s>>>(g, mid, ma);                                 \
    } while (0)
#define Z1_CALL(KP)                         \
    do {                                    \
        if (f32) Z1_LAST(float, KP);        \
        else Z1_LAST(uint16_t, KP);         \
    } while (0)
    Z1_KP(kp, Z1_CALL);
#undef Z1_CALL
#undef Z1_LAST
    return hipGetLastError();
}
#undef Z1_KP

}  // namespace z1
