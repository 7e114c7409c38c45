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
// 0.02-0.2 % before its own rounding to bf16 (0.17 %).  A and B need one half:
// their roundings are multiplied by X, not added to it.
//
// The norm enters as a power of two 2^e, exact on the way into fp16, and a
// factor r in [1, 2) folded into the first step: X = r Xs / S.
//
// Operands are padded with zeros to multiples of 128, so no product checks
// bounds; a zero row stays zero through the iteration.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "muon.h"

namespace z1 {
namespace {

using namespace dev;

typedef _Float16 half_t;
typedef half_t h4 __attribute__((ext_vector_type(4)));
typedef half_t h8 __attribute__((ext_vector_type(8)));

constexpr int kT = kPad;           // tile side

__device__ __forceinline__ float to_f32(uint16_t h) { return widen(h); }
__device__ __forceinline__ float to_f32(float x) { return x; }

// ------------------------------------------------------------- prepare
// Xs = 2^e u as hi (and lo where u is fp32: a bf16 u fits hi exactly), u
// transposed if tall, zeros in the padding.  One workgroup a 128 x 128 tile;
// a tall u goes through LDS so that both sides are read and written by rows.
template <typename U>
__global__ __launch_bounds__(kThreads) void ns_prepare_kernel(NsArgs g)
{
    constexpr bool LO = sizeof(U) == 4;
    __shared__ float sh[kT / 2][kT + 1];
    const GroupDesc& gd = g.groups[g.group];
    if ((int)blockIdx.x >= gd.n_full) return;
    const ProdTile pt = g.list[gd.full0 + blockIdx.x];
    const MatDesc& d = g.mats[pt.mat];
    const int e = g.norms[pt.mat].e;
    const U* u = static_cast<const U*>(d.u);
    half_t* hi = reinterpret_cast<half_t*>(g.area + d.x[0]);
    half_t* lo = reinterpret_cast<half_t*>(g.area + d.lo);
    const int i0 = pt.i * kT, j0 = pt.j * kT;
    const int c = threadIdx.x & 63, r0 = threadIdx.x >> 6;
    auto put = [&](int i, int j, float x) {
        const int64_t at = (int64_t)i * d.np + j;
        const half_t h = (half_t)x;
        hi[at] = h;
        if constexpr (LO) lo[at] = (half_t)(x - (float)h);
    };
    if (!d.tall) {
        for (int r = r0; r < kT; r += 4)
            for (int cc = c; cc < kT; cc += 64) {
                const int i = i0 + r, j = j0 + cc;
                const bool in = i < d.k && j < d.n;
                put(i, j, in ? ldexpf(to_f32(u[(int64_t)i * d.ldu + j]), e) : 0.0f);
            }
    } else {
        for (int half = 0; half < 2; ++half) {   // rows of u = columns j of X
            const int jb = j0 + half * (kT / 2);
            for (int r = r0; r < kT / 2; r += 4)
                for (int cc = c; cc < kT; cc += 64) {
                    const int j = jb + r, i = i0 + cc;
                    const bool in = i < d.k && j < d.n;
                    sh[r][cc] = in ? ldexpf(to_f32(u[(int64_t)j * d.ldu + i]), e) : 0.0f;
                }
            __syncthreads();
            for (int r = r0; r < kT; r += 4) put(i0 + r, jb + c, sh[c][r]);
            __syncthreads();
        }
    }
}

// ------------------------------------------------------------- products
// C = P Q^T of a 128 x 128 tile, four waves of 64 x 64, 32 of the inner
// dimension at a time.  P and Q are read by rows along the inner dimension;
// QT: Q is given transposed (inner dimension by rows).  The operands of the
// MFMA are swapped, so that a lane holds four neighbouring columns of C:
// acc[x][y][r] = C[16 x + (lane & 15)][16 y + 4 (lane >> 4) + r].
constexpr int kInner = 32, kLdsRow = kInner + 8;

typedef half_t Stage[kT][kLdsRow];

template <bool QT>
__device__ __forceinline__ void product(const half_t* P, int64_t ldp, const half_t* Q, int64_t ldq, int inner,
                                        Stage* sp, Stage* sq, f32x4 (&acc)[4][4])
{
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int wi = (wave >> 1) * 64, wj = (wave & 1) * 64;
    h8 rp[2], rq[2];
    auto fetch = [&](int k0) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int ch = tid + h * kThreads;
            rp[h] = *reinterpret_cast<const h8*>(P + (int64_t)(ch >> 2) * ldp + k0 + (ch & 3) * 8);
            if constexpr (!QT) rq[h] = *reinterpret_cast<const h8*>(Q + (int64_t)(ch >> 2) * ldq + k0 + (ch & 3) * 8);
            else rq[h] = *reinterpret_cast<const h8*>(Q + (int64_t)(k0 + (ch >> 4)) * ldq + (ch & 15) * 8);
        }
    };
    auto stash = [&](int b) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int ch = tid + h * kThreads;
            *reinterpret_cast<h8*>(&sp[b][ch >> 2][(ch & 3) * 8]) = rp[h];
            if constexpr (!QT) *reinterpret_cast<h8*>(&sq[b][ch >> 2][(ch & 3) * 8]) = rq[h];
            else {
#pragma unroll
                for (int v = 0; v < 8; ++v) sq[b][(ch & 15) * 8 + v][ch >> 4] = rq[h][v];
            }
        }
    };
#pragma unroll
    for (int x = 0; x < 4; ++x)
#pragma unroll
        for (int y = 0; y < 4; ++y) acc[x][y] = f32x4{0, 0, 0, 0};
    fetch(0);
    stash(0);
    __syncthreads();
    int b = 0;
    for (int k0 = 0; k0 < inner; k0 += kInner, b ^= 1) {
        const bool more = k0 + kInner < inner;
        if (more) fetch(k0 + kInner);
        h8 p[4], q[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            p[x] = *reinterpret_cast<const h8*>(&sp[b][wi + 16 * x + (lane & 15)][(lane >> 4) * 8]);
            q[x] = *reinterpret_cast<const h8*>(&sq[b][wj + 16 * x + (lane & 15)][(lane >> 4) * 8]);
        }
#pragma unroll
        for (int x = 0; x < 4; ++x)
#pragma unroll
            for (int y = 0; y < 4; ++y)
                acc[x][y] = __builtin_amdgcn_mfma_f32_16x16x32_f16(q[y], p[x], acc[x][y], 0, 0, 0);
        if (more) stash(b ^ 1);
        __syncthreads();
    }
}

enum Op : int { kGram = 0, kPoly = 1 };

// A = X X^T or B = b A + c A A: the tiles of the upper triangle, each stored
// with its mirror image.
template <int OP>
__global__ __launch_bounds__(kThreads) void ns_sym_kernel(NsArgs g, int it)
{
    __shared__ Stage sp[2], sq[2];
    const GroupDesc& gd = g.groups[g.group];
    if ((int)blockIdx.x >= gd.n_sym) return;
    const ProdTile pt = g.list[gd.sym0 + blockIdx.x];
    const MatDesc& d = g.mats[pt.mat];
    const half_t* src = reinterpret_cast<const half_t*>(g.area + (OP == kGram ? d.x[it & 1] : d.a));
    half_t* dst = reinterpret_cast<half_t*>(g.area + (OP == kGram ? d.a : d.b));
    const int64_t lds = OP == kGram ? d.np : d.kp;
    f32x4 acc[4][4];
    product<false>(src + (int64_t)pt.i * kT * lds, lds, src + (int64_t)pt.j * kT * lds, lds, (int)lds, sp, sq, acc);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int bi = pt.i * kT + (wave >> 1) * 64 + (lane & 15), bj = pt.j * kT + (wave & 1) * 64 + (lane >> 4) * 4;
    const float r = it == 0 ? g.norms[pt.mat].r : 1.0f;
    const float f = OP == kGram ? r * r / kNsScale : g.c / kNsScale;
#pragma unroll
    for (int x = 0; x < 4; ++x)
#pragma unroll
        for (int y = 0; y < 4; ++y) {
            const int i = bi + 16 * x, j = bj + 16 * y;
            h4 v;
            h4 av{};
            if constexpr (OP == kPoly) av = *reinterpret_cast<const h4*>(src + (int64_t)i * d.kp + j);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float z = f * acc[x][y][q];
                if constexpr (OP == kPoly) z += g.b * (float)av[q];
                v[q] = (half_t)z;
            }
            *reinterpret_cast<h4*>(dst + (int64_t)i * d.kp + j) = v;
            if (pt.i != pt.j) {
#pragma unroll
                for (int q = 0; q < 4; ++q) dst[(int64_t)(j + q) * d.kp + i] = v[q];
            }
        }
}

// X <- a X + B X; the last step writes o as bf16, or updates the master and
// the parameter with it, instead of X.
template <int LAST>
__global__ __launch_bounds__(kThreads) void ns_apply_kernel(NsArgs g, int it, int has_lo, MuonArgs ma)
{
    __shared__ Stage sp[2], sq[2];
    const GroupDesc& gd = g.groups[g.group];
    if ((int)blockIdx.x >= gd.n_full) return;
    const ProdTile pt = g.list[gd.full0 + blockIdx.x];
    const MatDesc& d = g.mats[pt.mat];
    const half_t* xi = reinterpret_cast<const half_t*>(g.area + d.x[it & 1]);
    half_t* xo = reinterpret_cast<half_t*>(g.area + d.x[(it & 1) ^ 1]);
    half_t* lo = reinterpret_cast<half_t*>(g.area + d.lo);
    const half_t* bm = reinterpret_cast<const half_t*>(g.area + d.b);
    f32x4 acc[4][4];
    product<true>(bm + (int64_t)pt.i * kT * d.kp, d.kp, xi + pt.j * kT, d.np, d.kp, sp, sq, acc);
    if constexpr (LAST == kNsUpdate) use_device_scalars(ma, nullptr);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int bi = pt.i * kT + (wave >> 1) * 64 + (lane & 15), bj = pt.j * kT + (wave & 1) * 64 + (lane >> 4) * 4;
    const float r = it == 0 ? g.norms[pt.mat].r : 1.0f;
    const float fa = g.a * r, fb = r / kNsScale;
#pragma unroll
    for (int x = 0; x < 4; ++x)
#pragma unroll
        for (int y = 0; y < 4; ++y) {
            const int i = bi + 16 * x, j = bj + 16 * y;
            const int64_t at = (int64_t)i * d.np + j;
            const h4 xh = *reinterpret_cast<const h4*>(xi + at);
            h4 xl{};
            if (has_lo) xl = *reinterpret_cast<const h4*>(lo + at);
            h4 vh, vl;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float z = fa * ((float)xh[q] + (float)xl[q]) + fb * acc[x][y][q];
                if constexpr (LAST == kNsMid) {
                    vh[q] = (half_t)z;
                    vl[q] = (half_t)(z - (float)vh[q]);
                } else {
                    const int row = d.tall ? j + q : i, col = d.tall ? i : j + q;
                    if (row < d.rows && col < d.cols) {
                        const float o = z / kNsScale;
                        if constexpr (LAST == kNsWriteO) {
                            d.o[(int64_t)row * d.ldo + col] = bf16_rne(o);
                        } else {
                            const int64_t p = (int64_t)row * d.ld + col;
                            const float v = muon_elem(d.master[p], o, ma.lr * d.scale, ma);
                            d.master[p] = v;
                            d.param[p] = bf16_rne(v);
                        }
                    }
                }
            }
            if constexpr (LAST == kNsMid) {
                *reinterpret_cast<h4*>(xo + at) = vh;
                *reinterpret_cast<h4*>(lo + at) = vl;
            }
        }
}

}  // namespace

// ------------------------------------------------------------------ launchers
hipError_t launch_ns_prepare(const NsArgs& g, bool u_f32, int grid, hipStream_t s)
{
    if (u_f32) ns_prepare_kernel<float><<<dim3(grid), dim3(kThreads), 0, s>>>(g);
    else ns_prepare_kernel<uint16_t><<<dim3(grid), dim3(kThreads), 0, s>>>(g);
    return hipGetLastError();
}

hipError_t launch_ns_gram(const NsArgs& g, int it, int grid, hipStream_t s)
{
    ns_sym_kernel<kGram><<<dim3(grid), dim3(kThreads), 0, s>>>(g, it);
    return hipGetLastError();
}

hipError_t launch_ns_poly(const NsArgs& g, int grid, hipStream_t s)
{
    ns_sym_kernel<kPoly><<<dim3(grid), dim3(kThreads), 0, s>>>(g, 1);
    return hipGetLastError();
}

hipError_t launch_ns_apply(const NsArgs& g, int it, bool u_f32, NsLast last, const MuonArgs& ma, int grid,
                           hipStream_t s)
{
    const int has_lo = it > 0 || u_f32 ? 1 : 0;
    const dim3 gr(grid), bl(kThreads);
    if (last == kNsMid) ns_apply_kernel<kNsMid><<<gr, bl, 0, s>>>(g, it, has_lo, ma);
    else if (last == kNsWriteO) ns_apply_kernel<kNsWriteO><<<gr, bl, 0, s>>>(g, it, has_lo, ma);
    else ns_apply_kernel<kNsUpdate><<<gr, bl, 0, s>>>(g, it, has_lo, ma);
    return hipGetLastError();
}

}  // namespace z1
