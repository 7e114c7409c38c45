// muon.hip -- the streaming kernels of the Muon step on gfx950: momentum over
// the W replicas' gradients, the sum of squares of u, and the update of the
// master with the bf16 parameter.
//
// All are HBM-bound (under one flop per byte).  A workgroup takes a tile of
// 512 quads (2048 elements) of one matrix; lane l handles quads l and 256 + l,
// so a wave's load covers one contiguous run of a row.  A quad is four
// neighbouring elements of one row: rows may start at any element (odd column
// counts, blocks cut out of wider matrices), because gfx950's vector loads and
// stores need no more than the element's alignment.  No load is conditional
// (the last quad of a row is loaded from a little earlier, a lane past the end
// loads row 0), so that a tile's loads are all in flight at once.  Matrices that are contiguous in all
// their arrays are one long row.
//
// Arithmetic: one binary32 operation at a time (no contraction), gradients
// summed in rank order as the reduce of the AdamW step does; sums of squares
// in fp64 over a fixed tree, so a rerun gives the same bits.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "muon.h"

#pragma clang fp contract(off)

namespace z1 {
namespace {

using namespace dev;

// Tiles [lo, hi) with a stride for this workgroup; split = 8 gives each XCD
// (workgroup b runs on XCD b % 8) one contiguous eighth.
struct Walk {
    int64_t lo, hi, step;
};

__device__ __forceinline__ Walk walk(int64_t n, int split)
{
    const int64_t G = gridDim.x, b = blockIdx.x;
    const int64_t nx = (split > 1 && G % split == 0) ? split : 1;
    const int64_t per = (n + nx - 1) / nx, lo = (b % nx) * per;
    return Walk{lo + b / nx, lo + per < n ? lo + per : n, G / nx};
}

// A lane's quad (see span4) and its row.  A lane past the matrix's end is given
// row 0, nothing of which it stores.
struct Quad {
    int64_t row, col;
    int skip;
};

template <bool SHORT>
__device__ __forceinline__ Quad quad_at(const MatDesc& d, const StreamTile& t, int lane_quad)
{
    int64_t row = 0, c;
    if (d.vrows == 1) {
        c = 4 * ((int64_t)t.idx * kQuadsPerTile + lane_quad);
    } else {   // qpr < 2^30 (cols < 2^31), so 32-bit division
        const uint32_t x = (uint32_t)t.q0 + (uint32_t)lane_quad, per = (uint32_t)d.qpr;
        const uint32_t r = x / per;
        row = (int64_t)t.row0 + r;
        c = 4 * (int64_t)(x - r * per);
    }
    const bool in = row < d.vrows;
    const Span4 s = span4<SHORT>(c, d.vcols, in);
    return Quad{in ? row : 0, s.col, s.skip};
}

// Fixed-order workgroup sum; the total is in thread 0.  `sh` alternates
// between two buffers from tile to tile, so one barrier a tile is enough.
__device__ __forceinline__ double tile_sum(double x, double* sh)
{
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) x += __shfl_xor(x, off, 64);
    if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = x;
    __syncthreads();
    return ((sh[0] + sh[1]) + sh[2]) + sh[3];
}

// The reduced gradient of the lane's two quads: slices added in rank order,
// the loads of up to eight slices in flight together; then the average.
template <bool SHORT, int N>
__device__ __forceinline__ void add_slices(const Reduce& r, int w0, const int64_t (&at)[2], const int (&skip)[2],
                                           float (&g)[2][4])
{
    if constexpr (SHORT) {
        for (int w = w0; w < w0 + N; ++w)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float x[4];
                load_quad<true>(r.gp.p[w] + at[h], skip[h], x);
#pragma unroll
                for (int j = 0; j < 4; ++j) g[h][j] = w == 0 ? x[j] : g[h][j] + x[j];
            }
    } else {
        u16x4 raw[N][2];
#pragma unroll
        for (int w = 0; w < N; ++w)
#pragma unroll
            for (int h = 0; h < 2; ++h) raw[w][h] = ld4(r.gp.p[w0 + w] + at[h]);
#pragma unroll
        for (int w = 0; w < N; ++w)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float x[4];
                widen4(raw[w][h], x);
#pragma unroll
                for (int j = 0; j < 4; ++j) g[h][j] = w == 0 && w0 == 0 ? x[j] : g[h][j] + x[j];
            }
    }
}

template <bool SHORT>
__device__ __forceinline__ void reduce_quads(const Reduce& r, const int64_t (&at)[2], const int (&skip)[2],
                                             float (&g)[2][4])
{
    int w = 0;
    for (; w + 8 <= r.W; w += 8) add_slices<SHORT, 8>(r, w, at, skip, g);
    if (w + 4 <= r.W) {
        add_slices<SHORT, 4>(r, w, at, skip, g);
        w += 4;
    }
    if (w + 2 <= r.W) {
        add_slices<SHORT, 2>(r, w, at, skip, g);
        w += 2;
    }
    if (w < r.W) add_slices<SHORT, 1>(r, w, at, skip, g);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float v = g[h][j];
            if (r.mode == kAvgMulPow2) v = v * r.inv_w;
            else if (r.mode == kAvgDiv) v = v / r.f_w;
            if (r.round_bf16) v = widen(bf16_rne(v));
            g[h][j] = v;
        }
}

// One tile of the momentum; returns the lane's sum of squares of u.
template <typename M, typename U, bool NORM, bool SHORT>
__device__ __forceinline__ double momentum_tile(const Reduce& r, const MatDesc& d, const StreamTile& tile, float mu,
                                                int nesterov, bool clip, float coef)
{
    Quad q[2];
    int64_t at[2], ga[2];
    int skip[2];
    float g[2][4], m[2][4], u[2][4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        q[h] = quad_at<SHORT>(d, tile, (int)threadIdx.x + h * kThreads);
        skip[h] = q[h].skip;
        at[h] = q[h].row * d.ld + q[h].col;
        ga[h] = d.shard_offset + at[h];
        load_quad<SHORT>(static_cast<const M*>(d.m) + at[h], skip[h], m[h]);
    }
    reduce_quads<SHORT>(r, ga, skip, g);
    double acc = 0.0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float gj = clip ? g[h][j] * coef : g[h][j];
            const float mj = mu * m[h][j] + gj;
            m[h][j] = mj;
            u[h][j] = nesterov ? gj + mu * mj : mj;
        }
        store_quad<SHORT>(static_cast<M*>(d.m) + at[h], skip[h], m[h]);
        store_quad<SHORT>(static_cast<U*>(d.u) + (q[h].row * d.ldu + q[h].col), skip[h], u[h]);
        if constexpr (NORM) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (owns<SHORT>(skip[h], j)) acc = fma((double)u[h][j], (double)u[h][j], acc);
        }
    }
    return acc;
}

// m = mu m + g; u = g + mu m (Nesterov) or m.  Moves 2W + 2 sizeof(m) +
// sizeof(u) bytes an element.
template <typename M, typename U, bool NORM>
__global__ __launch_bounds__(kThreads) void momentum_kernel(Reduce r, const MatDesc* __restrict__ mats,
                                                            const StreamTile* __restrict__ tiles, int n_tiles,
                                                            int nesterov, MuonArgs ma, MuonClip mc,
                                                            double* __restrict__ partials, int split)
{
    __shared__ NormInfo ni;
    __shared__ double sums[2][kThreads / 64];
    use_device_scalars(ma, &mc.max_norm);
    bool clip = false;
    float coef = 1.0f;
    if (mc.rank_sumsq) {   // the clip decision, as the AdamW update forms it
        if (threadIdx.x == 0) {
            double tot = 0.0;
            for (int q = 0; q < mc.n_ranks; ++q) tot = tot + mc.rank_sumsq[q];
            const double norm = sqrt(tot);
            const double c = mc.clip_eps ? mc.max_norm / (norm + 1e-6) : mc.max_norm / norm;
            const bool cl = mc.clip_eps ? (c < 1.0) : (norm > mc.max_norm);
            ni = NormInfo{tot, norm, cl ? (float)c : 1.0f, cl ? 1 : 0, (isnan(norm) || isinf(norm)) ? 1 : 0, 0};
            if (blockIdx.x == 0 && mc.info_out) *mc.info_out = ni;
        }
        __syncthreads();
        clip = ni.clip != 0;
        coef = ni.clip_coef;
    }
    const Walk wk = walk(n_tiles, split);
    int buf = 0;
    for (int64_t t = wk.lo; t < wk.hi; t += wk.step) {
        const StreamTile tile = tiles[t];
        const MatDesc& d = mats[tile.mat];
        const double acc = d.vcols >= 4 ? momentum_tile<M, U, NORM, false>(r, d, tile, ma.mu, nesterov, clip, coef)
                                        : momentum_tile<M, U, NORM, true>(r, d, tile, ma.mu, nesterov, clip, coef);
        if constexpr (NORM) {
            const double b = tile_sum(acc, sums[buf]);
            buf ^= 1;
            if (threadIdx.x == 0) partials[t] = b;
        }
    }
}

template <typename U, bool SHORT>
__device__ __forceinline__ double sumsq_tile(const MatDesc& d, const StreamTile& tile)
{
    float u[2][4];
    int skip[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const Quad q = quad_at<SHORT>(d, tile, (int)threadIdx.x + h * kThreads);
        skip[h] = q.skip;
        load_quad<SHORT>(static_cast<const U*>(d.u) + (q.row * d.ldu + q.col), q.skip, u[h]);
    }
    double acc = 0.0;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (owns<SHORT>(skip[h], j)) acc = fma((double)u[h][j], (double)u[h][j], acc);
    return acc;
}

template <typename U>
__global__ __launch_bounds__(kThreads) void u_sumsq_kernel(const MatDesc* __restrict__ mats,
                                                           const StreamTile* __restrict__ tiles, int n_tiles,
                                                           double* __restrict__ partials, int split)
{
    __shared__ double sums[2][kThreads / 64];
    const Walk wk = walk(n_tiles, split);
    int buf = 0;
    for (int64_t t = wk.lo; t < wk.hi; t += wk.step) {
        const StreamTile tile = tiles[t];
        const MatDesc& d = mats[tile.mat];
        const double acc = d.vcols >= 4 ? sumsq_tile<U, false>(d, tile) : sumsq_tile<U, true>(d, tile);
        const double b = tile_sum(acc, sums[buf]);
        buf ^= 1;
        if (threadIdx.x == 0) partials[t] = b;
    }
}

// One workgroup a matrix: the norm from its tiles' partials in a fixed order,
// and the scale the iteration starts with.
__global__ __launch_bounds__(kThreads) void ns_norms_kernel(const MatDesc* __restrict__ mats,
                                                            const double* __restrict__ partials, double eps,
                                                            NormRec* __restrict__ norms)
{
    __shared__ double sums[kThreads / 64];
    const MatDesc& d = mats[blockIdx.x];
    double a = 0.0;
    for (int i0 = threadIdx.x; i0 < d.n_tiles; i0 += 16 * kThreads) {   // 16 loads in flight
        double x[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) x[k] = i0 + k * kThreads < d.n_tiles ? partials[d.tile0 + i0 + k * kThreads] : 0.0;
#pragma unroll
        for (int k = 0; k < 16; ++k) a = a + x[k];
    }
    const double tot = tile_sum(a, sums);
    if (threadIdx.x == 0) {
        const double f = (double)kNsScale / (sqrt(tot) + eps);
        NormRec n;
        // a norm that is infinite, NaN, or zero with eps = 0: u / (norm + eps)
        // holds a NaN, and the iteration spreads it over the whole matrix
        if (!(f > 0.0) || isinf(f)) {
            n.r = __builtin_nanf("");
            n.e = 0;
        } else {
            n.e = ilogb(f);
            n.r = (float)ldexp(f, -n.e);
        }
        norms[blockIdx.x] = n;
    }
}

template <bool SHORT>
__device__ __forceinline__ void update_tile(const MatDesc& d, const StreamTile& tile, const MuonArgs& ma)
{
    const float eta = ma.lr * d.scale;
    Quad q[2];
    int64_t at[2];
    float p[2][4], o[2][4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        q[h] = quad_at<SHORT>(d, tile, (int)threadIdx.x + h * kThreads);
        at[h] = q[h].row * d.ld + q[h].col;
        load_quad<SHORT>(d.master + at[h], q[h].skip, p[h]);
        load_quad<SHORT>(d.o + (q[h].row * d.ldo + q[h].col), q[h].skip, o[h]);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int j = 0; j < 4; ++j) p[h][j] = muon_elem(p[h][j], o[h][j], eta, ma);
        store_quad<SHORT>(d.master + at[h], q[h].skip, p[h]);
        store_quad<SHORT>(d.param + at[h], q[h].skip, p[h]);
    }
}

// p = (p - eta o) delta, the bf16 parameter from the new p: 12 bytes an element.
__global__ __launch_bounds__(kThreads) void muon_update_kernel(const MatDesc* __restrict__ mats,
                                                               const StreamTile* __restrict__ tiles, int n_tiles,
                                                               MuonArgs ma, int split)
{
    use_device_scalars(ma, nullptr);
    const Walk wk = walk(n_tiles, split);
    for (int64_t t = wk.lo; t < wk.hi; t += wk.step) {
        const StreamTile tile = tiles[t];
        const MatDesc& d = mats[tile.mat];
        if (d.vcols >= 4) update_tile<false>(d, tile, ma);
        else update_tile<true>(d, tile, ma);
    }
}

}  // namespace

// ------------------------------------------------------------------ launchers
hipError_t launch_momentum(const Reduce& r, const MatDesc* mats, const StreamTile* tiles, int n_tiles, bool m_bf16,
                           bool u_f32, bool nesterov, const MuonArgs& ma, const MuonClip& mc, double* partials,
                           int nblocks, int split, hipStream_t s)
{
#define Z1_MOM(M, U, N)                                                                                          \
    momentum_kernel<M, U, N><<<dim3(nblocks), dim3(kThreads), 0, s>>>(r, mats, tiles, n_tiles, nesterov ? 1 : 0, \
                                                                      ma, mc, partials, split)
#define Z1_MOM_N(M, U)                  \
    do {                                \
        if (partials) Z1_MOM(M, U, true); \
        else Z1_MOM(M, U, false);       \
    } while (0)
    if (m_bf16) {
        if (u_f32) Z1_MOM_N(uint16_t, float);
        else Z1_MOM_N(uint16_t, uint16_t);
    } else {
        if (u_f32) Z1_MOM_N(float, float);
        else Z1_MOM_N(float, uint16_t);
    }
#undef Z1_MOM_N
#undef Z1_MOM
    return hipGetLastError();
}

hipError_t launch_u_sumsq(const MatDesc* mats, const StreamTile* tiles, int n_tiles, bool u_f32, double* partials,
                          int nblocks, int split, hipStream_t s)
{
    if (u_f32) u_sumsq_kernel<float><<<dim3(nblocks), dim3(kThreads), 0, s>>>(mats, tiles, n_tiles, partials, split);
    else u_sumsq_kernel<uint16_t><<<dim3(nblocks), dim3(kThreads), 0, s>>>(mats, tiles, n_tiles, partials, split);
    return hipGetLastError();
}

hipError_t launch_ns_norms(const MatDesc* mats, int n_mats, const double* partials, double eps, NormRec* norms,
                           hipStream_t s)
{
    ns_norms_kernel<<<dim3(n_mats), dim3(kThreads), 0, s>>>(mats, partials, eps, norms);
    return hipGetLastError();
}

hipError_t launch_muon_update(const MatDesc* mats, const StreamTile* tiles, int n_tiles, const MuonArgs& ma,
                              int nblocks, int split, hipStream_t s)
{
    muon_update_kernel<<<dim3(nblocks), dim3(kThreads), 0, s>>>(mats, tiles, n_tiles, ma, split);
    return hipGetLastError();
}

}  // namespace z1
