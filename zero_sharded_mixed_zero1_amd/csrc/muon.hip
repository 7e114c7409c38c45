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
// loads row 0), so that a tile's loads are all in flight at once.  Matrices that
// are contiguous in all their arrays are one long row.
//
// Measured: momentum of 4 x 4096 x 4096 over 8 slices (26 bytes an element) 307 us,
// 5.7 TB/s; over 3 slices, 5 odd matrices of 1001 x 777 cut out of wider ones 13.8
// us; update of 4 x 4096 x 4096 (12 bytes) 142 us, 5.7 TB/s.  A single 64 x 64
// takes 9 us, nearly all of it a launch.  The momentum's 97 to 111 registers leave
// four workgroups a CU, 1024 on the chip: about 2000 tiles are two rounds, and of one
// slice with 16-bit m and u (8 bytes an element, 11008 x 4096) it reaches 3.9 TB/s.
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

// The reduced gradient of the lane's Q quads: slices added in rank order, the
// loads of N slices in flight together; then the average.
template <bool SHORT, int N, int Q>
__device__ __forceinline__ void add_slices(const Reduce& r, int w0, const int64_t (&at)[Q], const int (&skip)[Q],
                                           float (&g)[Q][4])
{
    if constexpr (SHORT) {
        for (int w = w0; w < w0 + N; ++w)
#pragma unroll
            for (int h = 0; h < Q; ++h) {
                float x[4];
                load_quad<true>(r.gp.p[w] + at[h], skip[h], x);
#pragma unroll
                for (int j = 0; j < 4; ++j) g[h][j] = w == 0 ? x[j] : g[h][j] + x[j];
            }
    } else {
        u16x4 raw[N][Q];
#pragma unroll
        for (int w = 0; w < N; ++w)
#pragma unroll
            for (int h = 0; h < Q; ++h) raw[w][h] = ld4(r.gp.p[w0 + w] + at[h]);
#pragma unroll
        for (int w = 0; w < N; ++w)
#pragma unroll
            for (int h = 0; h < Q; ++h) {
                float x[4];
                widen4(raw[w][h], x);
#pragma unroll
                for (int j = 0; j < 4; ++j) g[h][j] = w == 0 && w0 == 0 ? x[j] : g[h][j] + x[j];
            }
    }
}

template <bool SHORT, bool FEW, int Q>
__device__ __forceinline__ void reduce_quads(const Reduce& r, const int64_t (&at)[Q], const int (&skip)[Q],
                                             float (&g)[Q][4])
{
    int w = 0;
    if constexpr (!FEW) {
        for (; w + 8 <= r.W; w += 8) add_slices<SHORT, 8>(r, w, at, skip, g);
        if (w + 4 <= r.W) {
            add_slices<SHORT, 4>(r, w, at, skip, g);
            w += 4;
        }
    }
    if (w + 2 <= r.W) {
        add_slices<SHORT, 2>(r, w, at, skip, g);
        w += 2;
    }
    if (w < r.W) add_slices<SHORT, 1>(r, w, at, skip, g);
#pragma unroll
    for (int h = 0; h < Q; ++h)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float v = g[h][j];
            if (r.mode == kAvgMulPow2) v = v * r.inv_w;
            else if (r.mode == kAvgDiv) v = v / r.f_w;
            if (r.round_bf16) v = widen(bf16_rne(v));
            g[h][j] = v;
        }
}

struct MomentumArgs {
    float mu;
    int nesterov;
    bool clip;
    float coef;
};

// N tiles of the momentum together (d: their matrices); acc: the lane's sum of
// squares of u in each.
template <typename M, typename U, bool NORM, bool SHORT, bool FEW, int N>
__device__ __forceinline__ void momentum_tiles(const Reduce& r, const MatDesc* const (&d)[N], const StreamTile (&tile)[N],
                                               const MomentumArgs& a, double (&acc)[N])
{
    constexpr int Q = 2 * N;
    int64_t at[Q], ga[Q], ua[Q];
    int skip[Q];
    float g[Q][4], m[Q][4];
#pragma unroll
    for (int h = 0; h < Q; ++h) {
        const MatDesc& e = *d[h / 2];
        const Quad q = quad_at<SHORT>(e, tile[h / 2], (int)threadIdx.x + (h & 1) * kThreads);
        skip[h] = q.skip;
        at[h] = q.row * e.ld + q.col;
        ua[h] = q.row * e.ldu + q.col;
        ga[h] = e.shard_offset + at[h];
        load_quad<SHORT>(static_cast<const M*>(e.m) + at[h], skip[h], m[h]);
    }
    reduce_quads<SHORT, FEW>(r, ga, skip, g);
#pragma unroll
    for (int h = 0; h < Q; ++h) {
        const MatDesc& e = *d[h / 2];
        float u[4];
        if ((h & 1) == 0) acc[h / 2] = 0.0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float gj = a.clip ? g[h][j] * a.coef : g[h][j];
            const float mj = a.mu * m[h][j] + gj;
            m[h][j] = mj;
            u[j] = a.nesterov ? gj + a.mu * mj : mj;
        }
        store_quad<SHORT>(static_cast<M*>(e.m) + at[h], skip[h], m[h]);
        store_quad<SHORT>(static_cast<U*>(e.u) + ua[h], skip[h], u);
        if constexpr (NORM) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (owns<SHORT>(skip[h], j)) acc[h / 2] = fma((double)u[j], (double)u[j], acc[h / 2]);
        }
    }
}

// m = mu m + g; u = g + mu m (Nesterov) or m.  Moves 2W + 2 sizeof(m) +
// sizeof(u) bytes an element.  FEW: one or two slices, whose tiles are taken two
// at a time (a tile of them alone is too little in flight).
template <typename M, typename U, bool NORM, bool FEW>
__global__ __launch_bounds__(kThreads) void momentum_kernel(Reduce r, const MatDesc* __restrict__ mats,
                                                            const StreamTile* __restrict__ tiles, int n_tiles,
                                                            int nesterov, MuonArgs ma, MuonClip mc,
                                                            double* __restrict__ partials, int split)
{
    __shared__ NormInfo ni;
    constexpr int N = FEW ? 2 : 1;
    __shared__ double sums[2][N][kThreads / 64];
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
    const MomentumArgs a{ma.mu, nesterov, clip, coef};
    const Walk wk = walk(n_tiles, split);
    int buf = 0;
    for (int64_t t = wk.lo; t < wk.hi; t += N * wk.step) {
        StreamTile tile[N];
        const MatDesc* d[N];
        bool one = false, shorts = false;   // the second tile is missing; rows shorter than a quad
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const int64_t tk = t + k * wk.step;
            one = one || tk >= wk.hi;
            tile[k] = tiles[tk < wk.hi ? tk : t];
            d[k] = mats + tile[k].mat;
            shorts = shorts || d[k]->vcols < 4;
        }
        double acc[N];
        if (N > 1 && (one || shorts)) {
#pragma unroll
            for (int k = 0; k < N; ++k) {
                if (t + k * wk.step >= wk.hi) break;
                const MatDesc* dk[1] = {d[k]};
                const StreamTile tk[1] = {tile[k]};
                double ak[1];
                if (d[k]->vcols < 4) momentum_tiles<M, U, NORM, true, FEW, 1>(r, dk, tk, a, ak);
                else momentum_tiles<M, U, NORM, false, FEW, 1>(r, dk, tk, a, ak);
                acc[k] = ak[0];
            }
        } else if (shorts) {
            momentum_tiles<M, U, NORM, true, FEW, N>(r, d, tile, a, acc);
        } else {
            momentum_tiles<M, U, NORM, false, FEW, N>(r, d, tile, a, acc);
        }
        if constexpr (NORM) {
            tile_sums<N>(acc, sums[buf]);
            if (threadIdx.x < N && t + threadIdx.x * wk.step < wk.hi)
                partials[t + threadIdx.x * wk.step] = four(sums[buf][threadIdx.x]);
            buf ^= 1;
        }
    }
}

// Four tiles a round, so that 8 quads a lane are in flight: 2 of 4096 x 11008 in
// bf16 54 us (3.3 TB/s), 12 of 768 x 768 7.8 us.
template <typename U>
__global__ __launch_bounds__(kThreads) void u_sumsq_kernel(const MatDesc* __restrict__ mats,
                                                           const StreamTile* __restrict__ tiles, int n_tiles,
                                                           double* __restrict__ partials, int split)
{
    constexpr int N = kSumsqTiles;
    __shared__ double sums[2][N][kThreads / 64];
    const Walk wk = walk(n_tiles, split);
    int buf = 0;
    for (int64_t t = wk.lo; t < wk.hi; t += N * wk.step) {
        float u[N][2][4];
        int skip[N][2];
#pragma unroll
        for (int k = 0; k < N; ++k) {   // (these matrices are not thin: no row is short)
            const int64_t tk = t + k * wk.step;
            const StreamTile tile = tiles[tk < wk.hi ? tk : t];
            const MatDesc& d = mats[tile.mat];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const Quad q = quad_at<false>(d, tile, (int)threadIdx.x + h * kThreads);
                skip[k][h] = q.skip;
                load_quad<false, true>(static_cast<const U*>(d.u) + (q.row * d.ldu + q.col), q.skip, u[k][h]);
            }
        }
        double acc[N];
#pragma unroll
        for (int k = 0; k < N; ++k) {
            acc[k] = 0.0;
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (owns<false>(skip[k][h], j)) acc[k] = fma((double)u[k][h][j], (double)u[k][h][j], acc[k]);
        }
        tile_sums<N>(acc, sums[buf]);
        if (threadIdx.x < N && t + threadIdx.x * wk.step < wk.hi)
            partials[t + threadIdx.x * wk.step] = four(sums[buf][threadIdx.x]);
        buf ^= 1;
    }
}

// One workgroup a matrix.
__global__ __launch_bounds__(kThreads) void ns_norms_kernel(const MatDesc* __restrict__ mats,
                                                            const double* __restrict__ partials, double eps,
                                                            NormRec* __restrict__ norms)
{
    __shared__ double sums[1][kThreads / 64];
    const NormRec n = matrix_norm(mats[blockIdx.x], partials, eps, sums);
    if (threadIdx.x == 0) norms[blockIdx.x] = n;
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
    const int nv = nesterov ? 1 : 0;
#define Z1_MOM(M, U, N, F) \
    momentum_kernel<M, U, N, F><<<dim3(nblocks), dim3(kThreads), 0, s>>>(r, mats, tiles, n_tiles, nv, ma, mc, partials, split)
#define Z1_MOM_N(M, U)                                     \
    do {                                                   \
        if (r.W <= 2) {                                    \
            if (partials) Z1_MOM(M, U, true, true);        \
            else Z1_MOM(M, U, false, true);                \
        } else {                                           \
            if (partials) Z1_MOM(M, U, true, false);       \
            else Z1_MOM(M, U, false, false);               \
        }                                                  \
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
