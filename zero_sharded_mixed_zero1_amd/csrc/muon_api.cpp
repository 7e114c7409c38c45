// muon_api.cpp -- the Muon entry points of the C ABI (declared in
// include/zero1.h): argument checks, the plan over a rank's matrices (tiles of
// the streaming kernels and of the products, groups, workspace layout) and the
// launch sequences.  No entry point allocates device memory or synchronizes
// (except zero1_muon_plan, which copies its table once, and
// ZERO1_SYNC_CHECK=1).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <exception>
#include <mutex>
#include <utility>
#include <vector>

#include "../../include/zero1.h"
#include "internal.h"
#include "muon.h"

using namespace z1;

static_assert(sizeof(MuonScal) == sizeof(zero1_muon_scalars) && sizeof(MuonScal) == 24 &&
                  offsetof(MuonScal, max_norm) == offsetof(zero1_muon_scalars, max_norm) &&
                  offsetof(MuonScal, delta) == offsetof(zero1_muon_scalars, decay),
              "muon scalars layout");

namespace {

// ------------------------------------------------------------------ errors
zero1_status fail(zero1_status st, const char* fmt, ...)
{
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    set_error(st, buf);
    return st;
}

zero1_status ok()
{
    set_error(ZERO1_OK, "");
    return ZERO1_OK;
}

#define Z1_HIP(call)                                                                      \
    do {                                                                                  \
        hipError_t e_ = (call);                                                           \
        if (e_ != hipSuccess)                                                             \
            return fail(ZERO1_EHIP, "%s failed: %s", #call, hipGetErrorString(e_));      \
    } while (0)

zero1_status finish(hipStream_t s)
{
    static const bool sync = [] {
        const char* e = std::getenv("ZERO1_SYNC_CHECK");
        return e && e[0] && e[0] != '0';
    }();
    if (sync) {
        hipStreamCaptureStatus cs = hipStreamCaptureStatusNone;
        Z1_HIP(hipStreamIsCapturing(s, &cs));
        if (cs == hipStreamCaptureStatusNone) Z1_HIP(hipStreamSynchronize(s));
        Z1_HIP(hipGetLastError());
    }
    return ok();
}

// ------------------------------------------------------------------ device
std::mutex g_mu;
int g_cus[64];   // CUs of each device once probed; -1: not gfx950

zero1_status current_device(int& dev, int& cus)
{
    Z1_HIP(hipGetDevice(&dev));
    if (dev < 0 || dev >= 64) return fail(ZERO1_ENOTSUPPORTED, "device index %d out of range", dev);
    std::lock_guard<std::mutex> lk(g_mu);
    if (g_cus[dev] == 0) {
        hipDeviceProp_t p;
        Z1_HIP(hipGetDeviceProperties(&p, dev));
        g_cus[dev] = std::strncmp(p.gcnArchName, "gfx950", 6) == 0 ? p.multiProcessorCount : -1;
    }
    if (g_cus[dev] < 0) return fail(ZERO1_ENOTSUPPORTED, "device %d is not a gfx950", dev);
    cus = g_cus[dev];
    return ZERO1_OK;
}

// The device the call runs on has to be the one that holds the plan's table.
zero1_status plan_device(const zero1_matrix_plan* plan, int& cus)
{
    int dev = 0;
    if (zero1_status st = current_device(dev, cus)) return st;
    if (dev != plan->device)
        return fail(ZERO1_EINVAL, "the plan was made on device %d, the current device is %d", plan->device, dev);
    return ZERO1_OK;
}

// ------------------------------------------------------------------ checks
constexpr uint32_t kPlanFlags = ZERO1_MV_BF16 | ZERO1_U_F32;
constexpr uint32_t kMuonFlags = ZERO1_SUM_ONLY | ZERO1_MV_BF16 | ZERO1_RECOMPUTE_G | ZERO1_STORE_G |
                                ZERO1_DECAY_FIRST | ZERO1_CLIP_EPS | ZERO1_G_BF16 | ZERO1_U_F32 |
                                ZERO1_NO_NESTEROV;
constexpr int64_t kMaxSide = ((int64_t)1 << 31) - 256;   // rows, cols
constexpr int64_t kMaxInner = 32768;                     // the smaller of the two
constexpr int kMaxSteps = 64;
constexpr int64_t kMaxTiles = (int64_t)1 << 26;          // streaming tiles of a plan: 2^37 elements
constexpr int64_t kMaxGrid = (((int64_t)1 << 32) - 1) / 576;  // workgroups a launch: fewer than 2^32 threads

enum Has : uint32_t { kHasMaster = 1, kHasM = 2, kHasU = 4, kHasO = 8 };

zero1_status check_flags(uint32_t flags, const char* fn)
{
    if (flags & ~kMuonFlags) return fail(ZERO1_EINVAL, "%s: unknown flag bits 0x%x", fn, flags & ~kMuonFlags);
    return ZERO1_OK;
}

zero1_status check_plan(const zero1_matrix_plan* plan, uint32_t need, const char* fn)
{
    if (!plan || !plan->table) return fail(ZERO1_EINVAL, "plan is NULL or has no table");
    if ((need & kHasM) && !(plan->has & kHasM)) return fail(ZERO1_EINVAL, "%s: the plan's matrices have no m", fn);
    if ((need & kHasU) && !(plan->has & kHasU)) return fail(ZERO1_EINVAL, "%s: the plan's matrices have no u", fn);
    if ((need & kHasO) && !(plan->has & kHasO)) return fail(ZERO1_EINVAL, "%s: the plan's matrices have no o", fn);
    if ((need & kHasMaster) && !(plan->has & kHasMaster))
        return fail(ZERO1_EINVAL, "%s: the plan's matrices have no master and param_bf16", fn);
    return ZERO1_OK;
}

zero1_status check_scalars(const zero1_muon_hparams* hp)
{
    if (!(hp->lr >= 0.0) || std::isinf(hp->lr)) return fail(ZERO1_EINVAL, "lr=%g must be finite and >= 0", hp->lr);
    if (!(hp->momentum >= 0.0 && hp->momentum < 1.0))
        return fail(ZERO1_EINVAL, "momentum=%g must be in [0, 1)", hp->momentum);
    if (!(hp->weight_decay >= 0.0) || std::isinf(hp->weight_decay))
        return fail(ZERO1_EINVAL, "weight_decay=%g must be finite and >= 0", hp->weight_decay);
    if (!(hp->max_norm > 0.0))
        return fail(ZERO1_EINVAL, "max_norm=%g must be > 0 (inf disables clipping)", hp->max_norm);
    return ZERO1_OK;
}

zero1_status check_hparams(const zero1_muon_hparams* hp)
{
    if (!hp) return fail(ZERO1_EINVAL, "hp is NULL");
    if (hp->device_scalars) {
        if (reinterpret_cast<uintptr_t>(hp->device_scalars) % 8)
            return fail(ZERO1_EINVAL, "hp->device_scalars must be 8-byte aligned");
        return ZERO1_OK;
    }
    return check_scalars(hp);
}

// What a step does to singular values s in [0, top], on t = s^2: the largest
// |p(s)| = s |q(t)|, |q(t)| = |a + b t + c t^2| and |b t + c t^2| (B's
// eigenvalues).
struct Reach {
    double p, q, b;
};

Reach reach(const zero1_muon_hparams* hp, double top)
{
    const double a = hp->ns_a, b = hp->ns_b, c = hp->ns_c, tt = top * top;
    Reach r{0.0, std::fabs(a), 0.0};   // at t = 0
    auto look = [&](double t) {
        if (!(t > 0.0 && t <= tt)) return;
        const double be = b * t + c * t * t, q = a + be;
        r.p = std::max(r.p, std::sqrt(t) * std::fabs(q));
        r.q = std::max(r.q, std::fabs(q));
        r.b = std::max(r.b, std::fabs(be));
    };
    look(tt);
    if (c != 0.0) {
        look(-b / (2.0 * c));                       // q' = 0
        const double disc = 9.0 * b * b - 20.0 * a * c;
        if (disc >= 0.0) {                          // p' = 0
            look((-3.0 * b + std::sqrt(disc)) / (10.0 * c));
            look((-3.0 * b - std::sqrt(disc)) / (10.0 * c));
        }
    } else if (b != 0.0) {
        look(-a / (3.0 * b));
    }
    return r;
}

// What bounds the singular values bounds every entry of X, A and B, which fp16
// holds times 2^12: 3, 9 and 12 leave a third of its range for roundings.
zero1_status check_iteration(const zero1_muon_hparams* hp)
{
    if (hp->ns_steps < 1 || hp->ns_steps > kMaxSteps)
        return fail(ZERO1_EINVAL, "ns_steps=%d must be in [1, %d]", hp->ns_steps, kMaxSteps);
    if (!(hp->ns_eps >= 0.0) || std::isinf(hp->ns_eps))
        return fail(ZERO1_EINVAL, "ns_eps=%g must be finite and >= 0", hp->ns_eps);
    if (!std::isfinite(hp->ns_a) || !std::isfinite(hp->ns_b) || !std::isfinite(hp->ns_c))
        return fail(ZERO1_EINVAL, "ns_a, ns_b and ns_c must be finite");
    double top = 1.0;
    for (int it = 0; it < hp->ns_steps; ++it) {
        const Reach r = reach(hp, top);
        if (!(r.b <= 12.0) || !(r.p <= 3.0))
            return fail(ZERO1_EINVAL,
                        "ns_a=%g, ns_b=%g, ns_c=%g let singular values reach %g (|b s^2 + c s^4| %g) in step %d; at most 3 "
                        "(12) is supported",
                        hp->ns_a, hp->ns_b, hp->ns_c, r.p, r.b, it + 1);
        top = r.p;
    }
    return ZERO1_OK;
}

// Steps of a thin matrix's iteration, from singular values within `top` on,
// that are taken as one product: as many as keep what the steps before the last
// do to singular values near zero within kThinGrowth.  Moves `top` along.
int segment_steps(const zero1_muon_hparams* hp, int left, double& top)
{
    double growth = 1.0;
    int m = 0;
    do {
        const Reach r = reach(hp, top);
        growth *= std::max(1.0, r.q);
        top = r.p;
        ++m;
    } while (m < left && growth <= kThinGrowth);
    return m;
}

MuonArgs muon_args(const zero1_muon_hparams* hp, uint32_t flags)
{
    MuonArgs m;
    std::memset(&m, 0, sizeof m);
    m.decay_first = (flags & ZERO1_DECAY_FIRST) ? 1 : 0;
    if (hp->device_scalars) {
        m.dev = static_cast<const MuonScal*>(hp->device_scalars);
        return m;
    }
    m.lr = (float)hp->lr;
    m.mu = (float)hp->momentum;
    m.delta = (float)(1.0 - hp->lr * hp->weight_decay);
    return m;
}

zero1_status check_grads(const uint16_t* const* grads, int W, int64_t begin, uint32_t flags, Reduce& r)
{
    if (W < 1 || W > kMaxW) return fail(ZERO1_EINVAL, "W=%d must be in [1, %d]", W, kMaxW);
    if (begin < 0) return fail(ZERO1_EINVAL, "begin=%lld is negative", (long long)begin);
    if (!grads) return fail(ZERO1_EINVAL, "grads (host array of W pointers) is NULL");
    std::memset(&r, 0, sizeof r);
    for (int w = 0; w < W; ++w) {
        if (!grads[w]) return fail(ZERO1_EINVAL, "grads[%d] is NULL", w);
        r.gp.p[w] = grads[w] + begin;
    }
    r.W = W;
    r.round_bf16 = (flags & ZERO1_G_BF16) ? 1 : 0;
    if ((flags & ZERO1_SUM_ONLY) || W == 1) {
        r.mode = kAvgNone;
    } else if ((W & (W - 1)) == 0) {
        r.mode = kAvgMulPow2;
        r.inv_w = 1.0f / (float)W;
    } else {
        r.mode = kAvgDiv;
        r.f_w = (float)W;
    }
    return ZERO1_OK;
}

zero1_status check_clip(const double* rank_sumsq, int n_ranks, const zero1_norm_info* info_out)
{
    if (rank_sumsq && n_ranks < 1) return fail(ZERO1_EINVAL, "n_ranks=%d must be >= 1", n_ranks);
    if (info_out && !rank_sumsq) return fail(ZERO1_EINVAL, "info_out needs rank_sumsq");
    return ZERO1_OK;
}

// ------------------------------------------------------------------ overlap
// rows x cols elements of `esize` bytes with a row stride of ld elements.
struct Block {
    uintptr_t lo, hi;   // first byte, one past the last
    int64_t rows, cols, ld;
    size_t esize;
    const char* what;
    int idx;
};

Block block(const void* p, int64_t rows, int64_t cols, int64_t ld, size_t esize, const char* what, int idx)
{
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    return Block{lo, lo + (uintptr_t)((rows - 1) * ld + cols) * esize, rows, cols, ld, esize, what, idx};
}

// Whether two blocks whose byte ranges overlap (a.lo <= b.lo < a.hi) share an
// element.  Blocks cut out of one array (the same stride and element size) are
// told apart by rows and columns; others are taken to share.
bool share(const Block& a, const Block& b)
{
    if (a.esize != b.esize || a.ld != b.ld || (b.lo - a.lo) % a.esize) return true;
    const int64_t delta = (int64_t)((b.lo - a.lo) / a.esize);
    const int64_t q = delta / a.ld, r = delta % a.ld;   // b starts at row q, column r of a's array
    if (r < a.cols && q < a.rows) return true;
    // b's columns past the array's row end continue at column 0 of the next row
    return r + b.cols > a.ld && q + 1 < a.rows;
}

zero1_status check_blocks(std::vector<Block>& v)
{
    std::sort(v.begin(), v.end(), [](const Block& a, const Block& b) { return a.lo < b.lo; });
    std::vector<size_t> open;   // earlier blocks that may reach this one
    for (size_t i = 0; i < v.size(); ++i) {
        size_t kept = 0;
        for (size_t k = 0; k < open.size(); ++k)
            if (v[open[k]].hi > v[i].lo) open[kept++] = open[k];
        open.resize(kept);
        for (size_t k : open)
            if (share(v[k], v[i]))
                return fail(ZERO1_EINVAL, "buffers overlap: %s[%d] and %s[%d]", v[k].what, v[k].idx, v[i].what,
                            v[i].idx);
        open.push_back(i);
    }
    return ZERO1_OK;
}

// ------------------------------------------------------------------ plan
size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
int64_t round_up64(int64_t x, int64_t a) { return (x + a - 1) / a * a; }

// Matrices share a group until their iteration buffers pass this: enough
// tiles in a launch to fill the chip several times, little enough to stay
// near the 256 MB MALL.  Larger plans take larger groups, so that a plan holds
// at most ZERO1_MUON_MAX_GROUPS of them.
constexpr int64_t kGroupBytes = (int64_t)512 << 20;

// Tile shapes (by TileShape) and what they take, in us: `start` a round of
// tiles for its first loads and its epilogue, then for every 64 of the inner
// dimension `one` where a tile has the chip to itself and `all` where every
// slot holds one (the chip's clock falls with the load).  For the whole chip of 256
// CUs: on a part of it the results are the same and the choice may be slower.
// Measured on MI355X in one session (shorter epilogues have taken 1 to 2 us off
// every entry since):
//   matrix        product (inner)  128 x 128   192 x 192   256 x 256
//   4096 x 11008  gram (11008)        257 us      202 us      232 us
//                 poly (4096)         101          84          97
//                 apply (4096)        361         419         346
//   1111 x 2501   gram (2501)          29          47          60   (3 matrices)
//                 apply (1111)         37          33          40
//   768 x 768     gram (768)           14          22          29   (12 matrices)
struct TileCost {
    int side;       // blocks
    int slots;      // tiles the chip holds at once
    double start, one, all;
};
constexpr TileCost kTiles[3] = {{2, 512, 6.0, 0.44, 0.95}, {3, 256, 11.0, 0.87, 1.10}, {4, 256, 14.0, 1.08, 1.60}};
constexpr int kXcds = 8;

double tile_time(const TileCost& c, double tiles, int inner)
{
    const double full = std::floor(tiles / c.slots), rest = tiles - full * c.slots;
    double t = full * (c.start + inner * c.all);
    if (rest > 0) t += c.start + inner * (c.one + (c.all - c.one) * rest / c.slots);
    return t;
}

struct Host {
    std::vector<MatDesc> mats;
    std::vector<StreamTile> tiles;
    std::vector<ProdTile> list;
    std::vector<zero1_matrix_group> groups;
    int64_t area = 0;
    uint32_t has = 0;
    int64_t elems = 0;
    int32_t n_dense = 0, dense_tiles = 0;   // matrices that are not thin (the first ones), their streaming tiles
    int32_t dense_most = 0;                 // and the most of one
    size_t off_tiles() const { return round_up(sizeof(MatDesc) * mats.size(), 256); }
    size_t off_list() const { return off_tiles() + round_up(sizeof(StreamTile) * tiles.size(), 256); }
    size_t bytes() const { return off_list() + sizeof(ProdTile) * list.size(); }
};

uint32_t buffers_of(const zero1_matrix& q)
{
    return (q.master ? +kHasMaster : 0u) | (q.m ? +kHasM : 0u) | (q.u ? +kHasU : 0u) | (q.o ? +kHasO : 0u);
}

// What the sizes of a plan's parts depend on.
zero1_status check_shape(const zero1_matrix& q, int i, uint32_t has0)
{
    if (q.rows < 1 || q.cols < 1 || q.rows > kMaxSide || q.cols > kMaxSide)
        return fail(ZERO1_EINVAL, "matrix %d: %lld x %lld: rows and cols must be in [1, %lld]", i, (long long)q.rows,
                    (long long)q.cols, (long long)kMaxSide);
    if (std::min(q.rows, q.cols) > kMaxInner)
        return fail(ZERO1_EINVAL, "matrix %d: %lld x %lld: the smaller side is at most %lld", i, (long long)q.rows,
                    (long long)q.cols, (long long)kMaxInner);
    const int64_t strides[3] = {q.ld, q.ldu, q.ldo};
    const char* names[3] = {"ld", "ldu", "ldo"};
    for (int k = 0; k < 3; ++k)
        if (strides[k] != 0 && (strides[k] < q.cols || strides[k] > kMaxSide))
            return fail(ZERO1_EINVAL, "matrix %d: %s=%lld must be 0 or in [cols=%lld, %lld]", i, names[k],
                        (long long)strides[k], (long long)q.cols, (long long)kMaxSide);
    for (int k = 0; k < 3; ++k)
        if ((q.rows - 1) * std::max(strides[k], q.cols) + q.cols > ((int64_t)1 << 44))
            return fail(ZERO1_EINVAL, "matrix %d: %lld rows of %s=%lld span more than 2^44 elements", i,
                        (long long)q.rows, names[k], (long long)std::max(strides[k], q.cols));
    const uint32_t has = buffers_of(q);
    if (!has) return fail(ZERO1_EINVAL, "matrix %d has no buffer", i);
    if (i > 0 && has != has0)
        return fail(ZERO1_EINVAL, "matrix %d: every matrix of a plan has the same buffers (NULL or not)", i);
    return ZERO1_OK;
}

zero1_status check_matrix(const zero1_matrix& q, int i, uint32_t flags)
{
    if (q.shard_offset < 0) return fail(ZERO1_EINVAL, "matrix %d: negative shard_offset", i);
    if (!std::isfinite(q.scale)) return fail(ZERO1_EINVAL, "matrix %d: scale must be finite", i);
    if (!q.master != !q.param_bf16)
        return fail(ZERO1_EINVAL, "matrix %d: master and param_bf16 go together", i);
    const size_t align[5] = {sizeof(float), 2, (flags & ZERO1_MV_BF16) ? (size_t)2 : 4,
                             (flags & ZERO1_U_F32) ? (size_t)4 : 2, 2};
    const void* p[5] = {q.master, q.param_bf16, q.m, q.u, q.o};
    const char* pn[5] = {"master", "param_bf16", "m", "u", "o"};
    for (int k = 0; k < 5; ++k)
        if (reinterpret_cast<uintptr_t>(p[k]) % align[k])
            return fail(ZERO1_EINVAL, "matrix %d: %s is not aligned to its elements", i, pn[k]);
    return ZERO1_OK;
}

// The buffers: values, alignment, and that no two share an element.
zero1_status check_buffers(const zero1_matrix* mats, int n, uint32_t flags)
{
    const size_t mb = (flags & ZERO1_MV_BF16) ? 2 : 4, ub = (flags & ZERO1_U_F32) ? 4 : 2;
    std::vector<Block> blocks;
    for (int i = 0; i < n; ++i) {
        const zero1_matrix& q = mats[i];
        if (zero1_status st = check_matrix(q, i, flags)) return st;
        const int64_t ld = q.ld ? q.ld : q.cols, ldu = q.ldu ? q.ldu : q.cols, ldo = q.ldo ? q.ldo : q.cols;
        if (q.master) {
            blocks.push_back(block(q.param_bf16, q.rows, q.cols, ld, 2, "param_bf16", i));
            blocks.push_back(block(q.master, q.rows, q.cols, ld, 4, "master", i));
        }
        if (q.m) blocks.push_back(block(q.m, q.rows, q.cols, ld, mb, "m", i));
        if (q.u) blocks.push_back(block(q.u, q.rows, q.cols, ldu, ub, "u", i));
        // o in place of a bf16 u is the one overlap that is allowed
        const bool in_place = q.o && (const void*)q.o == q.u && ub == 2 && ldo == ldu;
        if (q.o && !in_place) blocks.push_back(block(q.o, q.rows, q.cols, ldo, 2, "o", i));
    }
    return check_blocks(blocks);
}

// Rows that a thin matrix is padded to; 0: it is not thin.
int thin_rows(int64_t k) { return k > kThin ? 0 : k > 64 ? 128 : k > 32 ? 64 : 32; }

// Lays out a matrix's iteration buffers from byte `at` on; returns their end.
int64_t place(MatDesc& d, int64_t at)
{
    const int thin = thin_rows(d.k);
    if (thin) {
        d.kp = thin;
        d.n_parts = thin <= 64 && d.n <= kThinOne ? 1 : (int32_t)std::min<int64_t>(kThinMaxParts, (d.n + 127) / 128);
        d.split = (int32_t)round_up64((d.n + d.n_parts - 1) / d.n_parts, kPad);
        d.n_parts = (int32_t)(((int64_t)d.n + d.split - 1) / d.split);
        d.x[0] = at;
        d.lo = d.x[0] + round_up64((int64_t)d.k * d.np * 4, 256);
        d.a = d.lo + 256;
        d.b = d.a + (int64_t)d.n_parts * thin * thin * 4;
        return d.b + (int64_t)2 * thin * thin * 2;
    }
    const Buffers b = buffers(at, (uint32_t)(d.kp / kPad), (uint32_t)(d.np / kPad));   // multiples of 8 KiB
    d.x[0] = b.x0;
    d.x[1] = b.x1;
    d.lo = b.lo;
    d.a = b.a;
    d.b = b.b;
    return b.end;
}
static_assert((kThinMaxParts + 1) * sizeof(int32_t) <= 256, "exponents of the parts and of their sum");

// Block rows and columns of X, or of A and B.
struct Blocks {
    int rows, cols;
};

Blocks blocks_of(const MatDesc& d, bool sym) { return Blocks{d.kp / kPad, (sym ? d.kp : d.np) / kPad}; }

// 0: the gram is a product like the others; 1: split (kSplitRows); by the matrix alone.
int16_t split_gram(int64_t k, int64_t n)
{
    return k > kThin && (k + kPad - 1) / kPad <= kSplitRows && (n + kPad - 1) / kPad >= kSplitInner ? 1 : 0;
}

ProdTile tile_of(const Host& h, size_t m, int i, int j)
{
    const MatDesc& d = h.mats[m];
    return ProdTile{d.x[0], (int32_t)m, i, j, d.kp / kPad, d.np / kPad, 0};
}

// Appends a group's tiles of `side` blocks: all of X, or (sym) those of A and B
// that reach above the diagonal.  Workgroup b runs on XCD b % 8, which has an
// L2 of its own: of matrices alike, each XCD takes one contiguous eighth of the
// tiles, walked in strips of 8 tile columns, so that the 32 tiles it works on
// at once share 4 rows and 8 columns of the operands.
int32_t add_tiles(Host& h, size_t first, size_t end, int side, bool sym)
{
    const size_t start = h.list.size();
    std::vector<ProdTile> seq;
    for (size_t m = first; m < end;) {
        seq.clear();
        size_t e = m;
        for (; e < end && h.mats[e].kp == h.mats[m].kp && h.mats[e].np == h.mats[m].np; ++e) {
            const Blocks b = blocks_of(h.mats[e], sym);
            const int strip = 8 * side;
            for (int js = 0; js < b.cols; js += strip)
                for (int i = 0; i < b.rows; i += side)
                    for (int j = js; j < std::min(js + strip, b.cols); j += side)
                        if (!sym || j >= i) seq.push_back(tile_of(h, e, i, j));
        }
        const size_t base = h.list.size() - start;
        h.list.resize(h.list.size() + seq.size());
        size_t next = 0;
        for (size_t x = 0; x < kXcds; ++x)
            for (size_t t = (x + kXcds - base % kXcds) % kXcds; t < seq.size(); t += kXcds)
                h.list[start + base + t] = seq[next++];
        m = e;
    }
    return (int32_t)(h.list.size() - start);
}

// The tile shape that takes least for a group's symmetric products (gram and
// poly) or for its apply.
int16_t best_tile(const Host& h, size_t first, size_t end, bool sym)
{
    int16_t best = 0;
    double least = 0.0;
    for (int16_t s = 0; s < 3; ++s) {
        const int side = kTiles[s].side;
        double tiles = 0, gram = 0, apply = 0;
        for (size_t m = first; m < end; ++m) {
            const Blocks b = blocks_of(h.mats[m], sym);
            const double r = (b.rows + side - 1) / side, c = (b.cols + side - 1) / side;
            tiles += sym ? r * (r + 1) / 2 : r * c;
            gram = std::max(gram, (double)h.mats[m].np / kPad);
            apply = std::max(apply, (double)h.mats[m].kp / kPad);
        }
        double t = tile_time(kTiles[s], tiles, (int)apply);
        if (sym) t += tile_time(kTiles[s], tiles, (int)gram);
        if (s == 0 || t < least) {
            best = s;
            least = t;
        }
    }
    return best;
}

zero1_status add_group(Host& h, size_t first, size_t end)
{
    int64_t most = 0;   // 64 x 64 blocks, or 64 columns of thin matrices: no list of the group is longer
    for (size_t m = first; m < end; ++m)
        most += (int64_t)(h.mats[m].np / kPad) * (thin_rows(h.mats[m].k) ? 1 : h.mats[m].kp / kPad);
    if (most > kMaxGrid)
        return fail(ZERO1_EINVAL, "matrices of %lld blocks are iterated together, at most %lld can be",
                    (long long)most, (long long)kMaxGrid);
    zero1_matrix_group g;
    std::memset(&g, 0, sizeof g);
    g.first = (int32_t)first;
    g.thin = (int16_t)thin_rows(h.mats[first].k);
    auto here = [&h] { return (int64_t)h.list.size(); };
    g.sym0 = here();
    if (g.thin) {
        bool one = g.thin <= 64;
        for (size_t m = first; m < end; ++m) {
            const MatDesc& d = h.mats[m];
            one = one && d.n <= kThinOne;
            g.parts = std::max(g.parts, (int16_t)d.n_parts);
            for (int p = 0; p < d.n_parts; ++p) h.list.push_back(tile_of(h, m, p, p * (d.split / kPad)));
        }
        g.one = one ? 1 : 0;
        g.n_sym = (int32_t)(here() - g.sym0);
        g.full0 = here();
        for (size_t m = first; m < end; ++m)
            for (int j = 0; j < h.mats[m].np / kPad; ++j) h.list.push_back(tile_of(h, m, 0, j));
        g.n_full = (int32_t)(here() - g.full0);
        g.n_blocks = (int32_t)(end - first);
    } else {
        g.sym_tile = best_tile(h, first, end, true);
        g.full_tile = best_tile(h, first, end, false);
        g.n_sym = add_tiles(h, first, end, kTiles[g.sym_tile].side, true);
        g.full0 = here();
        g.n_full = add_tiles(h, first, end, kTiles[g.full_tile].side, false);
        g.blocks0 = here();
        g.n_blocks = add_tiles(h, first, end, 1, false);
        g.split = split_gram(h.mats[first].k, h.mats[first].n);
        g.gram0 = here();
        if (g.split) g.n_gram = add_tiles(h, first, end, 1, true);
    }
    h.groups.push_back(g);
    return ZERO1_OK;
}

void sides(const zero1_matrix& q, MatDesc& d)
{
    d.k = (int32_t)std::min(q.rows, q.cols);
    d.n = (int32_t)std::max(q.rows, q.cols);
    d.kp = (int32_t)round_up64(d.k, kPad);
    d.np = (int32_t)round_up64(d.n, kPad);
}

zero1_status build(const zero1_matrix* mats, int n, Host& h)
{
    if (!mats || n < 1) return fail(ZERO1_EINVAL, "need at least one matrix");
    h.has = buffers_of(mats[0]);
    std::vector<int> order(n);
    for (int i = 0; i < n; ++i) {
        if (zero1_status st = check_shape(mats[i], i, h.has)) return st;
        h.elems += mats[i].rows * mats[i].cols;
        if (h.elems > kMaxTiles * 4 * kQuadsPerTile) return fail(ZERO1_EINVAL, "too many elements in one plan");
        order[i] = i;
    }
    // largest products first: the tiles that run longest are dispatched first;
    // those of a split gram behind the others, thin ones last
    auto small = [&](int i) { return std::min(mats[i].rows, mats[i].cols); };
    auto large = [&](int i) { return std::max(mats[i].rows, mats[i].cols); };
    auto kind = [&](int i) { return small(i) <= kThin ? 2 : (int)split_gram(small(i), large(i)); };
    std::stable_sort(order.begin(), order.end(), [&](int a, int b) {
        const int ca = kind(a), cb = kind(b);
        if (ca != cb) return ca < cb;
        return small(a) != small(b) ? small(a) > small(b) : large(a) > large(b);
    });
    int64_t used = 0, total = 0;
    for (int i = 0; i < n; ++i) {
        MatDesc d;
        std::memset(&d, 0, sizeof d);
        sides(mats[i], d);
        total += place(d, 0);
    }
    // two groups in a row hold more than the budget, but for the classes' ends
    const int64_t budget = std::max(kGroupBytes, total / (ZERO1_MUON_MAX_GROUPS / 2 - 4));
    size_t group_first = 0;
    auto close_group = [&](size_t end) {
        h.area = std::max(h.area, used);
        used = 0;
        return add_group(h, std::exchange(group_first, end), end);
    };
    for (int k = 0; k < n; ++k) {
        const zero1_matrix& q = mats[order[k]];
        MatDesc d;
        std::memset(&d, 0, sizeof d);
        d.rows = q.rows;
        d.cols = q.cols;
        d.ld = q.ld ? q.ld : q.cols;
        d.ldu = q.ldu ? q.ldu : q.cols;
        d.ldo = q.ldo ? q.ldo : q.cols;
        d.shard_offset = q.shard_offset;
        d.param = q.param_bf16;
        d.master = q.master;
        d.m = q.m;
        d.u = q.u;
        d.o = q.o;
        d.scale = q.scale;
        d.tall = q.rows > q.cols ? 1 : 0;
        sides(q, d);
        const bool flat = q.rows == 1 || (d.ld == q.cols && d.ldu == q.cols && d.ldo == q.cols);
        d.vrows = flat ? 1 : (int32_t)q.rows;
        d.vcols = flat ? q.rows * q.cols : q.cols;
        d.qpr = (d.vcols + 3) / 4;
        const int64_t quads = d.vrows * d.qpr, nt = (quads + kQuadsPerTile - 1) / kQuadsPerTile;
        if ((int64_t)h.tiles.size() + nt > kMaxTiles) return fail(ZERO1_EINVAL, "too many elements in one plan");
        d.tile0 = (int32_t)h.tiles.size();
        d.n_tiles = (int32_t)nt;
        for (int64_t t = 0; t < nt; ++t) {
            StreamTile s{k, (int32_t)t, 0, 0};
            if (!flat) {
                s.row0 = (int32_t)(t * kQuadsPerTile / d.qpr);
                s.q0 = (int32_t)(t * kQuadsPerTile % d.qpr);
            }
            h.tiles.push_back(s);
        }
        if (h.has & kHasU) {   // its place in a group's buffers
            int64_t to = place(d, used);
            if (used > 0 && (to > budget || thin_rows(d.k) != thin_rows(h.mats.back().k) ||
                             split_gram(d.k, d.n) != split_gram(h.mats.back().k, h.mats.back().n))) {
                if (zero1_status st = close_group(h.mats.size())) return st;
                to = place(d, used);
            }
            used = to;
        }
        if (!thin_rows(d.k)) {
            ++h.n_dense;
            h.dense_tiles = (int32_t)h.tiles.size();
            h.dense_most = std::max(h.dense_most, d.n_tiles);
        }
        h.mats.push_back(d);
    }
    if (h.has & kHasU) {
        if (zero1_status st = close_group(h.mats.size())) return st;
        if (h.groups.size() > ZERO1_MUON_MAX_GROUPS) return fail(ZERO1_EINVAL, "too many groups in one plan");
    }
    return ZERO1_OK;
}

// Workspace: the streaming tiles' partial sums of squares, the norms, then a
// group's iteration buffers.
size_t ws_norms(const zero1_matrix_plan* p) { return round_up(sizeof(double) * (size_t)p->n_tiles, 256); }
size_t ws_area(const zero1_matrix_plan* p) { return ws_norms(p) + round_up(sizeof(NormRec) * (size_t)p->n_mats, 256); }

zero1_status check_ws(const zero1_matrix_plan* plan, const void* ws, size_t bytes)
{
    const size_t need = zero1_muon_workspace_bytes(plan);
    if (!ws) return fail(ZERO1_EWORKSPACE, "workspace is NULL (need %zu bytes)", need);
    if (reinterpret_cast<uintptr_t>(ws) % 256) return fail(ZERO1_EWORKSPACE, "workspace must be 256-byte aligned");
    if (bytes < need) return fail(ZERO1_EWORKSPACE, "workspace has %zu bytes, needs %zu", bytes, need);
    return ZERO1_OK;
}

const MatDesc* plan_mats(const zero1_matrix_plan* p) { return static_cast<const MatDesc*>(p->table); }
const StreamTile* plan_tiles(const zero1_matrix_plan* p)
{
    return reinterpret_cast<const StreamTile*>(static_cast<const char*>(p->table) + p->off_tiles);
}

// The streaming kernels' grid, as the AdamW update's: a workgroup a tile up
// to kMaxPartials tiles, then 8 a CU with each XCD on its own eighth.
struct Shape {
    int grid, split;
};

Shape stream_shape(int n_tiles, int cus)
{
    if (n_tiles <= kMaxPartials) return Shape{n_tiles, 1};
    return Shape{cus * 8 / 8 * 8, 8};
}

zero1_status momentum(const Reduce& r, const zero1_matrix_plan* plan, const zero1_muon_hparams* hp,
                      const double* rank_sumsq, int n_ranks, uint32_t flags, zero1_norm_info* info_out,
                      double* partials, int cus, hipStream_t s)
{
    const MuonClip mc{rank_sumsq, n_ranks, hp->max_norm, (flags & ZERO1_CLIP_EPS) ? 1 : 0,
                      reinterpret_cast<NormInfo*>(info_out)};
    const Shape sh = stream_shape(plan->n_tiles, cus);
    Z1_HIP(launch_momentum(r, plan_mats(plan), plan_tiles(plan), plan->n_tiles, (plan->flags & ZERO1_MV_BF16) != 0,
                           (plan->flags & ZERO1_U_F32) != 0, !(flags & ZERO1_NO_NESTEROV), muon_args(hp, flags), mc,
                           partials, sh.grid, sh.split, s));
    return ZERO1_OK;
}

// The iteration over every group, from u and its tiles' partials; `last` says
// what becomes of the result.
zero1_status iterate(const zero1_matrix_plan* plan, const zero1_muon_hparams* hp, uint32_t flags, NsLast last,
                     char* ws, hipStream_t s)
{
    const double* partials = reinterpret_cast<const double*>(ws);
    NormRec* norms = reinterpret_cast<NormRec*>(ws + ws_norms(plan));
    const bool norms_first = plan->dense_most > kNormTiles;
    if (norms_first) Z1_HIP(launch_ns_norms(plan_mats(plan), plan->n_dense, partials, hp->ns_eps, norms, s));
    const char* tb = static_cast<const char*>(plan->table);
    NsArgs g;
    std::memset(&g, 0, sizeof g);
    g.mats = plan_mats(plan);
    const ProdTile* list = reinterpret_cast<const ProdTile*>(tb + plan->off_list);
    g.area = ws + ws_area(plan);
    g.norms = norms;
    g.a = (float)hp->ns_a;
    g.b = (float)hp->ns_b;
    g.c = (float)hp->ns_c;
    const bool u_f32 = (plan->flags & ZERO1_U_F32) != 0;
    const MuonArgs ma = muon_args(hp, flags);
    for (int i = 0; i < plan->n_groups; ++i) {
        const zero1_matrix_group& q = plan->groups[i];
        g.first = q.first;
        g.sym = list + q.sym0;
        g.full = list + q.full0;
        g.blocks = list + q.blocks0;
        g.gram = list + q.gram0;
        if (q.thin) {
            double top = 1.0;
            for (int it = 0; it < hp->ns_steps;) {
                const int m = segment_steps(hp, hp->ns_steps - it, top), mid = it > 0 ? 1 : 0;
                const NsLast to = it + m == hp->ns_steps ? last : kNsMid;
                if (q.one && !mid && to != kNsMid) {
                    Z1_HIP(launch_thin_one(g, q.thin, u_f32, m, hp->ns_eps, norms, to, ma, q.n_blocks, s));
                } else {
                    Z1_HIP(launch_thin_gram(g, q.thin, u_f32 || mid, mid, q.n_sym, s));
                    if (q.parts > 1) Z1_HIP(launch_thin_sum(g, q.thin, q.n_blocks, s));
                    Z1_HIP(launch_thin_poly(g, q.thin, mid, m, hp->ns_eps, norms, q.n_blocks, s));
                    Z1_HIP(launch_thin_apply(g, q.thin, u_f32 || mid, mid, to, ma, q.n_full, s));
                }
                it += m;
            }
            continue;
        }
        const TileShape sym = (TileShape)q.sym_tile, full = (TileShape)q.full_tile;
        Z1_HIP(launch_ns_prepare(g, u_f32, norms_first ? nullptr : partials, hp->ns_eps, norms, q.n_blocks, s));
        for (int it = 0; it < hp->ns_steps; ++it) {
            if (q.split) Z1_HIP(launch_ns_gram_split(g, it, q.n_gram, s));
            else Z1_HIP(launch_ns_gram(g, it, sym, q.n_sym, s));
            Z1_HIP(launch_ns_poly(g, sym, q.n_sym, s));
            Z1_HIP(launch_ns_apply(g, it, u_f32, it + 1 == hp->ns_steps ? last : kNsMid, ma, full, q.n_full, s));
        }
    }
    return ZERO1_OK;
}

}  // namespace

// ====================================================================== ABI
extern "C" {

size_t zero1_muon_table_bytes(const zero1_matrix* mats, int n_mats)
{
    try {
        Host h;
        return build(mats, n_mats, h) == ZERO1_OK ? h.bytes() : 0;
    } catch (const std::exception& e) {
        fail(ZERO1_EINVAL, "zero1_muon_table_bytes: %s", e.what());
        return 0;
    }
}

zero1_status zero1_muon_plan(const zero1_matrix* mats, int n_mats, uint32_t flags, void* table, size_t table_bytes,
                             zero1_matrix_plan* plan_out)
{
    try {
        zero1_status st;
        if ((st = check_flags(flags, "zero1_muon_plan"))) return st;
        if (!plan_out) return fail(ZERO1_EINVAL, "plan_out is NULL");
        Host h;
        if ((st = build(mats, n_mats, h)) || (st = check_buffers(mats, n_mats, flags))) return st;
        const size_t need = h.bytes();
        if (!table) return fail(ZERO1_EWORKSPACE, "table is NULL (need %zu bytes)", need);
        if (reinterpret_cast<uintptr_t>(table) % 256) return fail(ZERO1_EWORKSPACE, "table must be 256-byte aligned");
        if (table_bytes < need) return fail(ZERO1_EWORKSPACE, "table has %zu bytes, needs %zu", table_bytes, need);
        int dev = 0, cus = 0;
        if ((st = current_device(dev, cus))) return st;
        std::vector<char> host(need, 0);
        std::memcpy(host.data(), h.mats.data(), sizeof(MatDesc) * h.mats.size());
        std::memcpy(host.data() + h.off_tiles(), h.tiles.data(), sizeof(StreamTile) * h.tiles.size());
        if (!h.list.empty()) std::memcpy(host.data() + h.off_list(), h.list.data(), sizeof(ProdTile) * h.list.size());
        Z1_HIP(hipMemcpy(table, host.data(), need, hipMemcpyHostToDevice));
        zero1_matrix_plan p;
        std::memset(&p, 0, sizeof p);
        p.table = table;
        p.elems = h.elems;
        p.off_tiles = (int64_t)h.off_tiles();
        p.off_list = (int64_t)h.off_list();
        p.area_bytes = h.area;
        p.n_mats = n_mats;
        p.n_tiles = (int32_t)h.tiles.size();
        p.n_groups = (int32_t)h.groups.size();
        std::copy(h.groups.begin(), h.groups.end(), p.groups);
        p.flags = flags & kPlanFlags;
        p.has = h.has;
        p.n_dense = h.n_dense;
        p.dense_tiles = h.dense_tiles;
        p.dense_most = h.dense_most;
        p.device = dev;
        *plan_out = p;
        return ok();
    } catch (const std::exception& e) {
        return fail(ZERO1_EINVAL, "zero1_muon_plan: %s", e.what());
    }
}

size_t zero1_muon_workspace_bytes(const zero1_matrix_plan* plan)
{
    if (!plan || !plan->table) return 0;
    return ws_area(plan) + round_up((size_t)plan->area_bytes, 256);
}

zero1_status zero1_muon_scalars_derive(const zero1_muon_hparams* hp, zero1_muon_scalars* out)
{
    if (!hp || !out) return fail(ZERO1_EINVAL, "hp or out is NULL");
    if (zero1_status st = check_scalars(hp)) return st;
    zero1_muon_hparams h = *hp;
    h.device_scalars = nullptr;
    const MuonArgs a = muon_args(&h, 0);
    zero1_muon_scalars o;
    std::memset(&o, 0, sizeof o);
    o.lr = a.lr;
    o.momentum = a.mu;
    o.decay = a.delta;
    o.max_norm = hp->max_norm;
    *out = o;
    return ok();
}

zero1_status zero1_muon_momentum(const uint16_t* const* grads, int W, int64_t begin, const zero1_matrix_plan* plan,
                                 const zero1_muon_hparams* hp, const double* rank_sumsq, int n_ranks, uint32_t flags,
                                 zero1_norm_info* info_out, void* stream)
{
    zero1_status st;
    int cus = 0;
    if ((st = check_flags(flags, "zero1_muon_momentum"))) return st;
    if ((st = check_plan(plan, kHasM | kHasU, "zero1_muon_momentum"))) return st;
    if ((st = check_hparams(hp))) return st;
    Reduce r;
    if ((st = check_grads(grads, W, begin, flags, r))) return st;
    if ((st = check_clip(rank_sumsq, n_ranks, info_out))) return st;
    if ((st = plan_device(plan, cus))) return st;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if ((st = momentum(r, plan, hp, rank_sumsq, n_ranks, flags, info_out, nullptr, cus, s))) return st;
    return finish(s);
}

zero1_status zero1_orthogonalize(const zero1_matrix_plan* plan, const zero1_muon_hparams* hp, uint32_t flags, void* ws,
                                 size_t ws_bytes, void* stream)
{
    zero1_status st;
    int cus = 0;
    if ((st = check_flags(flags, "zero1_orthogonalize"))) return st;
    if ((st = check_plan(plan, kHasU | kHasO, "zero1_orthogonalize"))) return st;
    if (!hp) return fail(ZERO1_EINVAL, "hp is NULL");
    if ((st = check_iteration(hp))) return st;
    if ((st = check_ws(plan, ws, ws_bytes))) return st;
    if ((st = plan_device(plan, cus))) return st;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (plan->n_dense > 0) {
        Shape sh = stream_shape(plan->dense_tiles, cus);
        if (sh.split == 1) sh.grid = (sh.grid + kSumsqTiles - 1) / kSumsqTiles;
        Z1_HIP(launch_u_sumsq(plan_mats(plan), plan_tiles(plan), plan->dense_tiles, (plan->flags & ZERO1_U_F32) != 0,
                              static_cast<double*>(ws), sh.grid, sh.split, s));
    }
    if ((st = iterate(plan, hp, flags, kNsWriteO, static_cast<char*>(ws), s))) return st;
    return finish(s);
}

zero1_status zero1_muon_update(const zero1_matrix_plan* plan, const zero1_muon_hparams* hp, uint32_t flags,
                               void* stream)
{
    zero1_status st;
    int cus = 0;
    if ((st = check_flags(flags, "zero1_muon_update"))) return st;
    if ((st = check_plan(plan, kHasMaster | kHasO, "zero1_muon_update"))) return st;
    if ((st = check_hparams(hp))) return st;
    if ((st = plan_device(plan, cus))) return st;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const Shape sh = stream_shape(plan->n_tiles, cus);
    Z1_HIP(launch_muon_update(plan_mats(plan), plan_tiles(plan), plan->n_tiles, muon_args(hp, flags), sh.grid,
                              sh.split, s));
    return finish(s);
}

zero1_status zero1_muon_step(const uint16_t* const* grads, int W, int64_t begin, const zero1_matrix_plan* plan,
                             const zero1_muon_hparams* hp, const double* rank_sumsq, int n_ranks, uint32_t flags,
                             zero1_norm_info* info_out, void* ws, size_t ws_bytes, void* stream)
{
    zero1_status st;
    int cus = 0;
    if ((st = check_flags(flags, "zero1_muon_step"))) return st;
    if ((st = check_plan(plan, kHasMaster | kHasM | kHasU, "zero1_muon_step"))) return st;
    if ((st = check_hparams(hp))) return st;
    if ((st = check_iteration(hp))) return st;
    Reduce r;
    if ((st = check_grads(grads, W, begin, flags, r))) return st;
    if ((st = check_clip(rank_sumsq, n_ranks, info_out))) return st;
    if ((st = check_ws(plan, ws, ws_bytes))) return st;
    if ((st = plan_device(plan, cus))) return st;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if ((st = momentum(r, plan, hp, rank_sumsq, n_ranks, flags, info_out,
                       plan->n_dense > 0 ? static_cast<double*>(ws) : nullptr, cus, s)))
        return st;
    if ((st = iterate(plan, hp, flags, kNsUpdate, static_cast<char*>(ws), s))) return st;
    return finish(s);
}

}  // extern "C"
