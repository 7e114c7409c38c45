// Plans of the Muon entry points, checked without a GPU: muon_api.cpp linked
// with the stand-ins below for the HIP runtime and the kernels' launchers.
// Over random lists of matrices it takes the plan's table apart (every quad,
// block and column of every matrix in exactly one tile; the iteration's buffers
// apart from one another and inside the workspace) and checks every launch
// (its grid, the lists it is given, what precedes it).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <random>
#include <set>
#include <string>
#include <tuple>
#include <vector>

#include "../../include/zero1.h"
#include "../../zero_sharded_mixed_zero1_amd/csrc/muon.h"

using namespace z1;

#define REQUIRE(cond)                                                                    \
    do {                                                                                 \
        if (!(cond)) {                                                                   \
            std::printf("%s:%d: %s (case %d)\n", __FILE__, __LINE__, #cond, g_case);     \
            std::exit(1);                                                                \
        }                                                                                \
    } while (0)

static int g_case = 0;
static int splits = 0;   // groups of split grams seen

// ------------------------------------------------------------------ stand-ins
extern "C" {
hipError_t hipGetDevice(int* d) { *d = 0; return hipSuccess; }
hipError_t hipGetDeviceProperties(hipDeviceProp_t* p, int)
{
    std::memset(p, 0, sizeof *p);
    std::strcpy(p->gcnArchName, "gfx950:sramecc+:xnack-");
    p->multiProcessorCount = 256;
    return hipSuccess;
}
hipError_t hipMemcpy(void* d, const void* s, size_t n, hipMemcpyKind) { std::memcpy(d, s, n); return hipSuccess; }
const char* hipGetErrorString(hipError_t) { return "error"; }
hipError_t hipGetLastError(void) { return hipSuccess; }
hipError_t hipStreamIsCapturing(hipStream_t, hipStreamCaptureStatus*) { return hipSuccess; }
hipError_t hipStreamSynchronize(hipStream_t) { return hipSuccess; }
}

static std::string g_error;
namespace z1 {
int set_error(int st, const char* msg) { g_error = msg; return st; }
}

static const zero1_matrix_plan* g_plan;
static std::vector<std::string> g_log;   // launches by name
static char *g_ws, *g_ws_end;
static bool g_norms_first;               // norms have a launch of their own

static void in_table(const void* p, size_t bytes, size_t total)
{
    const char *t = static_cast<const char*>(g_plan->table), *c = static_cast<const char*>(p);
    REQUIRE(c >= t && c + bytes <= t + total);
}

static size_t g_table_bytes;

static hipError_t launched(const char* name, int64_t grid, int64_t threads)
{
    REQUIRE(grid >= 1 && grid * threads < (int64_t)1 << 32);
    g_log.push_back(name);
    return hipSuccess;
}

static void group_args(const NsArgs& g)
{
    REQUIRE(g.mats == g_plan->table && g.area >= g_ws && g.area + g_plan->area_bytes <= g_ws_end);
    REQUIRE((uintptr_t)g.area % 256 == 0 && (char*)g.norms >= g_ws && (char*)(g.norms + g_plan->n_mats) <= g.area);
}

namespace z1 {
hipError_t launch_momentum(const Reduce& r, const MatDesc*, const StreamTile*, int n_tiles, bool, bool, bool,
                           const MuonArgs&, const MuonClip&, double* partials, int nblocks, int split, hipStream_t)
{
    REQUIRE(r.W >= 1 && n_tiles == g_plan->n_tiles && nblocks % split == 0);
    REQUIRE(!partials || (char*)(partials + n_tiles) <= g_ws_end);
    return launched("momentum", nblocks, kThreads);
}
hipError_t launch_u_sumsq(const MatDesc*, const StreamTile*, int n_tiles, bool, double* partials, int nblocks,
                          int split, hipStream_t)
{
    REQUIRE(n_tiles == g_plan->dense_tiles && nblocks % split == 0 && (char*)partials == g_ws);
    return launched("sumsq", nblocks, kThreads);
}
hipError_t launch_ns_norms(const MatDesc*, int n, const double*, double, NormRec*, hipStream_t)
{
    REQUIRE(n == g_plan->n_dense);
    return launched("norms", n, kThreads);
}
hipError_t launch_muon_update(const MatDesc*, const StreamTile*, int n_tiles, const MuonArgs&, int nblocks, int split,
                              hipStream_t)
{
    REQUIRE(n_tiles == g_plan->n_tiles && nblocks % split == 0);
    return launched("update", nblocks, kThreads);
}
hipError_t launch_ns_prepare(const NsArgs& g, bool, const double* partials, double, NormRec* norms, int grid, hipStream_t)
{
    group_args(g);
    REQUIRE(norms == g.norms && (partials == nullptr) == g_norms_first);
    REQUIRE(!partials || (char*)partials == g_ws);
    in_table(g.blocks, sizeof(ProdTile) * grid, g_table_bytes);
    return launched("prepare", grid, kThreads);
}
hipError_t launch_ns_gram(const NsArgs& g, int, TileShape, int grid, hipStream_t)
{
    group_args(g);
    in_table(g.sym, sizeof(ProdTile) * grid, g_table_bytes);
    return launched("gram", grid, 576);
}
hipError_t launch_ns_gram_split(const NsArgs& g, int, int grid, hipStream_t)
{
    group_args(g);
    in_table(g.gram, sizeof(ProdTile) * grid, g_table_bytes);
    return launched("gram split", grid, 256);
}
hipError_t launch_ns_poly(const NsArgs& g, TileShape, int grid, hipStream_t)
{
    group_args(g);
    return launched("poly", grid, 576);
}
hipError_t launch_ns_apply(const NsArgs& g, int, bool, NsLast last, const MuonArgs&, TileShape, int grid, hipStream_t)
{
    group_args(g);
    in_table(g.full, sizeof(ProdTile) * grid, g_table_bytes);
    return launched(last == kNsMid ? "apply" : "last", grid, 576);
}
hipError_t launch_thin_gram(const NsArgs& g, int kp, bool, int, int grid, hipStream_t)
{
    group_args(g);
    REQUIRE(kp == 32 || kp == 64 || kp == 128);
    in_table(g.sym, sizeof(ProdTile) * grid, g_table_bytes);
    return launched("thin gram", grid, kThreads);
}
hipError_t launch_thin_sum(const NsArgs& g, int kp, int n, hipStream_t)
{
    group_args(g);
    return launched("thin sum", (int64_t)n * (kp * kp / 4 / kThreads), kThreads);
}
hipError_t launch_thin_poly(const NsArgs& g, int kp, int, int steps, double, NormRec*, int grid, hipStream_t)
{
    group_args(g);
    REQUIRE(steps >= 1 && kp >= 32);
    return launched("thin poly", grid, 512);
}
hipError_t launch_thin_apply(const NsArgs& g, int, bool, int, NsLast last, const MuonArgs&, int grid, hipStream_t)
{
    group_args(g);
    in_table(g.full, sizeof(ProdTile) * grid, g_table_bytes);
    return launched(last == kNsMid ? "thin apply" : "thin last", grid, kThreads);
}
hipError_t launch_thin_one(const NsArgs& g, int kp, bool, int, double, NormRec*, NsLast last, const MuonArgs&, int n,
                           hipStream_t)
{
    group_args(g);
    REQUIRE(kp <= 64 && last != kNsMid);
    return launched("thin one", n, kThreads);
}
}  // namespace z1

// ------------------------------------------------------------------ the table
struct Range {
    int64_t lo, hi;
};

static void check_tiles(const zero1_matrix_plan& p, const MatDesc* mats, const ProdTile* list, const zero1_matrix_group& g,
                        int end, int64_t at, int n, int side, bool sym)
{
    std::set<std::tuple<int, int, int>> seen;   // blocks (i <= j of A when sym)
    for (int t = 0; t < n; ++t) {
        const ProdTile& q = list[at + t];
        REQUIRE(q.mat >= g.first && q.mat < end);
        const MatDesc& d = mats[q.mat];
        const int rows = d.kp / kPad, cols = (sym ? d.kp : d.np) / kPad;
        REQUIRE(q.i >= 0 && q.i < rows && q.j >= 0 && q.j < cols && q.i % side == 0 && q.j % side == 0);
        for (int i = q.i; i < std::min(q.i + side, rows); ++i)
            for (int j = q.j; j < std::min(q.j + side, cols); ++j)
                if (!sym || i <= j) REQUIRE(seen.insert({q.mat, i, j}).second);
    }
    size_t want = 0;
    for (int m = g.first; m < end; ++m) {
        const size_t r = mats[m].kp / kPad, c = mats[m].np / kPad;
        want += sym ? r * (r + 1) / 2 : r * c;
    }
    REQUIRE(seen.size() == want);
    (void)p;
}

static void check_table(const zero1_matrix_plan& p, const std::vector<zero1_matrix>& in)
{
    const char* tb = static_cast<const char*>(p.table);
    const MatDesc* mats = reinterpret_cast<const MatDesc*>(tb);
    const StreamTile* tiles = reinterpret_cast<const StreamTile*>(tb + p.off_tiles);
    const ProdTile* list = reinterpret_cast<const ProdTile*>(tb + p.off_list);
    REQUIRE(p.n_mats == (int)in.size());
    // every matrix once, streaming tiles one after the other over all quads
    std::multiset<std::pair<int64_t, int64_t>> a, b;
    int next = 0, dense = 0;
    for (int m = 0; m < p.n_mats; ++m) {
        const MatDesc& d = mats[m];
        a.insert({d.rows, d.cols});
        b.insert({in[m].rows, in[m].cols});
        REQUIRE(d.tile0 == next && d.n_tiles >= 1);
        REQUIRE((int64_t)d.vrows * d.vcols == d.rows * d.cols && d.qpr == (d.vcols + 3) / 4);
        REQUIRE(d.k == std::min(d.rows, d.cols) && d.n == std::max(d.rows, d.cols));
        REQUIRE((int64_t)(d.n_tiles - 1) * kQuadsPerTile < d.vrows * d.qpr);
        REQUIRE((int64_t)d.n_tiles * kQuadsPerTile >= d.vrows * d.qpr);
        for (int t = 0; t < d.n_tiles; ++t) {
            const StreamTile& s = tiles[next + t];
            REQUIRE(s.mat == m && s.idx == t);
            if (d.vrows > 1) REQUIRE(s.row0 * d.qpr + s.q0 == (int64_t)t * kQuadsPerTile && s.q0 >= 0 && s.q0 < d.qpr);
        }
        next += d.n_tiles;
        if (d.k > kThin) REQUIRE(++dense == m + 1);   // those that are not thin come first
    }
    REQUIRE(a == b && next == p.n_tiles && dense == p.n_dense);
    int most = 0;
    for (int m = 0; m < dense; ++m) most = std::max(most, mats[m].n_tiles);
    REQUIRE(p.dense_most == most);
    REQUIRE(p.dense_tiles == (dense ? mats[dense - 1].tile0 + mats[dense - 1].n_tiles : 0));
    if (!mats[0].u) {
        REQUIRE(p.n_groups == 0);
        return;
    }
    REQUIRE(p.n_groups >= 1 && p.n_groups <= ZERO1_MUON_MAX_GROUPS && p.groups[0].first == 0);
    for (int gi = 0; gi < p.n_groups; ++gi) {
        const zero1_matrix_group& g = p.groups[gi];
        const int end = gi + 1 < p.n_groups ? p.groups[gi + 1].first : p.n_mats;
        REQUIRE(end > g.first);
        std::vector<Range> used;
        int parts = 0, at = 0, cols = 0;
        for (int m = g.first; m < end; ++m) {
            const MatDesc& d = mats[m];
            const int64_t x = (int64_t)d.kp * d.np * 2, sq = (int64_t)d.kp * d.kp * 2;
            if (g.thin) {
                REQUIRE(d.k <= kThin && d.kp == g.thin && d.kp >= d.k && d.np % kPad == 0 && d.np >= d.n);
                REQUIRE(d.n_parts >= 1 && d.n_parts <= kThinMaxParts && d.split % kPad == 0);
                REQUIRE((int64_t)d.n_parts * d.split >= d.n && (int64_t)(d.n_parts - 1) * d.split < d.n);
                parts = std::max(parts, d.n_parts);
                for (int q = 0; q < d.n_parts; ++q, ++at) {
                    const ProdTile& t = list[g.sym0 + at];
                    REQUIRE(t.mat == m && t.i == q && (int64_t)t.j * kPad == (int64_t)q * d.split);
                }
                for (int j = 0; j < d.np / kPad; ++j, ++cols) {
                    const ProdTile& t = list[g.full0 + cols];
                    REQUIRE(t.mat == m && t.j == j);
                }
                if (g.one) REQUIRE(d.n_parts == 1 && d.n <= kThinOne && d.kp <= 64);
                used.push_back({d.x[0], d.x[0] + (int64_t)d.k * d.np * 4});
                used.push_back({d.lo, d.lo + 4 * (kThinMaxParts + 1)});
                used.push_back({d.a, d.a + (int64_t)d.n_parts * d.kp * d.kp * 4});
                used.push_back({d.b, d.b + 2 * (int64_t)d.kp * d.kp * 2});
            } else {
                REQUIRE(d.k > kThin && d.kp % kPad == 0 && d.kp >= d.k && d.np >= d.n);
                REQUIRE(g.split == (d.kp / kPad <= kSplitRows && d.np / kPad >= kSplitInner));
                used.push_back({d.x[0], d.x[0] + x});
                used.push_back({d.x[1], d.x[1] + x});
                used.push_back({d.lo, d.lo + x});
                used.push_back({d.a, d.a + sq});
                used.push_back({d.b, d.b + sq});
            }
        }
        std::sort(used.begin(), used.end(), [](const Range& r, const Range& s) { return r.lo < s.lo; });
        for (size_t r = 0; r < used.size(); ++r) {
            REQUIRE(used[r].lo >= 0 && used[r].lo % 256 == 0 && used[r].hi <= p.area_bytes);
            REQUIRE(r == 0 || used[r].lo >= used[r - 1].hi);
        }
        if (g.thin) {
            REQUIRE(parts == g.parts && at == g.n_sym && cols == g.n_full && g.n_blocks == end - g.first);
        } else {
            check_tiles(p, mats, list, g, end, g.sym0, g.n_sym, g.sym_tile + 2, true);
            check_tiles(p, mats, list, g, end, g.full0, g.n_full, g.full_tile + 2, false);
            check_tiles(p, mats, list, g, end, g.blocks0, g.n_blocks, 1, false);
            if (g.split) check_tiles(p, mats, list, g, end, g.gram0, g.n_gram, 1, true);
            splits += g.split;
        }
    }
}

// What a call launches for the plan's groups, in order.
static std::vector<std::string> expected(const zero1_matrix_plan& p, int steps, int segments)
{
    std::vector<std::string> e;
    if (p.dense_most > kNormTiles) e.push_back("norms");
    for (int gi = 0; gi < p.n_groups; ++gi) {
        const zero1_matrix_group& g = p.groups[gi];
        if (g.thin && g.one && segments == 1) {
            e.push_back("thin one");
        } else if (g.thin) {
            for (int s = 0; s < segments; ++s) {
                e.push_back("thin gram");
                if (g.parts > 1) e.push_back("thin sum");
                e.push_back("thin poly");
                e.push_back(s + 1 == segments ? "thin last" : "thin apply");
            }
        } else {
            e.push_back("prepare");
            for (int s = 0; s < steps; ++s) {
                e.push_back(g.split ? "gram split" : "gram");
                e.push_back("poly");
                e.push_back(s + 1 == steps ? "last" : "apply");
            }
        }
    }
    return e;
}

int main()
{
    std::mt19937_64 rng(12345);
    auto pick = [&](int64_t lo, int64_t hi) { return lo + (int64_t)(rng() % (uint64_t)(hi - lo + 1)); };
    const int64_t edges[] = {1, 2, 3, 4, 31, 32, 33, 63, 64, 65, 127, 128, 129, 192, 255, 256, 257, 511, 513};
    int64_t widest = 0;
    int large = 0;
    for (g_case = 0; g_case < 400; ++g_case) {
        const int n = (int)pick(1, g_case % 10 == 0 ? 60 : 8);
        const bool no_u = g_case % 13 == 5;
        std::vector<zero1_matrix> mats;
        uintptr_t at = (uintptr_t)1 << 40;
        for (int i = 0; i < n; ++i) {
            zero1_matrix q;
            std::memset(&q, 0, sizeof q);
            auto side = [&]() { return rng() % 2 ? edges[rng() % 19] : pick(1, g_case % 7 == 0 ? 3000 : 700); };
            q.rows = side();
            q.cols = side();
            if (g_case % 11 == 3 && i == 0) (rng() % 2 ? q.rows : q.cols) = pick(1, 3) << 20;
            q.ld = rng() % 2 ? 0 : q.cols + pick(0, 9);
            q.ldu = rng() % 2 ? 0 : q.cols + pick(0, 9);
            q.ldo = rng() % 2 ? 0 : q.cols + pick(0, 9);
            q.scale = 1.0f;
            auto take = [&](int64_t ld) {
                const uintptr_t p = at;
                at += ((uintptr_t)q.rows * (ld ? ld : q.cols) * 4 + 4095) / 4096 * 4096;
                return p;
            };
            q.param_bf16 = reinterpret_cast<uint16_t*>(take(q.ld));
            q.master = reinterpret_cast<float*>(take(q.ld));
            if (!no_u) {
                q.m = reinterpret_cast<void*>(take(q.ld));
                q.u = reinterpret_cast<void*>(take(q.ldu));
            }
            q.o = reinterpret_cast<uint16_t*>(take(q.ldo));
            mats.push_back(q);
            widest = std::max(widest, std::max(q.rows, q.cols));
        }
        const uint32_t flags = rng() % 2 ? ZERO1_U_F32 : 0;
        const size_t need = zero1_muon_table_bytes(mats.data(), n);
        REQUIRE(need > 0);
        char* table = static_cast<char*>(std::aligned_alloc(256, (need + 255) / 256 * 256));
        zero1_matrix_plan plan;
        REQUIRE(zero1_muon_plan(mats.data(), n, flags, table, need, &plan) == ZERO1_OK);
        g_plan = &plan;
        g_table_bytes = need;
        g_norms_first = plan.dense_most > kNormTiles;
        large += g_norms_first;
        check_table(plan, mats);

        g_ws = reinterpret_cast<char*>((uintptr_t)1 << 41);   // (nothing touches it here)
        const size_t ws = zero1_muon_workspace_bytes(&plan);
        g_ws_end = g_ws + ws;
        zero1_muon_hparams hp;
        std::memset(&hp, 0, sizeof hp);
        hp.lr = 1e-3;
        hp.momentum = 0.9;
        hp.max_norm = 1.0;
        hp.ns_a = 3.4445;
        hp.ns_b = -4.7750;
        hp.ns_c = 2.0315;
        hp.ns_eps = 1e-7;
        // five default steps are one segment (growth 3.44^4 <= 160), twelve three
        for (int steps : {1, 5, 6, 12}) {
            hp.ns_steps = steps;
            const int segments = (steps + 4) / 5;
            const uint16_t* grads[2] = {reinterpret_cast<uint16_t*>(4096), reinterpret_cast<uint16_t*>(8192)};
            g_log.clear();
            if (no_u) {
                REQUIRE(zero1_orthogonalize(&plan, &hp, 0, g_ws, ws, nullptr) == ZERO1_EINVAL);
                REQUIRE(zero1_muon_update(&plan, &hp, 0, nullptr) == ZERO1_OK);
                REQUIRE(g_log == std::vector<std::string>{"update"});
                continue;
            }
            std::vector<std::string> want = expected(plan, steps, segments), w = want;
            REQUIRE(zero1_orthogonalize(&plan, &hp, 0, g_ws, ws, nullptr) == ZERO1_OK);
            if (plan.n_dense) w.insert(w.begin(), "sumsq");
            REQUIRE(g_log == w);
            g_log.clear();
            w = want;
            REQUIRE(zero1_muon_step(grads, 2, 0, &plan, &hp, nullptr, 0, 0, nullptr, g_ws, ws, nullptr) == ZERO1_OK);
            w.insert(w.begin(), "momentum");
            REQUIRE(g_log == w);
            g_log.clear();
            REQUIRE(zero1_muon_step(grads, 2, 0, &plan, &hp, nullptr, 0, 0, nullptr, g_ws, ws - 1, nullptr) ==
                    ZERO1_EWORKSPACE);
            REQUIRE(g_log.empty());
        }
        std::free(table);
    }
    REQUIRE(widest >= 1 << 20 && large >= 10 && splits >= 10);
    std::printf("all ok\n");
    return 0;
}
