// The 8-bit matrices' entry points, checked without a GPU: f8_api.cpp linked with
// the stand-ins below for the HIP runtime and the kernels' launchers.  Over random
// shapes up to the ends of the ranges, every launch has to get what its kernel
// assumes: parts that cover the summed axis, grids within the limits, offsets that
// fit 32 bits, a workspace of its own size, alignment where it is claimed.
#include <hip/hip_runtime.h>

#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <random>
#include <string>

#include "../../include/zero1.h"
#include "../../zero_sharded_mixed_zero1_amd/csrc/f8.h"

using namespace z1;

#define REQUIRE(cond)                                                                \
    do {                                                                             \
        if (!(cond)) {                                                               \
            std::printf("%s:%d: %s (case %d)\n", __FILE__, __LINE__, #cond, g_case); \
            std::exit(1);                                                            \
        }                                                                            \
    } while (0)

static int g_case = 0;

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
const char* hipGetErrorString(hipError_t) { return "error"; }
hipError_t hipGetLastError(void) { return hipSuccess; }
hipError_t hipStreamIsCapturing(hipStream_t, hipStreamCaptureStatus*) { return hipSuccess; }
hipError_t hipStreamSynchronize(hipStream_t) { return hipSuccess; }
}

static std::string g_error;
static int g_quantized, g_multiplied, g_kinds[4], g_parts, g_bands[5];
static uintptr_t g_ws, g_ws_end;

namespace z1 {
int set_error(int st, const char* msg) { g_error = msg; return st; }

static int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

static void matrix(const F8& m)
{
    REQUIRE(m.ld % 16 == 0 && m.ld >= ceil_div(m.cols, 128) * 128 && 255 * m.ld + 127 < (int64_t)1 << 32);
    REQUIRE(m.ld_scales % 4 == 0 && m.ld_scales >= ceil_div(m.cols, 128) && 255 * m.ld_scales < (int64_t)1 << 32);
    REQUIRE(m.shift == 0 || m.shift == 7);
    REQUIRE((uintptr_t)m.codes % 16 == 0 && (uintptr_t)m.scales % 4 == 0);
}

hipError_t launch_f8_quantize(const void* src, bool, int64_t rows, int64_t cols, int64_t ld, const F8& q, const F8& qt,
                              hipStream_t)
{
    ++g_quantized;
    REQUIRE(src && rows > 0 && cols > 0 && ld >= cols && (q.codes || qt.codes));
    REQUIRE(ceil_div(rows, 128) * ceil_div(cols, 128) * 256 < (int64_t)1 << 32);
    if (q.codes) { matrix(q); REQUIRE(q.rows == rows && q.cols == cols); }
    if (qt.codes) { matrix(qt); REQUIRE(qt.rows == cols && qt.cols == rows); }
    return hipSuccess;
}

hipError_t launch_f8_product(const F8Product& p, hipStream_t)
{
    ++g_multiplied;
    const int64_t m = p.a.rows, n = p.b.rows, blocks = ceil_div(p.a.cols, 128);
    REQUIRE(m > 0 && n > 0 && p.a.cols == p.b.cols && p.d && p.ldd >= n);
    matrix(p.a);
    matrix(p.b);
    const int64_t eb = p.f32 ? 4 : 2;
    REQUIRE(!p.vec || ((uintptr_t)p.d % 16 == 0 && p.ldd * eb % 16 == 0));
    REQUIRE(p.parts >= 1 && p.part_steps >= 1 && (int64_t)p.parts * p.part_steps >= blocks);
    REQUIRE(p.parts == 1 || (int64_t)(p.parts - 1) * p.part_steps < blocks);   // each part has something
    int64_t groups = 0, threads = 256;
    ++g_kinds[p.kind];
    if (p.kind == kF8Thin) {
        REQUIRE(m <= 32 && p.parts == 1);
        groups = ceil_div(n, 32);
    } else if (p.kind == kF8Tile64 || p.kind == kF8Tile128) {
        const int64_t side = p.kind == kF8Tile64 ? 64 : 128;
        groups = ceil_div(m, side) * ceil_div(n, side) * p.parts;
        if (p.parts > 1) {
            ++g_parts;
            REQUIRE(p.ld_sums >= n && p.ld_sums % 4 == 0 && p.part_elems >= m * p.ld_sums);
            REQUIRE((uintptr_t)p.sums == g_ws && g_ws + 4 * (uintptr_t)(p.parts * p.part_elems) <= g_ws_end);
            REQUIRE(ceil_div(m * ceil_div(n, 4), 256) * 256 < (int64_t)1 << 32);
        }
    } else {
        REQUIRE(p.kind == kF8Tile256 && !p.f32 && p.parts == 1 && (p.bands == 2 || p.bands == 4));
        const int64_t tiles = ceil_div(m, 256) * ceil_div(n, 256);
        REQUIRE(p.whole >= 0 && p.whole <= tiles && (p.whole == tiles || p.whole % 8 == 0));
        ++g_bands[p.whole == tiles ? 1 : p.bands];
        groups = p.whole + (tiles - p.whole) * p.bands;
        threads = 512;
    }
    REQUIRE(groups >= 1 && groups * threads < (int64_t)1 << 32);
    return hipSuccess;
}
}  // namespace z1

int main()
{
    std::mt19937_64 rng(1);
    auto log_int = [&](double lo, double hi) {
        const double u = std::uniform_real_distribution<double>(std::log(lo), std::log(hi))(rng);
        return (int64_t)std::exp(u);
    };
    auto at = [](int k) { return reinterpret_cast<uint8_t*>((uintptr_t)1 << 56 | (uintptr_t)k << 50); };
    int refused = 0;
    for (g_case = 0; g_case < 200000; ++g_case) {
        const bool wide = g_case % 4 == 3;   // up to the ends of the ranges
        int64_t m = log_int(1, wide ? 2147483392.0 : 20000), n = log_int(1, wide ? 2147483392.0 : 20000),
                k = g_case % 50 ? log_int(1, wide ? 8388608.0 : 20000) : 0;
        if (g_case % 3 == 0) { m = (m + 127) / 128 * 128; if (m > 2147483392) m = 2147483392; }
        zero1_f8_matrix a = {m, k, 0, 0, at(0), at(1), rng() % 2 ? 1 : 128, rng() % 2 ? ZERO1_E5M2 : 0};
        zero1_f8_matrix b = {n, k, 0, 0, at(2), at(3), rng() % 2 ? 1 : 128, rng() % 2 ? ZERO1_E5M2 : 0};
        if (rng() % 4 == 0) { a.ld = (k + 127) / 128 * 128 + 16 * (int64_t)(rng() % 9); if (a.ld > 1 << 24) a.ld = 0; }
        const uint32_t flags = rng() % 2 ? ZERO1_F32 : 0;
        const int64_t ldd = rng() % 2 ? 0 : n + (int64_t)(rng() % 9);
        const size_t need = zero1_f8_product_workspace_bytes(&a, &b, flags);
        g_ws = need ? (uintptr_t)at(5) : 0;
        g_ws_end = g_ws + need;
        const int before = g_multiplied;
        zero1_status st = zero1_f8_product(&a, &b, at(4) + 4 * (rng() % 5), ldd, flags, (void*)g_ws, need, nullptr);
        const bool too_many = ((m + 127) / 128) * ((n + 127) / 128) > (int64_t)1 << 21;
        REQUIRE(st == (too_many ? ZERO1_EINVAL : ZERO1_OK) && g_multiplied == before + (too_many ? 0 : 1));
        refused += too_many;
        if (need && !too_many) {   // one byte less, misaligned, none
            REQUIRE(zero1_f8_product(&a, &b, at(4), ldd, flags, (void*)g_ws, need - 1, nullptr) == ZERO1_EWORKSPACE);
            REQUIRE(zero1_f8_product(&a, &b, at(4), ldd, flags, (void*)(g_ws + 8), need, nullptr) == ZERO1_EWORKSPACE);
            REQUIRE(zero1_f8_product(&a, &b, at(4), ldd, flags, nullptr, need, nullptr) == ZERO1_EWORKSPACE);
            REQUIRE(g_multiplied == before + 1);
        }
        // quantize: rows up to 2^23 where the transpose is asked for
        int64_t rows = m < (1 << 23) ? m : 1 << 23, cols = k;
        zero1_f8_matrix q = a, qt = {cols, rows, 0, 0, at(6), at(7), 1, 0};
        q.rows = rows;
        q.codes = at(0);
        const int qb = g_quantized;
        const int64_t tiles = ((rows + 127) / 128) * ((cols + 127) / 128);
        st = zero1_f8_quantize(at(8), rows, cols, 0, g_case % 5 ? &q : nullptr, g_case % 7 && g_case % 5 ? nullptr : &qt, flags, nullptr);
        REQUIRE(st == (tiles > 1 << 23 ? ZERO1_EINVAL : ZERO1_OK) && g_quantized == qb + (tiles > 0 && tiles <= 1 << 23 ? 1 : 0));
    }
    REQUIRE(refused > 100 && g_kinds[0] && g_kinds[1] && g_kinds[2] && g_kinds[3] && g_parts && g_bands[1] && g_bands[2] && g_bands[4]);
    std::printf("kinds %d %d %d %d parts %d bands %d %d %d refused %d\nall ok\n", g_kinds[0], g_kinds[1], g_kinds[2], g_kinds[3], g_parts,
                g_bands[1], g_bands[2], g_bands[4], refused);
    return 0;
}
