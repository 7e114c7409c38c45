// f8_api.cpp -- the 8-bit floating point entry points of the C ABI (declared in
// include/zero1.h): argument checks and launches.  No entry point allocates device
// memory or synchronizes (except ZERO1_SYNC_CHECK=1).
#include <hip/hip_runtime.h>

#include <cstdarg>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <mutex>

#include "../../include/zero1.h"
#include "f8.h"
#include "internal.h"

using namespace z1;

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

zero1_status current_device(int& cus)
{
    int dev = 0;
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

// ------------------------------------------------------------------ checks
constexpr uint32_t kF8Flags = ZERO1_F32;
constexpr int64_t kMaxRows = ((int64_t)1 << 31) - 256, kMaxCols = (int64_t)1 << 23, kMaxLd = (int64_t)1 << 40;
constexpr int64_t kMaxGrid = (int64_t)1 << 23;   // workgroups of 256: 2^31 threads a launch

int64_t blocks(int64_t n) { return (n + kF8Block - 1) / kF8Block; }
int64_t up(int64_t x, int64_t a) { return (x + a - 1) / a * a; }

zero1_status check_flags(uint32_t flags, const char* fn)
{
    if (flags & ~kF8Flags) return fail(ZERO1_EINVAL, "%s: unknown flag bits 0x%x", fn, flags & ~kF8Flags);
    return ZERO1_OK;
}

// A matrix's fields, with the strides of 0 filled in.
zero1_status check_matrix(const zero1_f8_matrix& m, const char* fn, const char* name, F8& out)
{
    if (m.rows < 0 || m.rows > kMaxRows)
        return fail(ZERO1_EINVAL, "%s: %s.rows=%lld must be in [0, 2^31 - 256]", fn, name, (long long)m.rows);
    if (m.cols < 0 || m.cols > kMaxCols)
        return fail(ZERO1_EINVAL, "%s: %s.cols=%lld must be in [0, 2^23]", fn, name, (long long)m.cols);
    if (m.block_rows != 1 && m.block_rows != kF8Block)
        return fail(ZERO1_EINVAL, "%s: %s.block_rows=%d must be 1 or 128", fn, name, m.block_rows);
    if (m.flags & ~ZERO1_E5M2)
        return fail(ZERO1_EINVAL, "%s: %s: unknown flag bits 0x%x", fn, name, m.flags & ~ZERO1_E5M2);
    const int64_t wide = up(m.cols, kF8Block), per = blocks(m.cols);
    out.ld = m.ld ? m.ld : wide;
    out.ld_scales = m.ld_scales ? m.ld_scales : up(per, 4);
    if (out.ld < wide || out.ld % 16 || out.ld > kMaxCols * 2)
        return fail(ZERO1_EINVAL, "%s: %s.ld=%lld must be a multiple of 16, at least %lld and at most 2^24", fn, name,
                    (long long)out.ld, (long long)wide);
    if (out.ld_scales < per || out.ld_scales % 4 || out.ld_scales > kMaxCols * 2)
        return fail(ZERO1_EINVAL, "%s: %s.ld_scales=%lld must be a multiple of 4, at least %lld and at most 2^24", fn, name,
                    (long long)out.ld_scales, (long long)per);
    if (m.rows > 0 && m.cols > 0) {
        if (!m.codes || !m.scales) return fail(ZERO1_EINVAL, "%s: %s: NULL buffer", fn, name);
        if (reinterpret_cast<uintptr_t>(m.codes) % 16)
            return fail(ZERO1_EINVAL, "%s: %s.codes must be 16-byte aligned", fn, name);
        if (reinterpret_cast<uintptr_t>(m.scales) % 4)
            return fail(ZERO1_EINVAL, "%s: %s.scales must be 4-byte aligned", fn, name);
    }
    out.codes = m.codes;
    out.scales = m.scales;
    out.rows = m.rows;
    out.cols = m.cols;
    out.shift = m.block_rows == 1 ? 0 : 7;
    out.e5m2 = (m.flags & ZERO1_E5M2) ? 1 : 0;
    return ZERO1_OK;
}

struct Range {
    uintptr_t lo, hi;
    const char* what;
};

// The bytes from a matrix's first element to its last; empty where it has none.  Where
// the last lies past the end of the address space (2^63: the kernels' offsets are signed),
// hi is the largest address.
Range range_of(const void* p, int64_t rows, int64_t ld_bytes, int64_t row_bytes, const char* what)
{
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    if (!p || rows <= 0 || row_bytes <= 0) return Range{lo, lo, what};
    const unsigned __int128 hi = lo + (unsigned __int128)(rows - 1) * (uint64_t)ld_bytes + (uint64_t)row_bytes;
    return Range{lo, hi > (uint64_t)1 << 63 ? UINTPTR_MAX : (uintptr_t)hi, what};
}

Range codes_of(const F8& m, const char* what) { return range_of(m.codes, m.rows, m.ld, up(m.cols, kF8Block), what); }
Range scales_of(const F8& m, const char* what)
{
    return range_of(m.scales, m.rows > 0 ? ((m.rows - 1) >> m.shift) + 1 : 0, m.ld_scales, blocks(m.cols), what);
}

// Every range lies in the address space; none of the first n_out (written) overlaps another.
zero1_status check_disjoint(const char* fn, const Range* r, int n, int n_out)
{
    for (int i = 0; i < n; ++i)
        if (r[i].lo < r[i].hi && r[i].hi == UINTPTR_MAX)
            return fail(ZERO1_EINVAL, "%s: %s reaches past the end of the address space", fn, r[i].what);
    for (int i = 0; i < n_out; ++i)
        for (int j = i + 1; j < n; ++j)
            if (r[i].lo < r[i].hi && r[j].lo < r[j].hi && r[i].lo < r[j].hi && r[j].lo < r[i].hi)
                return fail(ZERO1_EINVAL, "%s: buffers overlap: %s and %s", fn, r[i].what, r[j].what);
    return ZERO1_OK;
}

}  // namespace

extern "C" {

zero1_status zero1_f8_quantize(const void* src, int64_t rows, int64_t cols, int64_t ld, const zero1_f8_matrix* q,
                               const zero1_f8_matrix* qt, uint32_t flags, void* stream)
{
    const char* fn = "zero1_f8_quantize";
    zero1_status st;
    if ((st = check_flags(flags, fn))) return st;
    if (!q && !qt) return fail(ZERO1_EINVAL, "%s: q and qt are both NULL", fn);
    if (rows < 0 || cols < 0) return fail(ZERO1_EINVAL, "%s: rows=%lld and cols=%lld must be >= 0", fn, (long long)rows, (long long)cols);
    F8 fq, ft;
    std::memset(&fq, 0, sizeof fq);
    std::memset(&ft, 0, sizeof ft);
    if (q) {
        if ((st = check_matrix(*q, fn, "q", fq))) return st;
        if (q->rows != rows || q->cols != cols)
            return fail(ZERO1_EINVAL, "%s: q is %lld x %lld, src %lld x %lld", fn, (long long)q->rows, (long long)q->cols,
                        (long long)rows, (long long)cols);
    }
    if (qt) {
        if ((st = check_matrix(*qt, fn, "qt", ft))) return st;
        if (qt->rows != cols || qt->cols != rows)
            return fail(ZERO1_EINVAL, "%s: qt is %lld x %lld, src's transpose %lld x %lld", fn, (long long)qt->rows,
                        (long long)qt->cols, (long long)cols, (long long)rows);
    }
    if (ld == 0) ld = cols;
    const int64_t eb = flags & ZERO1_F32 ? 4 : 2;
    if (ld < cols || ld > kMaxLd) return fail(ZERO1_EINVAL, "%s: ld=%lld must be at least cols=%lld", fn, (long long)ld, (long long)cols);
    if (rows > 0 && cols > 0) {
        if (!src) return fail(ZERO1_EINVAL, "%s: src is NULL", fn);
        if (reinterpret_cast<uintptr_t>(src) % eb) return fail(ZERO1_EINVAL, "%s: src must be aligned to its elements", fn);
    }
    const Range r[5] = {codes_of(fq, "q.codes"), scales_of(fq, "q.scales"), codes_of(ft, "qt.codes"),
                        scales_of(ft, "qt.scales"), range_of(src, rows, ld * eb, cols * eb, "src")};
    if ((st = check_disjoint(fn, r, 5, 4))) return st;
    if (blocks(rows) * blocks(cols) > kMaxGrid) return fail(ZERO1_EINVAL, "%s: more than 2^23 blocks of 128 x 128", fn);
    int cus = 0;
    if ((st = current_device(cus))) return st;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (rows > 0 && cols > 0) Z1_HIP(launch_f8_quantize(src, (flags & ZERO1_F32) != 0, rows, cols, ld, fq, ft, s));
    return finish(s);
}

// What a workgroup takes, in us: a block of 128 of the summed axis where its CU has
// one workgroup and where it has two, and what comes beside the blocks.  From
// products of 64 to 8192 rows by 512 to 11008 by 768 to 11008 on an MI355X; the
// choice is that of the least measured time in all but a few of them, where it is
// within 15 % of that (1024 x 4096 x 4096: tiles of 64 27.7 us, 128 26.3, 256 in bands of
// 64 rows 22.8; 512 x 4096 x 4096: 15.9, 25.0, 20.3; 2048 x 4096 x 4096: 52, 34.7, 34.9;
// 8192 x 11008 x 4096: 607, 407, 326; one session's, another's differ by up to 5 %).
struct TileCost {
    int side;
    double one, two, fixed;
};
static constexpr TileCost kCosts[2][2] = {{{64, 0.26, 0.44, 1.5}, {128, 0.73, 1.04, 2.0}},    // into bf16
                                          {{64, 0.44, 0.70, 1.5}, {128, 0.93, 1.78, 2.0}}};   // into fp32
static constexpr double kBandCost[3] = {1.7, 0.95, 0.64}, kBandFixed[3] = {4.0, 3.0, 2.5};     // 256, 128, 64 rows of 256
static constexpr double kJoinFixed = 3.0, kJoinBytes = 6e6;                                    // us, bytes a us
constexpr int kMaxParts = 16, kChip = 256;   // CUs the rule counts with (it decides speed, not results' bits alone)

// Kernel and parts of a product.
static void choose(F8Product& p)
{
    const int64_t m = p.a.rows, n = p.b.rows, per = blocks(p.a.cols);
    p.parts = 1;
    p.part_steps = (int)(per > 0 ? per : 1);
    p.whole = 0;
    p.bands = 2;
    p.sums = nullptr;
    p.ld_sums = up(n, 4);
    p.part_elems = m * p.ld_sums;
    if (m <= 32 || n == 0) {   // (without rows of B nothing is launched, and no workspace asked for)
        p.kind = kF8Thin;
        return;
    }
    double best = 1e300;
    for (int k = 0; k < 2; ++k) {
        const TileCost& c = kCosts[p.f32][k];
        const int64_t tiles = (m + c.side - 1) / c.side * ((n + c.side - 1) / c.side);
        for (int parts = 1; parts <= kMaxParts; parts *= 2) {
            const int64_t steps = per > 0 ? (per + parts - 1) / parts : 1;
            const int64_t groups = tiles * (per > 0 ? (per + steps - 1) / steps : 1);
            if (groups > kMaxGrid || (parts > 1 && (steps < 2 || tiles * parts > 2 * kChip))) break;
            const double t = groups <= kChip ? steps * c.one + c.fixed
                                             : (double)((groups + 2 * kChip - 1) / (2 * kChip)) * (steps * c.two + c.fixed);
            const double join = parts > 1 ? kJoinFixed + 8.0 * parts * (double)m * (double)n / kJoinBytes : 0.0;
            if (t + join < best) {
                best = t + join;
                p.kind = k == 0 ? kF8Tile64 : kF8Tile128;
                p.part_steps = (int)steps;
                p.parts = (int)(per > 0 ? (per + steps - 1) / steps : 1);
            }
        }
    }
    if (!p.f32) {
        const int64_t tiles = (m + 255) / 256 * ((n + 255) / 256), rest = tiles % kChip;
        const int bands = rest == 0 || rest > kChip / 2 ? 1 : rest > kChip / 4 ? 2 : 4;
        const int64_t whole = bands == 1 ? tiles : tiles - rest;
        double t = (double)((whole + kChip - 1) / kChip) * (per * kBandCost[0] + kBandFixed[0]);
        if (bands > 1) t += per * kBandCost[bands / 2] + kBandFixed[bands / 2];
        if (t < best) {
            p.kind = kF8Tile256;
            p.parts = 1;
            p.part_steps = (int)(per > 0 ? per : 1);
            p.whole = whole;
            p.bands = bands == 1 ? 2 : bands;
        }
    }
}

// Shared checks of the product and its workspace's size.
static zero1_status product_of(const zero1_f8_matrix* a, const zero1_f8_matrix* b, uint32_t flags, const char* fn,
                               F8Product& p)
{
    zero1_status st;
    if ((st = check_flags(flags, fn))) return st;
    if (!a || !b) return fail(ZERO1_EINVAL, "%s: a or b is NULL", fn);
    if ((st = check_matrix(*a, fn, "a", p.a))) return st;
    if ((st = check_matrix(*b, fn, "b", p.b))) return st;
    if (a->cols != b->cols)
        return fail(ZERO1_EINVAL, "%s: a has %lld columns, b %lld", fn, (long long)a->cols, (long long)b->cols);
    p.f32 = (flags & ZERO1_F32) ? 1 : 0;
    p.d = nullptr;
    p.ldd = b->rows;
    p.vec = 0;
    choose(p);
    return ZERO1_OK;
}

size_t zero1_f8_product_workspace_bytes(const zero1_f8_matrix* a, const zero1_f8_matrix* b, uint32_t flags)
{
    F8Product p;
    if (product_of(a, b, flags, "zero1_f8_product_workspace_bytes", p)) return 0;
    return p.parts > 1 ? (size_t)p.parts * (size_t)p.part_elems * sizeof(float) : 0;
}

zero1_status zero1_f8_product(const zero1_f8_matrix* a, const zero1_f8_matrix* b, void* d, int64_t ldd, uint32_t flags,
                              void* ws, size_t ws_bytes, void* stream)
{
    const char* fn = "zero1_f8_product";
    zero1_status st;
    F8Product p;
    if ((st = product_of(a, b, flags, fn, p))) return st;
    const int64_t eb = p.f32 ? 4 : 2;
    if (ldd == 0) ldd = p.b.rows;
    if (ldd < p.b.rows || ldd > kMaxLd)
        return fail(ZERO1_EINVAL, "%s: ldd=%lld must be at least b's rows, %lld", fn, (long long)ldd, (long long)p.b.rows);
    if (p.a.rows > 0 && p.b.rows > 0) {
        if (!d) return fail(ZERO1_EINVAL, "%s: d is NULL", fn);
        if (reinterpret_cast<uintptr_t>(d) % eb) return fail(ZERO1_EINVAL, "%s: d must be aligned to its elements", fn);
    }
    const Range r[5] = {range_of(d, p.a.rows, ldd * eb, p.b.rows * eb, "d"), codes_of(p.a, "a.codes"),
                        scales_of(p.a, "a.scales"), codes_of(p.b, "b.codes"), scales_of(p.b, "b.scales")};
    if ((st = check_disjoint(fn, r, 5, 1))) return st;
    if (blocks(p.a.rows) * blocks(p.b.rows) > kMaxGrid / 4)   // (32 rows of B a workgroup where A has few)
        return fail(ZERO1_EINVAL, "%s: d has more than 2^21 blocks of 128 x 128", fn);
    int cus = 0;
    if ((st = current_device(cus))) return st;
    p.d = d;
    p.ldd = ldd;
    if (p.parts > 1) {
        const size_t need = (size_t)p.parts * (size_t)p.part_elems * sizeof(float);
        if (!ws) return fail(ZERO1_EWORKSPACE, "workspace is NULL (need %zu bytes)", need);
        if (reinterpret_cast<uintptr_t>(ws) % 256) return fail(ZERO1_EWORKSPACE, "workspace must be 256-byte aligned");
        if (ws_bytes < need) return fail(ZERO1_EWORKSPACE, "workspace has %zu bytes, needs %zu", ws_bytes, need);
        const Range w[6] = {range_of(ws, 1, 0, (int64_t)need, "workspace"), r[0], r[1], r[2], r[3], r[4]};
        if ((st = check_disjoint(fn, w, 6, 1))) return st;
        p.sums = static_cast<float*>(ws);
    }
    p.vec = reinterpret_cast<uintptr_t>(d) % 16 == 0 && ldd * eb % 16 == 0;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (p.a.rows > 0 && p.b.rows > 0) Z1_HIP(launch_f8_product(p, s));
    return finish(s);
}

}  // extern "C"
