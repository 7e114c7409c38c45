// The 8-bit matrices' entry points at the edges of what zero1.h allows, checked
// without a GPU: f8_api.cpp linked with the stand-ins below for the HIP runtime and
// the kernels' launchers, which count their calls.
#include <hip/hip_runtime.h>

#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <string>

#include "../../include/zero1.h"
#include "../../zero_sharded_mixed_zero1_amd/csrc/f8.h"

using namespace z1;

#define REQUIRE(cond)                                                                                    \
    do {                                                                                                 \
        if (!(cond)) {                                                                                   \
            std::printf("%s:%d: %s (%s)\n", __FILE__, __LINE__, #cond, g_error.c_str());                 \
            std::exit(1);                                                                                \
        }                                                                                                \
    } while (0)

static std::string g_error;
static int g_quantized, g_multiplied;

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

namespace z1 {
int set_error(int st, const char* msg) { g_error = msg; return st; }
hipError_t launch_f8_quantize(const void*, bool, int64_t, int64_t, int64_t, const F8&, const F8&, hipStream_t)
{
    ++g_quantized;
    return hipSuccess;
}
hipError_t launch_f8_product(const F8Product&, hipStream_t)
{
    ++g_multiplied;
    return hipSuccess;
}
}  // namespace z1

static uint8_t* at(int k) { return reinterpret_cast<uint8_t*>((uintptr_t)1 << 44 | (uintptr_t)k << 40); }

static zero1_f8_matrix matrix(int64_t rows, int64_t cols, int k)
{
    return zero1_f8_matrix{rows, cols, 0, 0, at(2 * k), at(2 * k + 1), 1, 0};
}

// A product without rows is an empty call: no workspace, nothing launched, whatever the
// other sizes.
static void empty_products()
{
    for (int64_t rows : {1, 7, 32, 33, 64, 300, 5000})
        for (int64_t k : {0, 1, 128, 8192, 1 << 23})
            for (uint32_t flags : {0u, (uint32_t)ZERO1_F32}) {
                const zero1_f8_matrix some = matrix(rows, k, 0), none = matrix(0, k, 1);
                g_multiplied = 0;
                REQUIRE(zero1_f8_product_workspace_bytes(&some, &none, flags) == 0);
                REQUIRE(zero1_f8_product_workspace_bytes(&none, &some, flags) == 0);
                REQUIRE(zero1_f8_product(&some, &none, at(8), 0, flags, nullptr, 0, nullptr) == ZERO1_OK);
                REQUIRE(zero1_f8_product(&none, &some, at(8), 0, flags, nullptr, 0, nullptr) == ZERO1_OK);
                REQUIRE(zero1_f8_product(&none, &none, nullptr, 0, flags, nullptr, 0, nullptr) == ZERO1_OK);
                REQUIRE(g_multiplied == 0);
            }
}

// The workspace is written: it may not lie over d or what is read, and need not keep
// clear of anything where it is not used.
static void workspaces()
{
    const zero1_f8_matrix a = matrix(300, 8000, 0), b = matrix(300, 8000, 1);
    const size_t need = zero1_f8_product_workspace_bytes(&a, &b, 0);
    REQUIRE(need > 0 && need % 4 == 0);
    const int64_t ld = 8064, lds = 64;   // (of both: bytes of a row of codes, of scales)
    g_multiplied = 0;
    const struct { uint8_t* p; size_t bytes; const char* what; } others[] = {
        {at(8), 2 * 300 * 300, "d"}, {a.codes, (size_t)(300 * ld), "a.codes"}, {a.scales, (size_t)(300 * lds), "a.scales"},
        {b.codes, (size_t)(300 * ld), "b.codes"}, {b.scales, (size_t)(300 * lds), "b.scales"}};
    for (const auto& o : others) {
        for (uint8_t* ws : {o.p, o.p + 256, o.p + (o.bytes - 256) / 256 * 256, o.p - (need - 1) / 256 * 256}) {
            REQUIRE(zero1_f8_product(&a, &b, at(8), 0, 0, ws, need, nullptr) == ZERO1_EINVAL);
            REQUIRE(g_error.find("overlap") != std::string::npos && g_error.find("workspace") != std::string::npos &&
                    g_error.find(o.what) != std::string::npos);
        }
        // just beside it; and a longer buffer, of which the call takes only what it needs
        REQUIRE(zero1_f8_product(&a, &b, at(8), 0, 0, o.p + (o.bytes + 255) / 256 * 256, need, nullptr) == ZERO1_OK);
        REQUIRE(zero1_f8_product(&a, &b, at(8), 0, 0, o.p - (need + 255) / 256 * 256, need + 4096, nullptr) == ZERO1_OK);
    }
    REQUIRE(g_multiplied == 10);
    const zero1_f8_matrix few = matrix(7, 8000, 0);   // takes none
    REQUIRE(zero1_f8_product(&few, &b, at(8), 0, 0, at(8), 4096, nullptr) == ZERO1_OK && g_multiplied == 11);
}

// Strides and rows within their limits whose product passes 64 bits, or the end of the
// address space: no memory is that large, and the index arithmetic would wrap.
static void beyond_any_memory()
{
    const int64_t wide = (int64_t)1 << 40;
    g_quantized = g_multiplied = 0;
    auto refused = [](zero1_status st, const char* what) {
        return st == ZERO1_EINVAL && g_error.find("address space") != std::string::npos && g_error.find(what) != std::string::npos;
    };
    for (uint32_t flags : {0u, (uint32_t)ZERO1_F32}) {
        for (int64_t rows : {(int64_t)1 << 23, ((int64_t)1 << 24) + 1, ((int64_t)1 << 24) + 3, (int64_t)1 << 30}) {
            const zero1_f8_matrix q = matrix(rows, 100, 0);
            REQUIRE(refused(zero1_f8_quantize(at(8), rows, 100, wide, &q, nullptr, flags, nullptr), "src"));
        }
        // rows * ld * element wraps to a few bytes behind 2^64
        const zero1_f8_matrix q = matrix(((int64_t)1 << 26) + 1, 100, 0), qt = matrix(100, ((int64_t)1 << 23) - 5, 1);
        REQUIRE(refused(zero1_f8_quantize(at(8), q.rows, 100, (int64_t)1 << (flags ? 36 : 37), &q, nullptr, flags, nullptr), "src"));
        REQUIRE(refused(zero1_f8_quantize(at(8), qt.cols, 100, wide, nullptr, &qt, flags, nullptr), "src"));
        for (int64_t rows : {(int64_t)1 << 23, ((int64_t)1 << 24) + 1, (int64_t)1 << 28}) {
            const zero1_f8_matrix a = matrix(rows, 256, 0), b = matrix(5, 256, 1);
            REQUIRE(refused(zero1_f8_product(&a, &b, at(8), wide, flags, nullptr, 0, nullptr), " d "));
        }
    }
    zero1_f8_matrix a = matrix(1 << 20, 256, 0), b = matrix(5, 256, 1);
    a.codes = reinterpret_cast<uint8_t*>(~(uintptr_t)0 << 20);
    REQUIRE(refused(zero1_f8_product(&a, &b, at(8), 0, 0, nullptr, 0, nullptr), "a.codes"));
    REQUIRE(refused(zero1_f8_quantize(at(8), a.rows, a.cols, 0, &a, nullptr, 0, nullptr), "q.codes"));
    REQUIRE(g_quantized == 0 && g_multiplied == 0);
    // the widest rows that fit are taken
    a = matrix(1000, 256, 0);
    REQUIRE(zero1_f8_quantize(at(8), 1000, 256, wide, &a, nullptr, ZERO1_F32, nullptr) == ZERO1_OK && g_quantized == 1);
    REQUIRE(zero1_f8_product(&a, &b, at(8), wide, ZERO1_F32, nullptr, 0, nullptr) == ZERO1_OK && g_multiplied == 1);
}

int main()
{
    empty_products();
    workspaces();
    beyond_any_memory();
    std::printf("all ok\n");
    return 0;
}
