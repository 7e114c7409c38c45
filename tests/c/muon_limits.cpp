// The Muon plan's sizes at the ends of their range, without a GPU (the stand-ins
// of muon_plans.cpp): no arithmetic on them overflows, and what is beyond a plan is
// refused.  Built with the undefined-behaviour sanitizer.
#define main plans_main
#include "muon_plans.cpp"
#undef main

static zero1_matrix shape(int64_t rows, int64_t cols)
{
    zero1_matrix q;
    std::memset(&q, 0, sizeof q);
    q.rows = rows;
    q.cols = cols;
    q.scale = 1.0f;
    q.u = reinterpret_cast<void*>((uintptr_t)1 << 40);
    return q;
}

int main()
{
    (void)&plans_main;   // (that file's own run)
    const int64_t side = ((int64_t)1 << 31) - 256;
    for (int64_t k : {1, 3, 128, 129, 32768})
        for (int64_t n : {side, side - 1, ((int64_t)1 << 31) - (1 << 26)}) {
            zero1_matrix wide = shape(k, n), tall = shape(n, k);
            g_error.clear();
            REQUIRE(zero1_muon_table_bytes(&wide, 1) == 0 && !g_error.empty());
            REQUIRE(zero1_muon_table_bytes(&tall, 1) == 0 && !g_error.empty());
            // without u there is nothing to iterate, only tiles to stream
            wide.u = nullptr;
            wide.o = reinterpret_cast<uint16_t*>((uintptr_t)1 << 40);
            if (k == 1) REQUIRE(zero1_muon_table_bytes(&wide, 1) > 0);
        }
    // more elements in all than 63 bits count
    std::vector<zero1_matrix> many(600000, shape(8192, side));
    g_error.clear();
    REQUIRE(zero1_muon_table_bytes(many.data(), (int)many.size()) == 0);
    REQUIRE(g_error.find("too many elements") != std::string::npos);
    std::printf("all ok\n");
    return 0;
}
