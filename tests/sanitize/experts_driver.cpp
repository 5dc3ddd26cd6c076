// Calls the C entries around a MoE layer's own experts with arguments that
// their host-side checks must reject, and their size functions over a grid of
// sizes, for an AddressSanitizer / UndefinedBehaviorSanitizer build of the host
// code.  The kernel launchers are replaced by stubs that abort: reaching one
// fails.
#include <math.h>
#include <stdio.h>
#include <stdlib.h>

#include <initializer_list>

#include "moe_exl3.h"

#define CHECK(c) do { if (!(c)) { fprintf(stderr, "check failed: %s (line %d)\n", #c, __LINE__); return 1; } } while (0)

int main()
{
    // never read: addresses far apart
    char *at = (char *)(uintptr_t)0x100000000000u;
    auto p = [&](int i) { return (void *)(at + ((int64_t)i << 40)); };
    auto q = [&](int i) { return (int32_t *)p(i); };
    auto f = [&](int i) { return (float *)p(i); };
    const size_t big = (size_t)1 << 44;
    for (int32_t E : {1, 7, 1024})
        for (int32_t k : {1, 8, 16}) {
            const moe_exl3_tokens_desc d = {4096, E, k, MOE_EXL3_DT_BF16};
            size_t last = 0;
            for (int64_t T : {(int64_t)0, (int64_t)1, (int64_t)300, (int64_t)16384, (int64_t)INT32_MAX / 16, (int64_t)INT32_MAX,
                              (int64_t)1 << 40, INT64_MAX}) {
                size_t n = 0;
                const int rc = moe_exl3_sort_workspace_size(&d, T, &n);
                CHECK(rc == (T <= INT32_MAX / k ? MOE_EXL3_OK : MOE_EXL3_ERR_UNSUPPORTED));
                if (rc)
                    continue;
                CHECK(n >= last);
                last = n;
                CHECK(moe_exl3_sort(&d, q(0), T, q(1), q(2), q(3), q(4), p(5), n - 1, nullptr) == MOE_EXL3_ERR_WORKSPACE);
            }
        }
    for (int32_t K : {32, 1376, 65536})
        for (int32_t N : {8, 1032, 65528}) {
            const moe_exl3_w4_desc d = {K, N, 5, 32, MOE_EXL3_DT_F16, MOE_EXL3_ACT_SILU};
            const moe_exl3_w4 w = {p(1), p(2), (const uint8_t *)p(3)};
            for (int64_t R : {(int64_t)1, (int64_t)64, (int64_t)16384, (int64_t)1 << 31, (int64_t)1 << 62}) {
                size_t n = 0;
                const int rc = moe_exl3_w4_workspace_size(&d, R, &n);
                CHECK(rc == MOE_EXL3_OK || rc == MOE_EXL3_ERR_UNSUPPORTED);
                if (rc == MOE_EXL3_OK) {
                    CHECK(moe_exl3_w4_linear(&d, p(0), K, &w, q(4), nullptr, 0, R, p(6), N, p(7), n - 1, nullptr) ==
                          MOE_EXL3_ERR_WORKSPACE);
                    CHECK(moe_exl3_w4_glu(&d, p(0), K, &w, &w, q(4), R, p(6), N, p(7), n - 1, nullptr) ==
                          MOE_EXL3_ERR_WORKSPACE);
                } else {
                    CHECK(moe_exl3_w4_linear(&d, p(0), K, &w, q(4), nullptr, 0, R, p(6), N, p(7), big, nullptr) ==
                          MOE_EXL3_ERR_UNSUPPORTED);
                }
            }
        }
    const moe_exl3_tokens_desc d = {512, 40, 4, MOE_EXL3_DT_F16};
    const moe_exl3_w4_desc e = {512, 256, 4, 64, MOE_EXL3_DT_F16, MOE_EXL3_ACT_SILU};
    const moe_exl3_w4 w = {p(1), p(2), nullptr};
    for (int64_t v : {INT64_MIN, (int64_t)-1, INT64_MAX, (int64_t)1 << 40}) {
        const moe_exl3_drop drop = {0.5, (const uint64_t *)p(9)};
        CHECK(moe_exl3_sort(&d, q(0), v, q(1), q(2), q(3), q(4), p(5), big, nullptr) != MOE_EXL3_OK);
        CHECK(moe_exl3_dispatch(&d, p(0), 512, q(1), f(2), v, 32, p(3), 512, nullptr) != MOE_EXL3_OK);
        CHECK(moe_exl3_dispatch(&d, p(0), 512, q(1), f(2), 8, v, p(3), 512, nullptr) != MOE_EXL3_OK);
        CHECK(moe_exl3_dispatch(&d, p(0), v, q(1), f(2), 8, 32, p(3), 512, nullptr) != MOE_EXL3_OK);
        CHECK(moe_exl3_dispatch_backward(&d, p(0), 512, p(1), 512, q(2), f(3), v, 32, p(4), 512, f(5), nullptr) != MOE_EXL3_OK);
        CHECK(moe_exl3_dispatch_backward(&d, p(0), v, p(1), 512, q(2), f(3), 8, 32, p(4), 512, f(5), nullptr) != MOE_EXL3_OK);
        CHECK(moe_exl3_combine(&d, p(0), 512, q(1), f(2), p(3), 512, &drop, 8, v, p(5), 512, nullptr) != MOE_EXL3_OK);
        CHECK(moe_exl3_combine(&d, p(0), 512, q(1), f(2), p(3), v, &drop, 8, 32, p(5), 512, nullptr) != MOE_EXL3_OK);
        CHECK(moe_exl3_combine_backward(&d, p(0), 512, p(1), 512, q(2), f(3), &drop, v, 32, p(5), 512, f(6), nullptr) !=
              MOE_EXL3_OK);
        CHECK(moe_exl3_combine_backward(&d, p(0), 512, p(1), 512, q(2), f(3), &drop, 8, 32, p(5), v, f(6), nullptr) !=
              MOE_EXL3_OK);
        CHECK(moe_exl3_dropout(MOE_EXL3_DT_F32, p(0), 512, nullptr, 0, &drop, v, 512, p(1), 512, nullptr) != MOE_EXL3_OK);
        CHECK(moe_exl3_dropout(MOE_EXL3_DT_F32, p(0), 512, nullptr, 0, &drop, 8, v, p(1), 512, nullptr) != MOE_EXL3_OK);
        CHECK(moe_exl3_dropout(MOE_EXL3_DT_F32, p(0), v, nullptr, 0, &drop, 8, 512, p(1), 512, nullptr) != MOE_EXL3_OK);
        CHECK(moe_exl3_w4_linear(&e, p(0), 512, &w, q(3), nullptr, 0, v, p(4), 256, p(5), big, nullptr) != MOE_EXL3_OK);
        CHECK(moe_exl3_w4_linear(&e, p(0), v, &w, q(3), nullptr, 0, 8, p(4), 256, p(5), big, nullptr) != MOE_EXL3_OK);
        CHECK(moe_exl3_w4_glu(&e, p(0), 512, &w, &w, q(3), 8, p(4), v, p(5), big, nullptr) != MOE_EXL3_OK);
    }
    for (double v : {-1e-300, 1.0000001, (double)NAN, (double)INFINITY, -(double)INFINITY}) {
        const moe_exl3_drop drop = {v, (const uint64_t *)p(9)};
        CHECK(moe_exl3_dropout(MOE_EXL3_DT_F32, p(0), 512, nullptr, 0, &drop, 8, 512, p(1), 512, nullptr) ==
              MOE_EXL3_ERR_INVALID_ARG);
    }
    printf("experts driver: ok\n");
    return 0;
}
