// Calls the dense operators' C entries with arguments their host-side checks
// must reject, and their size functions over a grid of shapes, for an
// AddressSanitizer / UndefinedBehaviorSanitizer build of the host code.  The
// kernel launchers are replaced by stubs that abort: reaching one fails.
#include <stdio.h>
#include <stdlib.h>

#include <initializer_list>

#include "moe_exl3.h"

#define CHECK(c) do { if (!(c)) { fprintf(stderr, "check failed: %s (line %d)\n", #c, __LINE__); return 1; } } while (0)

int main()
{
    // never read: addresses far apart
    char *at = (char *)(uintptr_t)0x100000000000u;
    auto p = [&](int i) { return (void *)(at + ((int64_t)i << 36)); };
    const size_t big = (size_t)1 << 44;
    const int64_t sizes[] = {8, 16, 264, 1032, 4096, 65536};
    for (int64_t a : sizes)
        for (int64_t b : sizes) {
            moe_exl3_glu_desc g = {(int32_t)a, (int32_t)b, MOE_EXL3_DT_F16, MOE_EXL3_ACT_SILU};
            moe_exl3_lora_desc l = {(int32_t)a, (int32_t)b, 3, 40, MOE_EXL3_DT_BF16};
            size_t last[3] = {};
            for (int64_t T : {0, 1, 15, 64, 65, 128, 1000, 16384, 200000, 100000000}) {
                size_t n[3] = {};
                const int rc[3] = {moe_exl3_glu_workspace_size(&g, T, &n[0]),
                                   moe_exl3_glu_backward_workspace_size(&g, T, &n[1]),
                                   moe_exl3_lora_workspace_size(&l, T, &n[2])};
                for (int i = 0; i < 3; ++i) {
                    CHECK(rc[i] == MOE_EXL3_OK || rc[i] == MOE_EXL3_ERR_UNSUPPORTED);
                    CHECK(rc[i] != MOE_EXL3_OK || n[i] >= last[i]);
                    if (rc[i] == MOE_EXL3_OK)
                        last[i] = n[i];
                }
                if (rc[1] != MOE_EXL3_OK)
                    continue;
                // the plans of every size, stopped by a workspace one byte short
                if (T > 0) {
                    CHECK(moe_exl3_glu(&g, p(0), a, p(1), p(2), T, p(3), b, (float *)p(4), p(5), n[0] - 1, nullptr) ==
                          MOE_EXL3_ERR_WORKSPACE);
                    moe_exl3_lora_adapters ad = {p(1), p(2), nullptr, nullptr};
                    if (rc[2] == MOE_EXL3_OK)
                        CHECK(moe_exl3_lora_linear(&l, p(0), a, nullptr, &ad, (int32_t *)p(6), nullptr, 0, T, p(3), b,
                                                   p(5), n[2] - 1, nullptr) == MOE_EXL3_ERR_WORKSPACE);
                }
                CHECK(moe_exl3_glu_backward(&g, p(0), a, p(1), p(2), (float *)p(4), p(3), b, T, p(6), a, p(7), p(8), p(5),
                                            n[1] - 1, nullptr) == MOE_EXL3_ERR_WORKSPACE);
            }
        }
    moe_exl3_glu_desc g = {512, 256, MOE_EXL3_DT_BF16, MOE_EXL3_ACT_GELU_TANH};
    moe_exl3_lora_desc l = {512, 256, 4, 16, MOE_EXL3_DT_BF16};
    const moe_exl3_lora_adapters ad = {p(1), p(2), nullptr, nullptr};
    const int64_t edges[] = {INT64_MIN, -1, INT64_MAX, (int64_t)1 << 40};
    for (int64_t v : edges) {
        // token counts and row strides far out of range
        CHECK(moe_exl3_glu(&g, p(0), 512, p(1), p(2), v, p(3), 256, nullptr, p(5), big, nullptr) != MOE_EXL3_OK);
        CHECK(moe_exl3_glu(&g, p(0), v, p(1), p(2), 8, p(3), 256, nullptr, p(5), big, nullptr) != MOE_EXL3_OK);
        CHECK(moe_exl3_glu(&g, p(0), 512, p(1), p(2), 8, p(3), v, nullptr, p(5), big, nullptr) != MOE_EXL3_OK);
        CHECK(moe_exl3_glu_backward(&g, p(0), 512, p(1), p(2), (float *)p(4), p(3), 256, v, p(6), 512, p(7), p(8), p(5),
                                    big, nullptr) != MOE_EXL3_OK);
        CHECK(moe_exl3_glu_backward(&g, p(0), 512, p(1), p(2), (float *)p(4), p(3), v, 8, p(6), 512, p(7), p(8), p(5),
                                    big, nullptr) != MOE_EXL3_OK);
        CHECK(moe_exl3_lora_linear(&l, p(0), 512, p(4), &ad, (int32_t *)p(6), nullptr, 0, v, p(3), 256, p(5), big,
                                   nullptr) != MOE_EXL3_OK);
        CHECK(moe_exl3_lora_linear(&l, p(0), v, p(4), &ad, (int32_t *)p(6), nullptr, 0, 8, p(3), 256, p(5), big,
                                   nullptr) != MOE_EXL3_OK);
        CHECK(moe_exl3_lora_linear(&l, p(0), 512, p(4), &ad, (int32_t *)p(6), p(7), v, 8, p(3), 256, p(5), big,
                                   nullptr) != MOE_EXL3_OK);
        size_t n = 0;
        CHECK(moe_exl3_glu_workspace_size(&g, v, &n) != MOE_EXL3_OK);
        CHECK(moe_exl3_glu_backward_workspace_size(&g, v, &n) != MOE_EXL3_OK);
        CHECK(moe_exl3_lora_workspace_size(&l, v, &n) != MOE_EXL3_OK);
    }
    printf("dense driver: ok\n");
    return 0;
}
