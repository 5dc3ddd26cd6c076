// Prints the launches that the 4-bit products plan for calls read from stdin, a
// line each: rows, K, N, experts, group, zeros, gated pair.  A launch is its
// tile's rows and columns, its wavefronts, tiles of columns a block, tiles of rows
// and blocks; with lists the crowded experts' launch comes last.  Checks what the
// kernels and the workspace rely on, and fails on the first call that breaks it.
#include <stdio.h>

#include "w4_plan.h"

#define CHECK(c) do { if (!(c)) { fprintf(stderr, "check failed: %s (line %d)\n", #c, __LINE__); return 1; } } while (0)

int main()
{
    moe::W4Size s;
    int group, zeros, glu;
    while (scanf("%d %d %d %d %d %d %d", &s.R, &s.K, &s.N, &s.E, &group, &zeros, &glu) == 7) {
        s.group_log2 = group == 32 ? 5 : group == 64 ? 6 : 7;
        s.zeros = zeros;
        s.glu = glu;
        const moe::W4Plan p = moe::w4_plan(s);
        const size_t scratch = moe::w4_scratch(s.R, s.E);
        if (p.listed) {
            CHECK(s.R >= moe::kW4Listed && s.E > 1 && p.limit > 0 && p.limit < s.R);
            CHECK(16 + 16 * ((size_t)p.most[0] + 1 + p.most[1] + 1) <= scratch);
        }
        for (int i = 0; i < (p.listed ? 2 : 1); ++i) {
            const moe::W4Launch &l = p.launch[i];
            const int rows[] = {4, 4, 16, 16, 32, 64, 128}, cols[] = {16, 32, 16, 32, 32, 128, 256};
            const int m = rows[l.v], n = glu ? l.v == moe::W4_4x16 || l.v == moe::W4_16x16 ? 16 : cols[l.v] / 2 : cols[l.v];
            CHECK(!glu || (l.v != moe::W4_4x32 && l.v != moe::W4_16x32));
            CHECK(l.waves == (m == 64 ? 4 : m == 128 ? 8 : l.waves) && (l.waves == 4 || l.waves == 8));
            CHECK(l.tiles >= 1 && l.tiles <= 4 && (l.tiles == 1 || m <= 16));
            const unsigned across = (unsigned)((s.N + n * l.tiles - 1) / (n * l.tiles));
            CHECK(l.grid % across == 0 && (uint64_t)l.grid * 64 * l.waves < (uint64_t)1 << 32);
            // blocks for as many tiles of rows as offsets can make: a last one each
            // for experts that have rows (of the second launch: more than the limit)
            const int64_t over = i ? p.limit : 0, experts = s.E == 1 ? 1 : s.R / (over + 1) < s.E ? s.R / (over + 1) : s.E;
            const int64_t most = s.E == 1 ? (s.R + m - 1) / m : s.R / m + experts;
            const int64_t have = l.grid / across;
            CHECK(have >= most);
            if (p.listed)
                CHECK(p.rows[i] == m && p.most[i] >= most);
            printf("%s%d %d %d %d %lld %u", i ? ";" : "", m, n, l.waves, l.tiles, (long long)have, l.grid);
        }
        printf("\n");
    }
    return 0;
}
