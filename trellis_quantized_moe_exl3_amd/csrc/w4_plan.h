// What the host chooses for a call of the 4-bit products, from its sizes alone:
// the tiles and the launches.  Plain C++, shared by the launcher and the entry
// points.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>

namespace moe {

// The variants: rows and columns of a tile (of a gated pair half as many columns
// from 32 on).
enum W4Variant { W4_4x16, W4_4x32, W4_16x16, W4_16x32, W4_32x32, W4_64x128, W4_128x256 };

struct W4Size {
    int R, K, N, E;
    int group_log2;   // 5, 6 or 7
    bool zeros;       // of either matrix
    bool glu;
};

// One launch of the product.
struct W4Launch {
    W4Variant v;
    int tiles;       // tiles of columns that a block takes in turn (narrow tiles)
    int waves;       // of a block
    unsigned grid;   // blocks
};

struct W4Plan {
    // the only launch; with `listed` that of a list of tiles, before it the second
    // one of a list of crowded experts' tiles
    bool listed;
    W4Launch launch[2];
    // of the lists: a tile's rows, room for how many of them, estimated us of a tile of
    // rows and at least of the second launch, rows of an expert that may go to it
    int rows[2], most[2];
    float us[2], least_us;
    int limit;
};

// Rows from which a call may take two launches over lists of its experts' tiles
// (in one launch each block finds its own tile).
constexpr int kW4Listed = 128;

// Bytes of the lists and their lengths: tiles of 4 rows and of 16 at least, one
// for each expert's last rows, one entry to read past the end.
inline size_t w4_scratch(int64_t R, int64_t E)
{
    const int64_t n = E < R ? E : R;
    return R < kW4Listed || E == 1 ? 0 : (size_t)(16 + 16 * (R / 4 + n + 1 + R / 16 + n + 1));
}

// Tiles of at most `rows` rows that a launch can have, of experts with more than
// `over` rows.
inline unsigned w4_tiles(const W4Size &s, int rows, int over = 0)
{
    return (unsigned)(s.E > 1 ? s.R / rows + std::min(s.E, s.R / (over + 1)) : (s.R + rows - 1) / rows);
}

// A narrow tile that has its CU to itself gets eight wavefronts for its k and not
// four, if each has 128 k at least (4096 x 4096: 1 row 5.85 us with four, 5.4 with eight,
// 16 rows 6.75, 6.3, 64 rows of group 64 11.0, 9.9; 2048 x 1024: 4.6, 4.2).
inline bool w4_eight(double blocks, int K) { return blocks <= 256 && K >= 1024; }

// Estimates of the variants' time in us: a part that a block takes alone on a CU, and
// one that 256 blocks (one a CU, others beside them) add, each with a part per 128
// k.  Fitted to 1 to 4096 rows of 4096 x 4096, 2048 x 4096 (pairs) and 512 x 8192,
// with four wavefronts to every narrow tile and wide tiles a twentieth slower than now;
// they are there to order the variants, which they do but for near ties.  Measured
// (4096 x 4096, us of the seven in this order, each as it is launched):
//   1 row      5.8   6.8   6.5   7.6   8.8   35   50
//   16        11.5  10.1   6.9   7.8   9.0   35   50
//   64        36    31    15.8  11.6   9.4   35   50
//   256      110    88    46    40    26     36   66
//   1024     402   305   140   112    90     53   66
//   4096    1425  1135   544   425   350    194  147
// and 64 experts of 2048 x 4096 with 256 rows in all: 95, 78, 90, 77, 122, 101, 110;
// with 4096: 866, 693, 352, 287, 300, 168, 167.
struct W4Cost {
    W4Variant v;
    double rows, cols, alone, alone_k, more, more_k;
    int at_once;   // blocks that start together, where a last few cost a round
};

template <bool GLU>
struct W4Estimate {
    // (a pair's narrow tiles have the work of 32 columns)
    static constexpr W4Cost kCosts[] = {
        {W4_4x16, 4, 16, 4.2, 0.065, 0.3, GLU ? 0.085 : 0.05, 1},
        {W4_4x32, 4, 32, 4.1, 0.105, 0.57, 0.07, 1},
        {W4_16x16, 16, 16, 4.8, 0.07, 0.3, GLU ? 0.095 : 0.06, 1},
        {W4_16x32, 16, 32, 4.3, 0.127, 0.7, 0.105, 1},
        {W4_32x32, 32, GLU ? 16 : 32, 4.7, 0.17, 1.7, 0.11, 1},
        {W4_64x128, 64, GLU ? 64 : 128, 4.5, 0.95, 2.0, 0.70, 512},
        {W4_128x256, 128, GLU ? 128 : 256, 6.8, 1.85, 5.7, 2.29, 256},
    };
    int K;
    double k, N, fine;

    explicit W4Estimate(const W4Size &s) : K(s.K), k(s.K / 128.0), N(s.N)
    {
        // finer groups, and zeros, cost the wide tiles' products more
        fine = (s.group_log2 == 5 ? 1.5 : s.group_log2 == 6 ? 1.2 : 1.0) * (s.zeros ? 1.1 : 1.0);
    }
    double steps(const W4Cost &c) const { return (c.rows >= 64 ? fine : 1.0) * k; }
    // 256 blocks' part of what this many tiles of rows cost.
    double more(const W4Cost &c, double tiles) const
    {
        double blocks = tiles * std::ceil(N / c.cols);
        if (c.at_once > 1 && blocks > 256)
            blocks = std::ceil(blocks / c.at_once) * c.at_once;
        return blocks / 256 * (c.more + c.more_k * steps(c));
    }
    // The variant for `rows` rows at each of n experts (half a tile is lost to
    // each one's last rows).
    const W4Cost &best(double n, double rows) const
    {
        const W4Cost *found = nullptr;
        double least = 0;
        for (const W4Cost &c : kCosts) {
            if (GLU && (c.v == W4_4x32 || c.v == W4_16x32))
                continue;
            const double tiles = n > 1 ? n * std::max(1.0, rows / c.rows + 0.5) : std::ceil(rows / c.rows);
            const double part = c.rows < 64 && w4_eight(tiles * std::ceil(N / c.cols), K) ? 0.7 : 1.0;
            const double us = std::max(c.alone + part * c.alone_k * steps(c), 3 + more(c, tiles));
            if (!found || us < least) {
                least = us;
                found = &c;
            }
        }
        return *found;
    }
    // The rows of an expert up to which variant a costs less than b.
    int limit(const W4Cost &a, const W4Cost &b) const
    {
        auto cost = [&](const W4Cost &c, int rows) {
            return std::ceil(rows / c.rows) * std::ceil(N / c.cols) * (c.more + c.more_k * steps(c));
        };
        for (const int rows : {16, 32, 48, 64, 96, 128, 192, 256, 384, 512})
            if (cost(b, rows + 1) < cost(a, rows + 1))
                return rows;
        return INT32_MAX;
    }
};

// The launch of a variant.  Narrow tiles of columns are dealt so that about as many
// blocks are left as the CUs hold at once, but at most four to a block (64 rows of
// 40 experts, 2048 x 4096: 55 us with one each, 43 with two, 39 with four, 42 with
// eight; 64 at 58 experts' pairs of 4096 x 2048: 124, 106, 106, 109; one row, 4096 x
// 4096, whose 256 blocks leave room on each CU: 6.2, 9.1, 14.9, 26.3).  From 16 on
// the wide tiles of rows are rounded up to a multiple of eight, one for each XCD.
inline W4Launch w4_launch(const W4Size &s, const W4Cost &c, int over)
{
    const int rows = (int)c.rows, cols = (int)c.cols;
    const unsigned nt = (unsigned)((s.N + cols - 1) / cols);
    unsigned mt = w4_tiles(s, rows, over);
    if (rows >= 64) {
        if (mt >= 16)
            mt = (mt + 7) / 8 * 8;
        return {c.v, 1, rows == 64 ? 4 : 8, mt * nt};
    }
    const unsigned at_once = cols == 16 && !s.glu ? 1536 : 800;
    const unsigned tiles = rows <= 16 ? std::min(std::max((mt * nt + at_once / 2) / at_once, 1u), std::min(4u, nt)) : 1;
    const unsigned grid = mt * ((nt + tiles - 1) / tiles);
    return {c.v, (int)tiles, w4_eight(grid, s.K) ? 8 : 4, grid};
}

// Of experts the host knows the number alone.  The first variant is the one for
// rows spread over all of them.  From kW4Listed rows on, where another one is better
// for all rows at one expert, a launch in that variant takes the crowded ones if
// there are enough of them (us without and with it: 8071 rows at 3 of 261
// experts, pairs of 1472 x 2000: 678, 184; 348 at 8 of 67, 928 x 6792: 87, 38; 4096 at
// 2 of 256, 2048 x 4096: 252, 128; but with a list and a launch for nothing 256 rows
// spread over 64 experts: 77, 85, 1000: 115, 115).  Fewer rows are always taken as
// spread (100 rows, 4096 x 4096, tiles of 4 rows and of 16: at 100 of 288 experts 173
// us and 253, but at one of them 47 and 30).
template <bool GLU>
W4Plan w4_plan(const W4Size &s)
{
    const W4Estimate<GLU> est(s);
    W4Plan p{};
    const W4Cost &all = est.best(1, s.R);
    if (s.E == 1) {
        p.launch[0] = w4_launch(s, all, 0);
        return p;
    }
    const double n = std::min(s.E, s.R);
    const W4Cost &spread = est.best(n, s.R / n);
    const int limit = est.limit(spread, all);
    if (s.R < kW4Listed || all.rows <= spread.rows || limit >= s.R) {
        p.launch[0] = w4_launch(s, spread, 0);
        return p;
    }
    p.listed = true;
    p.limit = limit;
    p.least_us = (float)(all.alone + all.alone_k * est.steps(all));
    const W4Cost *both[] = {&spread, &all};
    for (int i = 0; i < 2; ++i) {
        const W4Cost &c = *both[i];
        p.rows[i] = (int)c.rows;
        p.us[i] = (float)(std::ceil(est.N / c.cols) / 256 * (c.more + c.more_k * est.steps(c)));
        p.most[i] = (int)w4_tiles(s, p.rows[i]);
        p.launch[i] = w4_launch(s, c, i == 1 ? limit : 0);
    }
    return p;
}

inline W4Plan w4_plan(const W4Size &s) { return s.glu ? w4_plan<true>(s) : w4_plan<false>(s); }

}  // namespace moe
