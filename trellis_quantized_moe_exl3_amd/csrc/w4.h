// Internal launcher of the products with 4-bit weights, shared with their host
// entry points.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "moe_exl3.h"

namespace moe {

struct W4Args {
    const uint16_t *x;
    int64_t ldx;
    const uint8_t *codes[2];   // [E][N][K/2]; two: a gated pair
    const uint16_t *scales[2]; // [E][N][K/group]
    const uint8_t *zeros[2];   // [E][N][K/group] or NULL: 8
    const int32_t *offsets;    // [E + 1] or NULL: one expert, every row
    const uint16_t *base;      // added rows or NULL
    int64_t ldbase;
    uint16_t *y;
    int64_t ldy;
    int32_t *status;
    int R, K, N, E;
    int group_log2;            // 5, 6 or 7
    int act;                   // of a gated pair
    int32_t *scratch;          // from kW4Listed rows on: w4_scratch() bytes
    // a launch over a list of at most `most` tiles (else NULL), of experts with more
    // than `over` rows
    const int4 *list;
    const int32_t *count;
    int most, over;
    int tiles;                 // tiles of columns that a block takes in turn
};

// Rows from which a call may take two launches over lists of its experts' tiles
// (in one launch each block finds its own tile).
constexpr int kW4Listed = 128;

// The two lists of a call.
struct W4Lists {
    int4 *list[2];
    int32_t *count[2];
    int most[2];            // tiles that they have room for, and one more
    int rows[2];            // of a tile
    float us[2], least_us;  // estimates: a tile of rows in either, the second launch at least
    int limit;              // experts of more rows may go to the second
};

// Bytes of the lists and their lengths: tiles of 4 rows and of 16 at least, one
// for each expert's last rows, one entry to read past the end.
inline size_t w4_scratch(int64_t R, int64_t E)
{
    const int64_t n = E < R ? E : R;
    return R < kW4Listed || E == 1 ? 0 : (size_t)(16 + 16 * (R / 4 + n + 1 + R / 16 + n + 1));
}

hipError_t launch_w4(bool bf16, bool glu, const W4Args &a, hipStream_t s);

}  // namespace moe
