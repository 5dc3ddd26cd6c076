// Internal launcher of the products with 4-bit weights, shared with their host
// entry points.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "moe_exl3.h"
#include "w4_plan.h"

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
    // a launch over a list of at most `most` tiles (else NULL)
    const int4 *list;
    const int32_t *count;
    int most;
    int tiles;                 // tiles of columns that a block takes in turn
};

// The two lists of a call (W4Plan), and where they and their lengths go.
struct W4Lists {
    int4 *list[2];
    int32_t *count[2];
    int most[2];            // tiles that they have room for, and one more
    int rows[2];            // of a tile
    float us[2], least_us;  // estimates: a tile of rows in either, the second launch at least
    int limit;              // experts of more rows may go to the second
};

hipError_t launch_w4(bool bf16, bool glu, const W4Args &a, hipStream_t s);

}  // namespace moe
