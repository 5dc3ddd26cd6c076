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
    uint32_t xbytes;           // from the first to the last element
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
    int tiles;                 // tiles of columns that a block takes in turn
};

hipError_t launch_w4(bool bf16, bool glu, const W4Args &a, hipStream_t s);

}  // namespace moe
