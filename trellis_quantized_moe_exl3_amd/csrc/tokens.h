// Internal launchers of the operators around a MoE layer's experts (tokens
// sorted by expert and back, dropout), shared with their host entry points.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "moe_exl3.h"

namespace moe {

constexpr int kMaxTopK = 16;
constexpr int kMaxExperts = 1024;
// Slots of one block of the sort, and up to how many one block does it all.
constexpr int kSortChunk = 2048;
constexpr int kSortAlone = 4096;
// Blocks up to which each block of the sort adds up the others' counts itself.
constexpr int kSortScan = 64;

struct SortArgs {
    const int32_t *idx;
    int64_t n;            // slots
    int E;
    int nblk;
    int32_t *hist;        // [nblk + 1][E + 1]: the blocks' counts, the last column of slots with a bad
                          // index; with more than kSortScan blocks sums of the blocks before, the
                          // last row of all
    int32_t *counts, *offsets, *sorted, *pos;   // counts, sorted: or NULL
    int32_t *status;
};

// Dropout's generator as the kernels take it; rng NULL: nothing is dropped.
struct Drop {
    const uint64_t *rng;   // device {seed, offset}
    uint32_t least;        // smallest 16 bits that keep an element
    float factor;          // of the kept elements
};

// Rows of tokens against the sorted rows of their slots.
struct TokenArgs {
    const uint16_t *x;     // token rows read
    int64_t ldx;
    const uint16_t *z;     // sorted rows read
    int64_t ldz;
    uint16_t *out;         // rows written: sorted ones (spread) or tokens' (gather)
    int64_t ldo;
    const uint16_t *base;  // gather: rows added, or NULL
    int64_t ldbase;
    const int32_t *pos;    // [T][k]
    const float *w;        // [T][k] or NULL: 1
    float *dw;             // [T][k] or NULL: <x or its dropped form, z>
    int64_t T, rows;       // tokens, sorted rows
    int64_t first;         // token of a launch
    int H, k;
    Drop drop;
};

struct DropoutArgs {
    const void *x, *residual;
    void *y;
    int64_t ldx, ldr, ldy, rows;
    int cols;
    uint64_t counter;   // of the first row, beside the generator's offset
    Drop drop;
};

hipError_t launch_sort(const SortArgs &a, hipStream_t s);
// out[pos[a]] = w[a] D(x[a / k]); dw[a] = <D(x[a / k]), z[pos[a]]>
hipError_t launch_spread(bool bf16, const TokenArgs &a, hipStream_t s);
// out[t] = base[t] + D(sum_j w[a] z[pos[a]]); dw[a] = <x[t], z[pos[a]]>
hipError_t launch_gather(bool bf16, const TokenArgs &a, hipStream_t s);
hipError_t launch_dropout(int dtype, const DropoutArgs &a, hipStream_t s);

}  // namespace moe
