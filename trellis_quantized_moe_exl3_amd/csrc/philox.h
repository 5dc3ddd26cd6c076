// Philox4x32-10 (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as
// easy as 1, 2, 3", 2011): ten rounds of two 32 x 32 -> 64-bit products over a
// 128-bit counter, and dropout's use of its bits.
#pragma once

#include "common.h"
#include "tokens.h"

namespace moe {

MOE_DEV u32x4 philox(uint64_t counter, uint64_t key)
{
    u32x4 x = {(uint32_t)counter, (uint32_t)(counter >> 32), 0u, 0u};
    uint32_t k0 = (uint32_t)key, k1 = (uint32_t)(key >> 32);
#pragma unroll
    for (int i = 0; i < 10; ++i) {
        const uint64_t a = (uint64_t)x[0] * 0xD2511F53u, b = (uint64_t)x[2] * 0xCD9E8D57u;
        x = (u32x4){(uint32_t)(b >> 32) ^ x[1] ^ k0, (uint32_t)b, (uint32_t)(a >> 32) ^ x[3] ^ k1, (uint32_t)a};
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return x;
}

// Dropout of the eight elements of one group: 16 bits an element, so that one
// counter serves eight and the generator (20 products of a quarter of the
// vector rate) keeps up with memory; p is a multiple of 2^-16, and the factor
// is exact for that p.  A dropped element is a zero whatever it was.
MOE_DEV void drop8(const Drop &d, uint64_t seed, uint64_t counter, float (&v)[8])
{
    const u32x4 r = philox(counter, seed);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = (r[i] & 0xFFFFu) >= d.least ? v[2 * i] * d.factor : 0.0f;
        v[2 * i + 1] = (r[i] >> 16) >= d.least ? v[2 * i + 1] * d.factor : 0.0f;
    }
}

}  // namespace moe
