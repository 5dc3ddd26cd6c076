// Tile pieces of the dense operators' matrix products: operand loaders,
// fragment reads and the pipelined k loop.
//
// D[m][n] = sum_k P[m][k] Q[n][k] on v_mfma_f32_16x16x32 with Q as the
// instruction's row operand, so that a lane ends with four consecutive n of
// one m: lane l of a 16 x 16 block holds m = l % 16, n = 4 (l / 16) + 0..3,
// one 8-byte store of 16-bit results.  Both operands pass through LDS in a
// ring of stages of BK = 32 or 64 k, filled by LDS-direct buffer loads (16 bytes a
// lane, 1 KiB an instruction); lanes past the matrix or past k read through an
// offset beyond the descriptor's range, for which the load writes zeros.
//
// An operand's layout in memory decides its LDS image:
//   KC  k contiguous ([row][k]): rows of 16-byte pieces, 64 bytes of four (piece
//       p of row r in slot p ^ 2 (r / 8 % 2)) or 128 bytes of eight (slot p ^ (r /
//       2 % 8)).  A 16-byte LDS read serves the lanes {0-3, 12-15, 20-27}, {4-11,
//       16-19, 28-31} and the same of the upper half together (measured: which
//       lane pairs count bank conflicts); with these orders each such group of a
//       fragment's lanes hits 16 distinct 4-bank groups (of 64 banks).  Slots
//       p ^ (r / 4 % 4), right for 16 lanes in a row, cost twice the clocks.
//   KS  k strided ([k][row]): one LDS row per k, its 16-row chunks of 32 bytes
//       in slot c ^ f(k), f(k) = k % 4 + 4 (k / 8 % 2): the eight k rows
//       32 lanes read at once hit distinct 8-bank groups.  The fragment comes
//       out of the transposing LDS read.
#pragma once

#include "common.h"
#include "dense.h"
#include "gemm.h"

namespace moe {

typedef short i16x4 __attribute__((ext_vector_type(4)));

enum Layout { KC = 0, KS = 1 };

constexpr uint32_t kOutOfRange = 0x7FFFFFF0u;   // every tensor is below 2 GiB

template <bool BF16>
MOE_DEV f32x4 dense_mfma(u32x4 q, u32x4 p, f32x4 c)
{
    if constexpr (BF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, q), __builtin_bit_cast(bf16x8, p), c,
                                                        0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, q), __builtin_bit_cast(f16x8, p), c,
                                                       0, 0, 0);
}

// Two fp32 rounded to nearest even (one instruction for bf16).
template <bool BF16>
MOE_DEV uint32_t pack16(float lo, float hi)
{
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    if constexpr (BF16)
        return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2){lo, hi}, bf16x2));
    else
        return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2){lo, hi}, f16x2));
}

// The transposing LDS read: in a group of 16 lanes, lane i passes the address of
// 8 bytes, part i % 4 of row i / 4, and receives column i of the four rows.
MOE_DEV u32x2 tr_read(const LDS_AS char *at)
{
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS_AS i16x4 *)const_cast<LDS_AS char *>(at)));
}

// One operand of R tile rows and BK k, loaded by NW wavefronts.
template <int R, int LAYOUT, int NW, int BK>
struct Operand {
    static constexpr int kLoads = R * BK / 512 / NW;   // 1-KiB loads per wavefront and stage
    static constexpr bool kWide = BK == 64;
    static_assert(kLoads * 512 * NW == R * BK && (BK == 32 || (kWide && kLoads % 2 == 0)), "whole loads");
    uint32_t off[kLoads];                  // byte offset of the lane's 16 bytes at k = 0
    int kp[LAYOUT == KS ? kLoads : 2];     // first k of the lane's 16 bytes (KC: of even and odd loads)

    // The tile's load number that is load j of wavefront w, and the tile row of
    // the lane's piece of it (KC).
    MOE_DEV static int load_at(int w, int j) { return kWide ? kLoads * w + j : w + NW * j; }
    MOE_DEV static int kc_row(int w, int l, int j)
    {
        return kWide ? 8 * load_at(w, j) + (l >> 3) : 16 * load_at(w, j) + (l >> 2);
    }

    // KC: `row(r)` is the memory row of tile row r
    template <class F>
    MOE_DEV void init_kc(int w, int l, int64_t ld, F row)
    {
#pragma unroll
        for (int j = 0; j < 2; ++j)
            kp[j] = 8 * (kWide ? (l & 7) ^ (4 * j + (l >> 4)) : (l & 3) ^ ((l >> 4) & 2));
#pragma unroll
        for (int j = 0; j < kLoads; ++j)
            off[j] = (uint32_t)(row(kc_row(w, l, j)) * ld * 2 + 2 * kp[j & 1]);
    }
    // KS: tile rows are memory columns c0 ..
    MOE_DEV void init_ks(int w, int l, int64_t ld, int c0)
    {
        constexpr int kPieces = R / 8;   // 16-byte pieces of an LDS row
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            const int piece = 64 * load_at(w, j) + l;
            const int k = piece / kPieces, q = piece % kPieces;
            const int f = (k & 3) | ((k >> 1) & 4);
            const int c = 16 * ((q >> 1) ^ f) + 8 * (q & 1);
            kp[j] = k;
            off[j] = (uint32_t)(k * ld * 2 + (c0 + c) * 2);
        }
    }
    // The loads of the stage at k0 (kend: first k past the operand or the
    // block's share of it; the lanes from there on read zeros).
    MOE_DEV void issue(__amdgpu_buffer_rsrc_t rs, LDS_AS uint16_t *lds, int w, int k0, int kend, uint32_t kbytes)
    {
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            const int k = k0 + kp[LAYOUT == KS ? j : j & 1];
            const uint32_t o = k < kend ? off[j] + (uint32_t)k0 * kbytes : kOutOfRange;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (LDS_AS void *)(lds + 512 * load_at(w, j)), 16, o, 0, 0, 0);
        }
    }
    // Fragment of the 16 tile rows r0 + 16 i and the 32 k number h of a stage:
    // lane l holds row l % 16, k = 32 h + 8 (l / 16) + 0..7.
    MOE_DEV static uint32_t frag_base(int l, int r0)
    {
        if constexpr (LAYOUT == KC && kWide)
            return (uint32_t)((r0 + (l & 15)) * 128 + (((l >> 4) ^ ((l & 15) >> 1)) << 4));
        if constexpr (LAYOUT == KC)
            return (uint32_t)((r0 + (l & 15)) * 64 + (((l >> 4) ^ ((l >> 2) & 2)) << 4));
        const int i = l & 15, g = l >> 4, k = 8 * g + (i >> 2);
        const int f = (k & 3) | ((k >> 1) & 4);
        return (uint32_t)(k * 2 * R + (((r0 >> 4) ^ f) << 5) + (i & 3) * 8);
    }
    MOE_DEV static u32x4 frag(const LDS_AS uint16_t *lds, uint32_t base, int i, int h)
    {
        if constexpr (LAYOUT == KC)
            return *(const LDS_AS u32x4 *)((const LDS_AS char *)lds + (base ^ (64u * h)) + 32 * BK * i);
        const uint32_t o = base ^ (uint32_t)(i << 5);   // r0 is a multiple of 16 x the blocks read
        const LDS_AS char *at = (const LDS_AS char *)lds + 64 * R * h;
        const u32x2 lo = tr_read(at + o), hi = tr_read(at + o + 4 * 2 * R);
        return (u32x4){lo[0], lo[1], hi[0], hi[1]};
    }
};

// Tile of a block: contiguous runs of tiles per XCD (blocks are dealt to the 8
// XCDs round-robin), walked in groups of 8 row tiles so that the 32 tiles an
// XCD holds at a time share their rows and columns in its L2.
MOE_DEV void dense_tile(int L, int total, int mt, int nt, int &m, int &n)
{
    const int x = L & 7, j = L >> 3, q = total >> 3, r = total & 7;
    const int id = x * q + min(x, r) + j;
    const int group = id / (8 * nt), in = id - group * 8 * nt;
    const int rows = min(8, mt - 8 * group);
    m = 8 * group + in % rows;
    n = in / rows;
}

}  // namespace moe
