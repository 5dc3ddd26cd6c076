// Internal launchers of the dense operators (the gated feed-forward block and
// the projection with adapters), shared with their host entry points.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "moe_exl3.h"

namespace moe {

// Rows and columns of the output tiles (a GLU tile's columns are half gate,
// half up), and the k that their launch plans count in.
constexpr int kDenseTile = 64;   // wavefronts cut k (dense_stream.h)
constexpr int kDenseSmall = 128;
constexpr int kDenseLarge = 256;
constexpr int kDenseK = 64;
// Tokens up to which the forward operators take the few-token kernel.
constexpr int64_t kSkinnyTokens = 64;
// Largest rank, bytes of A and columns up to which the few-token kernel computes
// one token's x A^T itself, in every block.  Up to 4096 columns that is one
// block a CU (2048 x 4096, rank 16: 11.8 -> 9.2 us a call; 4096 x 2048, rank 32:
// 12.1 -> 10.8; but 8192 x 8192, rank 16: 34.9 -> 42.7).  Two tokens' adapters,
// one after the other, take longer than the launch they save (4096 x 4096, rank
// 8: 12.2 -> 14.7).
constexpr int kFusedRank = 32;
constexpr int64_t kFusedBytes = 256 << 10;
constexpr int64_t kFusedCols = 4096;
// Largest rank of an adapter.
constexpr int kMaxRank = 256;

// What a tile launch computes, D[m][n] = sum_k P[m][k] Q[n][k]:
//   GLU  P = x [T][H], Q = gate and up rows: h = act(g) * u, pre = (g, u)
//   DX   P = dg | du [T][I], Q = Wg | Wu [I][H] read along their rows (k is
//        the slow index): dx = dg Wg + du Wu
//   DW   P = dg or du, Q = x, both with the token as the slow index:
//        dWg = dg^T x, dWu = du^T x
//   LIN  P = x [T][K], Q = W [N][K]: y = x W^T + base + the adapters' rows
enum DenseMode { DENSE_GLU = 0, DENSE_DX = 1, DENSE_DW = 2, DENSE_LIN = 3 };

// The adapters of a LIN launch.
struct LoraArgs {
    const uint16_t *a;       // [n][rank][K]
    const uint16_t *b;       // [n][N][rank]
    const int32_t *ids;      // [T], < 0: no adapter
    const float *scales;     // [n] or NULL (1)
    const int32_t *ranks;    // [n] or NULL (rank)
    int32_t *status;         // status word of the call
    void *mid;               // [T][rpad] s_a x A_a^T, zeros from the adapter's rank on: fp32 for the
                             // few-token kernel, in 16 bits for the tile kernels
    int n, rank, rpad;       // rpad: rank rounded up to 32
    int k;                   // columns of x and of A's rows
    bool fused;              // one token: x A^T in the same launch, mid is not used
};

struct DenseArgs {
    const uint16_t *p[2], *q[2];
    int64_t ldp, ldq;        // elements between rows in memory
    uint32_t pbytes, qbytes; // bytes of each tensor, from its first to its last element
    int M, N, K;             // DX: K = I per segment; DW: M = I per tensor; GLU: N = I
    uint16_t *out[2];
    int64_t ldo;
    float *pre;              // GLU: fp32 [2][T][I] or NULL
    int act;
    int bm;                  // tile: kDenseTile, kDenseSmall or kDenseLarge
    int mt, nt;              // tiles (DW: mt counts both tensors')
    int splits, per;         // k splits and stages of each
    float *part;             // splits > 1: partial tiles, fragment order
    const uint16_t *base;    // LIN: added rows or NULL
    int64_t ldbase;
    LoraArgs lora;
};

hipError_t launch_dense(int mode, bool bf16, const DenseArgs &a, hipStream_t s);
// DX in 64 x 64 tiles and DW in 64 x 64 or 128 x 128 ones, in one launch, DW's
// blocks before or behind DX's.
hipError_t launch_dense_grads(bool bf16, const DenseArgs &dx, const DenseArgs &dw, bool dw_first, hipStream_t s);
// GLU or LIN of at most kSkinnyTokens tokens.
hipError_t launch_dense_skinny(int mode, bool bf16, const DenseArgs &a, hipStream_t s);
hipError_t launch_glu_grad(bool bf16, int act, const float *pre, const uint16_t *dh, int64_t lddh, int64_t T, int I,
                           uint16_t *dg, uint16_t *du, hipStream_t s);
hipError_t launch_lora_shrink(bool bf16, const uint16_t *x, int64_t ldx, uint32_t xbytes, int64_t T, int K,
                              const LoraArgs &l, hipStream_t s);

}  // namespace moe
