// The few-token kernel of the forward operators.
//
// Up to 64 tokens the weights' bytes bound the call, and each is used once per
// call: they go from memory straight into the registers of the matrix
// instruction that uses them.  A block owns 16 weight rows (GLU: 8 gate and
// the same 8 up columns, so that a 2048-column block still makes 256 blocks)
// and its eight wavefronts cut k into interleaved shares of 64 (a 128-byte
// line of every row); the tokens' rows come from L2.  The wavefronts' sums
// meet in LDS, in a fixed order.
#pragma once

#include "dense_kernel.h"

namespace moe {

constexpr int kSkinnyWaves = 8;

// delta[t][16 columns]: the adapters' rows of tokens t = w, w + 8, ..: lane l
// takes column l % 16 and the k octets l / 16 + 0, 4, .. of the token's
// adapter, all in fp32.
template <bool BF16>
MOE_DEV void skinny_expand(const DenseArgs &a, int n0, int w, int l, float (*delta)[16])
{
    const LoraArgs &lo = a.lora;
    const int c = l & 15, n = min(n0 + c, a.N - 1);
    for (int t = w; t < a.M; t += kSkinnyWaves) {
        const int id = lo.ids[t];
        const bool on = id >= 0 && id < lo.n;
        const int e = on ? id : 0;
        const int rk = on ? (lo.ranks ? min(max(lo.ranks[e], 0), lo.rank) : lo.rank) : 0;
        const float sc = lo.scales ? lo.scales[e] : 1.0f;
        float sum = 0.0f;
        for (int k = 8 * (l >> 4); k < rk; k += 32) {
            float u[8] = {};
            for (int z = 0; z < lo.splits; ++z) {
                const f32x4 *p = (const f32x4 *)(lo.mid + ((int64_t)z * a.M + t) * lo.rpad + k);
                const f32x4 x0 = p[0], x1 = p[1];
#pragma unroll
                for (int d = 0; d < 4; ++d) {
                    u[d] += x0[d];
                    u[4 + d] += x1[d];
                }
            }
            const u32x4 b = *(const u32x4 *)(lo.b + ((int64_t)e * a.N + n) * lo.rank + k);
#pragma unroll
            for (int d = 0; d < 8; ++d) {
                const float bv = act_to_f32<BF16>((uint16_t)(b[d >> 1] >> (16 * (d & 1))));
                sum += k + d < rk ? u[d] * bv : 0.0f;
            }
        }
        sum += __shfl_xor(sum, 16);
        sum += __shfl_xor(sum, 32);
        if (l < 16)
            delta[t][c] = sum * sc;
    }
}

template <int MODE, bool BF16, int NI>
__global__ __launch_bounds__(64 * kSkinnyWaves) void dense_skinny_kernel(DenseArgs a)
{
    __shared__ f32x4 red[kSkinnyWaves][NI][64];
    __shared__ __align__(16) float delta[MODE == DENSE_LIN ? 16 * NI : 1][16];
    const int tid = threadIdx.x, l = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int c = l & 15, kl = 8 * (l >> 4);
    constexpr int kCols = MODE == DENSE_GLU ? 8 : 16;
    const int n0 = blockIdx.x * kCols;
    // rows past the matrices repeat the last one; what they give is not stored
    const uint16_t *q = MODE == DENSE_GLU ? (c < 8 ? a.q[0] : a.q[1]) + (int64_t)(n0 + (c & 7)) * a.ldq
                                          : a.q[0] + (int64_t)min(n0 + c, a.N - 1) * a.ldq;
    q += kl;
    const uint16_t *p[NI];
#pragma unroll
    for (int i = 0; i < NI; ++i)
        p[i] = a.p[0] + (int64_t)min(16 * i + c, a.M - 1) * a.ldp + kl;

    f32x4 acc[NI];
#pragma unroll
    for (int i = 0; i < NI; ++i)
        acc[i] = (f32x4){};
    // whole 64-k shares, kBatch at a time: all their loads first, so that a
    // wavefront waits for memory once a batch (past the end they repeat the
    // rows' start, and are not used)
    constexpr int kBatch = NI <= 2 ? 8 : 4;
    const int full = a.K / 64;
    for (int it = w; it < full; it += kBatch * kSkinnyWaves) {
        u32x4 qv[kBatch][2], pv[kBatch][NI][2];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int s = it + b * kSkinnyWaves;
            const int64_t k = s < full ? 64 * (int64_t)s : 0;
            qv[b][0] = *(const u32x4 *)(q + k);
            qv[b][1] = *(const u32x4 *)(q + k + 32);
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                pv[b][i][0] = *(const u32x4 *)(p[i] + k);
                pv[b][i][1] = *(const u32x4 *)(p[i] + k + 32);
            }
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int b = 0; b < kBatch; ++b)
            if (it + b * kSkinnyWaves < full)
#pragma unroll
                for (int i = 0; i < NI; ++i) {
                    acc[i] = dense_mfma<BF16>(qv[b][0], pv[b][i][0], acc[i]);
                    acc[i] = dense_mfma<BF16>(qv[b][1], pv[b][i][1], acc[i]);
                }
    }
    if (full % kSkinnyWaves == w && a.K % 64) {
        for (int k = 64 * full; k < a.K; k += 32) {
            const bool in = k + kl < a.K;
            const u32x4 qv = in ? *(const u32x4 *)(q + k) : (u32x4){};
#pragma unroll
            for (int i = 0; i < NI; ++i)
                acc[i] = dense_mfma<BF16>(qv, in ? *(const u32x4 *)(p[i] + k) : (u32x4){}, acc[i]);
        }
    }
    if constexpr (MODE == DENSE_LIN)
        skinny_expand<BF16>(a, n0, w, l, delta);
#pragma unroll
    for (int i = 0; i < NI; ++i)
        red[w][i][l] = acc[i];
    __syncthreads();
    if (w >= NI)
        return;
    const int m = 16 * w + c;
    auto total = [&](int lane) {
        f32x4 v = red[0][w][lane];
#pragma unroll
        for (int s = 1; s < kSkinnyWaves; ++s)
            v += red[s][w][lane];
        return v;
    };
    if constexpr (MODE == DENSE_GLU) {
        // lanes 0..31 hold gate columns 4 (l / 16) + 0..3, lanes 32..63 the same
        // columns of up
        if (l < 32 && m < a.M) {
            const f32x4 v[2] = {total(l), total(l + 32)};
            glu_store<BF16>(a, m, n0 + 4 * (l >> 4), v[0], v[1]);
        }
    } else if (m < a.M && n0 + 4 * (l >> 4) < a.N) {
        const f32x4 d = *(const f32x4 *)&delta[m][4 * (l >> 4)];
        lin_store<BF16>(a, m, n0 + 4 * (l >> 4), total(l) + d);
    }
}

template <int MODE, bool BF16>
hipError_t launch_skinny(const DenseArgs &a, hipStream_t s)
{
    constexpr int kCols = MODE == DENSE_GLU ? 8 : 16;
    const dim3 grid((unsigned)((a.N + kCols - 1) / kCols)), block(64 * kSkinnyWaves);
    if (a.M <= 16)
        dense_skinny_kernel<MODE, BF16, 1><<<grid, block, 0, s>>>(a);
    else if (a.M <= 32)
        dense_skinny_kernel<MODE, BF16, 2><<<grid, block, 0, s>>>(a);
    else
        dense_skinny_kernel<MODE, BF16, 4><<<grid, block, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace moe
