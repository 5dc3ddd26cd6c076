// A shared projection with the low-rank adapters of many requests: the
// shrink x A^T per token, and the tile kernel whose epilogue expands it.
#include "dense_kernel.h"

namespace moe {

// mid[split][t][0..rpad) = the split's share of x[t] A_a^T, a = ids[t]; zeros
// from the adapter's own rank on; tokens without an adapter are not written.
//
// Block (f, split): `tpf` tokens (16, or 1 for few tokens) against their
// adapters, the k share cut over the four wavefronts.  Tokens are the matrix
// instruction's columns, so a 16-token block that names several adapters runs
// once per adapter and keeps each token's own result.  One token a block lets
// all the adapters of a decode step stream at once.
template <bool BF16, int NR>
__global__ __launch_bounds__(256) void lora_shrink_kernel(const uint16_t *x, int64_t ldx, int T, int K, int tpf,
                                                          LoraArgs lo)
{
    __shared__ f32x4 red[4][NR][64];
    const int tid = threadIdx.x, l = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int f = blockIdx.x, z = blockIdx.y, c = l & 15, kl = 8 * (l >> 4);

    if (f == 0 && z == 0) {
        // the call's status word: ids and ranks outside their ranges
        int bad = 0;
        for (int t = tid; t < T; t += 256)
            bad |= (lo.ids[t] < -1 || lo.ids[t] >= lo.n) ? (int)MOE_EXL3_STATUS_BAD_INDEX : 0;
        if (lo.ranks)
            for (int e = tid; e < lo.n; e += 256)
                bad |= (lo.ranks[e] < 0 || lo.ranks[e] > lo.rank) ? (int)MOE_EXL3_STATUS_BAD_WIDTH : 0;
        const int any = __syncthreads_or(bad & (int)MOE_EXL3_STATUS_BAD_INDEX);
        const int wide = __syncthreads_or(bad & (int)MOE_EXL3_STATUS_BAD_WIDTH);
        if (tid == 0)
            *lo.status = (any ? (int)MOE_EXL3_STATUS_BAD_INDEX : 0) | (wide ? (int)MOE_EXL3_STATUS_BAD_WIDTH : 0);
    }

    const int t = f * tpf + c;
    int id = c < tpf && t < T ? lo.ids[t] : -1;
    if (id >= lo.n)
        id = -1;
    const int steps = (K + 31) / 32;
    const int per = (steps + 4 * lo.splits - 1) / (4 * lo.splits);
    const int s0 = (4 * z + w) * per, s1 = min(s0 + per, steps);
    const uint16_t *xr = x + (int64_t)t * ldx;

    f32x4 sum[NR];
#pragma unroll
    for (int j = 0; j < NR; ++j)
        sum[j] = (f32x4){};
    bool left = id >= 0;
    for (;;) {
        const uint64_t any = __ballot(left);
        if (!any)
            break;
        const int e = __builtin_amdgcn_readlane(id, __ffsll((unsigned long long)any) - 1);
        const int rk = lo.ranks ? min(max(lo.ranks[e], 0), lo.rank) : lo.rank;
        const uint16_t *ar = lo.a + ((int64_t)e * lo.rank + c) * K;
        const bool hit = id == e;
        f32x4 acc[NR];
#pragma unroll
        for (int j = 0; j < NR; ++j)
            acc[j] = (f32x4){};
#pragma unroll 4
        for (int s = s0; s < s1; ++s) {
            const int k = 32 * s + kl;
            u32x4 p = {};
            if (hit && k < K)
                p = *(const u32x4 *)(xr + k);
#pragma unroll
            for (int j = 0; j < NR; ++j) {
                u32x4 q = {};
                if (16 * j + c < rk && k < K)
                    q = *(const u32x4 *)(ar + (int64_t)16 * j * K + k);
                acc[j] = dense_mfma<BF16>(q, p, acc[j]);
            }
        }
        if (hit) {
#pragma unroll
            for (int j = 0; j < NR; ++j)
                sum[j] = acc[j];
            left = false;
        }
    }
#pragma unroll
    for (int j = 0; j < NR; ++j)
        red[w][j][l] = sum[j];
    __syncthreads();
    for (int j = w; j < NR; j += 4) {
        const f32x4 v = (red[0][j][l] + red[1][j][l]) + (red[2][j][l] + red[3][j][l]);
        const int r = 16 * j + 4 * (l >> 4);
        if (id >= 0 && r < lo.rpad)
            *(f32x4 *)(lo.mid + ((int64_t)z * T + t) * lo.rpad + r) = v;
    }
}

template <bool BF16>
static void shrink(const uint16_t *x, int64_t ldx, int T, int K, int tpf, const LoraArgs &l, hipStream_t s)
{
    const dim3 grid((unsigned)((T + tpf - 1) / tpf), (unsigned)l.splits);
    if (l.rpad <= 32)
        lora_shrink_kernel<BF16, 2><<<grid, 256, 0, s>>>(x, ldx, T, K, tpf, l);
    else if (l.rpad <= 64)
        lora_shrink_kernel<BF16, 4><<<grid, 256, 0, s>>>(x, ldx, T, K, tpf, l);
    else if (l.rpad <= 128)
        lora_shrink_kernel<BF16, 8><<<grid, 256, 0, s>>>(x, ldx, T, K, tpf, l);
    else
        lora_shrink_kernel<BF16, 16><<<grid, 256, 0, s>>>(x, ldx, T, K, tpf, l);
}

hipError_t launch_lora_shrink(bool bf16, const uint16_t *x, int64_t ldx, int64_t T, int K, const LoraArgs &l,
                              hipStream_t s)
{
    const int tpf = T <= kLoraTokenBlocks ? 1 : 16;
    if (bf16)
        shrink<true>(x, ldx, (int)T, K, tpf, l, s);
    else
        shrink<false>(x, ldx, (int)T, K, tpf, l, s);
    return hipGetLastError();
}

hipError_t launch_dense_lin(bool bf16, const DenseArgs &a, hipStream_t s)
{
    return launch_dense_mode<DENSE_LIN>(bf16, a, s);
}

}  // namespace moe
