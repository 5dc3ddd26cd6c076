// A shared projection with the low-rank adapters of many requests: the
// shrink x A^T per token, and the tile kernel whose epilogue expands it.
#include "dense_skinny.h"

namespace moe {

constexpr int kShrinkWaves = 8;

// mid[split][t][0..rpad) = the split's share of x[t] A_a^T, a = ids[t]; zeros
// from the adapter's own rank on; tokens without an adapter are not written.
//
// Block (f, split): `tpf` tokens (16, or 1 for few tokens) against their
// adapters, the k share cut over the eight wavefronts.  Tokens are the matrix
// instruction's columns, so a 16-token block that names several adapters runs
// once per adapter and keeps each token's own result.  One token a block lets
// all the adapters of a decode step stream at once.
template <bool BF16, int NR>
__global__ __launch_bounds__(64 * kShrinkWaves) void lora_shrink_kernel(const uint16_t *x, int64_t ldx, int T, int K, int tpf,
                                                          LoraArgs lo)
{
    __shared__ f32x4 red[kShrinkWaves][NR][64];
    const int tid = threadIdx.x, l = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int f = blockIdx.x, z = blockIdx.y, c = l & 15, kl = 8 * (l >> 4);

    const int r0 = blockIdx.z * 16 * NR;   // ranks above 128 take several blocks

    if (f == 0 && z == 0 && r0 == 0) {
        // the call's status word: ids and ranks outside their ranges
        int bad = 0;
        for (int t = tid; t < T; t += 64 * kShrinkWaves)
            bad |= (lo.ids[t] < -1 || lo.ids[t] >= lo.n) ? (int)MOE_EXL3_STATUS_BAD_INDEX : 0;
        if (lo.ranks)
            for (int e = tid; e < lo.n; e += 64 * kShrinkWaves)
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
    // shares of 32 k, interleaved over the wavefronts of all splits
    const int steps = (K + 31) / 32, whole = K / 32;
    const int waves = kShrinkWaves * lo.splits, s0 = kShrinkWaves * z + w;
    const uint16_t *xr = x + (int64_t)min(f * tpf + min(c, tpf - 1), T - 1) * ldx + kl;

    f32x4 sum[NR];
#pragma unroll
    for (int j = 0; j < NR; ++j)
        sum[j] = (f32x4){};
    int rank = 0;   // of this lane's token
    bool left = id >= 0;
    for (;;) {
        const uint64_t any = __ballot(left);
        if (!any)
            break;
        const int e = __builtin_amdgcn_readlane(id, __ffsll((unsigned long long)any) - 1);
        const int rk = lo.ranks ? min(max(lo.ranks[e], 0), lo.rank) : lo.rank;
        // rows from the adapter's own rank on repeat its last one; what they
        // give is left out below
        const uint16_t *ar[NR];
#pragma unroll
        for (int j = 0; j < NR; ++j)
            ar[j] = lo.a + ((int64_t)e * lo.rank + max(0, min(r0 + 16 * j + c, rk - 1))) * K + kl;
        f32x4 acc[NR];
#pragma unroll
        for (int j = 0; j < NR; ++j)
            acc[j] = (f32x4){};
        // kBatch shares' loads first, then their products
        constexpr int kBatch = NR <= 2 ? 8 : NR == 4 ? 4 : 2;
        for (int s = s0; s < whole; s += kBatch * waves) {
            u32x4 p[kBatch], q[kBatch][NR];
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                const int64_t k = s + b * waves < whole ? 32 * (int64_t)(s + b * waves) : 0;
                p[b] = *(const u32x4 *)(xr + k);
#pragma unroll
                for (int j = 0; j < NR; ++j)
                    q[b][j] = *(const u32x4 *)(ar[j] + k);
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int b = 0; b < kBatch; ++b)
                if (s + b * waves < whole)
#pragma unroll
                    for (int j = 0; j < NR; ++j)
                        acc[j] = dense_mfma<BF16>(q[b][j], p[b], acc[j]);
        }
        if (steps > whole && whole % waves == s0) {
            const bool in = 32 * whole + kl < K;
            const u32x4 p = in ? *(const u32x4 *)(xr + 32 * whole) : (u32x4){};
#pragma unroll
            for (int j = 0; j < NR; ++j)
                acc[j] = dense_mfma<BF16>(in ? *(const u32x4 *)(ar[j] + 32 * whole) : (u32x4){}, p, acc[j]);
        }
        if (id == e) {
#pragma unroll
            for (int j = 0; j < NR; ++j)
                sum[j] = acc[j];
            rank = rk;
            left = false;
        }
    }
#pragma unroll
    for (int j = 0; j < NR; ++j)
        red[w][j][l] = sum[j];
    __syncthreads();
    for (int j = w; j < NR; j += kShrinkWaves) {
        f32x4 v = red[0][j][l];
#pragma unroll
        for (int s = 1; s < kShrinkWaves; ++s)
            v += red[s][j][l];
        const int r = r0 + 16 * j + 4 * (l >> 4);
#pragma unroll
        for (int d = 0; d < 4; ++d)
            v[d] = r + d < rank ? v[d] : 0.0f;
        if (id >= 0 && r < lo.rpad)
            *(f32x4 *)(lo.mid + ((int64_t)z * T + t) * lo.rpad + r) = v;
    }
}

template <bool BF16>
static void shrink(const uint16_t *x, int64_t ldx, int T, int K, int tpf, const LoraArgs &l, hipStream_t s)
{
    const unsigned nb = (unsigned)((T + tpf - 1) / tpf), nz = (unsigned)l.splits;
    if (l.rpad <= 32)
        lora_shrink_kernel<BF16, 2><<<dim3(nb, nz), 64 * kShrinkWaves, 0, s>>>(x, ldx, T, K, tpf, l);
    else if (l.rpad <= 64)
        lora_shrink_kernel<BF16, 4><<<dim3(nb, nz), 64 * kShrinkWaves, 0, s>>>(x, ldx, T, K, tpf, l);
    else
        lora_shrink_kernel<BF16, 8><<<dim3(nb, nz, (l.rpad + 127) / 128), 64 * kShrinkWaves, 0, s>>>(x, ldx, T, K, tpf,
                                                                                                   l);
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

hipError_t launch_skinny_lin(bool bf16, const DenseArgs &a, hipStream_t s)
{
    return bf16 ? launch_skinny<DENSE_LIN, true>(a, s) : launch_skinny<DENSE_LIN, false>(a, s);
}

}  // namespace moe
