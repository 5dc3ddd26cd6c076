// A shared projection with the low-rank adapters of many requests: the
// shrink x A^T per token, and the tile kernel whose epilogue expands it.
#include "dense_stream.h"

namespace moe {

// The call's status word: ids outside their range, and ranks of the adapters
// that they name.
template <int THREADS>
MOE_DEV void check_adapters(const LoraArgs &lo, int T, int tid)
{
    int bad = 0;
    constexpr int kBatch = 8;   // loads in flight a thread
    for (int t = tid; t < T; t += kBatch * THREADS) {
        int id[kBatch];
#pragma unroll
        for (int b = 0; b < kBatch; ++b)
            id[b] = lo.ids[min(t + b * THREADS, T - 1)];
#pragma unroll
        for (int b = 0; b < kBatch; ++b)
            bad |= id_faults(lo, id[b]);
    }
    const int index = __syncthreads_or(bad & (int)MOE_EXL3_STATUS_BAD_INDEX);
    const int width = __syncthreads_or(bad & (int)MOE_EXL3_STATUS_BAD_WIDTH);
    if (tid == 0)
        *lo.status = (index ? (int)MOE_EXL3_STATUS_BAD_INDEX : 0) | (width ? (int)MOE_EXL3_STATUS_BAD_WIDTH : 0);
}

// mid[t][0..rpad) = scales[e] x[t] A_e^T, e = ids[t]: in 16 bits for the matrix
// cores of the tile kernels, in fp32 for the few-token kernel, which multiplies
// in fp32; zeros from the adapter's own rank on.  Tokens without an adapter are
// not written.
//
// Block (f, r): `tpf` tokens (1, 8 or 16) against 16 NR rows of their adapters, k
// cut over the NW wavefronts.  Tokens are the matrix instruction's columns, so
// a 16-token block that names several adapters runs once per adapter and each
// token keeps its own result.  One token a block lets all the adapters of a
// decode step stream at once, at the price of reading an adapter once per
// token; 16 tokens a block read it once where a request's tokens stand together.
// Bound by latency: 64 tokens, 2048 k, rank 64: 5.2 us (4 MB of A); 7168 tokens,
// 2048 k, rank 32: 10 us for 30 MB of x.
template <bool BF16, int NW, int NR, int RING>
__global__ __launch_bounds__(64 * NW) void lora_shrink_kernel(const uint16_t *x, int64_t ldx, uint32_t xbytes, int T,
                                                              int K, int tpf, LoraArgs lo)
{
    using S = Stream<BF16, 1, NR, RING>;
    __shared__ __align__(1024) uint16_t ring0[NW * S::kHalves], ring1[NW * S::kHalves], ring2[NW * S::kHalves],
        ring3[RING == 4 ? NW * S::kHalves : 8];
    const int tid = threadIdx.x, l = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int f = blockIdx.x, r0 = 16 * NR * blockIdx.y, c = l & 15;
    if (f * tpf >= T) {   // the last block
        if (r0 == 0)
            check_adapters<64 * NW>(lo, T, tid);
        return;
    }
    const int t = f * tpf + c;
    int id, rank;   // of this lane's token
    token_adapter(lo, c < tpf ? t : T, T, id, rank);
    const int at = w * S::kHalves;
    f32x4 sum[NR] = {};
    lora_rows<BF16, NR, RING>(
        lo, id, rank, r0, l, w, NW, K, ldx, buf_rsrc(x, xbytes),
        // rows past the block's tokens read zeros
        [&](int r) { return (int64_t)(r < tpf ? f * tpf + r : T); }, (LDS_AS uint16_t *)ring0 + at,
        (LDS_AS uint16_t *)ring1 + at, (LDS_AS uint16_t *)ring2 + at, (LDS_AS uint16_t *)ring3 + (RING == 4 ? at : 0),
        sum);
    // the wavefronts' sums, each in its own part of the first ring array
    LDS_AS f32x4 *red = (LDS_AS f32x4 *)((LDS_AS uint16_t *)ring0);
    constexpr int kStep = S::kHalves / 8;
#pragma unroll
    for (int j = 0; j < NR; ++j)
        red[w * kStep + 64 * j + l] = sum[j];
    __syncthreads();
    if (w >= NR || id < 0)
        return;
    f32x4 v = red[64 * w + l];
#pragma unroll
    for (int s = 1; s < NW; ++s)
        v += red[s * kStep + 64 * w + l];
    // the rows from the adapter's own rank on were read as zeros, which an
    // infinity in x makes NaNs of
    const int k = r0 + 16 * w + 4 * (l >> 4);
#pragma unroll
    for (int d = 0; d < 4; ++d)
        v[d] = k + d < rank ? v[d] : 0.0f;
    const int64_t o = (int64_t)t * lo.rpad + k;
    if (T <= (int)kSkinnyTokens)
        *(f32x4 *)((float *)lo.mid + o) = v;
    else
        *(u32x2 *)((uint16_t *)lo.mid + o) = (u32x2){pack16<BF16>(v[0], v[1]), pack16<BF16>(v[2], v[3])};
}

// One token a block while all blocks together read at most this much of the
// adapters (about 15 us from L2) and are at most this many (1024 tokens of 64
// mixed adapters, 4096 k, rank 16: 9 us; 16 tokens a block run each adapter
// after the other, 98 us, and win where a request's tokens stand together:
// 7168 tokens, 2048 k, rank 32: 10 us for 940 MB).
constexpr int64_t kShrinkBytes = 192 << 20;
constexpr int64_t kShrinkBlocks = 2048;

template <bool BF16>
static void shrink(const uint16_t *x, int64_t ldx, uint32_t xbytes, int T, int K, const LoraArgs &l, hipStream_t s)
{
    if ((int64_t)T * l.rank * K * 2 <= kShrinkBytes && (int64_t)T * (l.rpad / 16) <= kShrinkBlocks) {
        // one block more, for the status word; every wavefront of a 2048-k
        // token has all its shares in flight
        const dim3 grid((unsigned)(T + 1), (unsigned)(l.rpad / 16));
        if ((int64_t)T * grid.y <= 512)
            lora_shrink_kernel<BF16, 8, 1, 4><<<grid, 512, 0, s>>>(x, ldx, xbytes, T, K, 1, l);
        else
            lora_shrink_kernel<BF16, 4, 1, 4><<<grid, 256, 0, s>>>(x, ldx, xbytes, T, K, 1, l);
    } else {
        // 8 tokens a block where 16 would leave most CUs idle (whole calls with 8
        // and with 16: 300 tokens, 4096 k, 64 adapters of 128: 72 us, 78; 732
        // tokens, 6696 k, rank 48: 43.5, 47.4; but 1000 tokens, 4096 k, 64 adapters
        // of 64: 32, 28)
        const int tpf = (int64_t)((T + 15) / 16) * (l.rpad / 32) <= 96 ? 8 : 16;
        const dim3 grid((unsigned)((T + tpf - 1) / tpf + 1), (unsigned)(l.rpad / 32));
        // eight wavefronts a block while that is one block a CU (144 KiB of
        // LDS), four and two blocks beyond
        if ((int64_t)(grid.x - 1) * grid.y <= 256)
            lora_shrink_kernel<BF16, 8, 2, 3><<<grid, 512, 0, s>>>(x, ldx, xbytes, T, K, tpf, l);
        else
            lora_shrink_kernel<BF16, 4, 2, 3><<<grid, 256, 0, s>>>(x, ldx, xbytes, T, K, tpf, l);
    }
}

hipError_t launch_lora_shrink(bool bf16, const uint16_t *x, int64_t ldx, uint32_t xbytes, int64_t T, int K,
                              const LoraArgs &l, hipStream_t s)
{
    if (bf16)
        shrink<true>(x, ldx, xbytes, (int)T, K, l, s);
    else
        shrink<false>(x, ldx, xbytes, (int)T, K, l, s);
    return hipGetLastError();
}

hipError_t launch_dense_lin(bool bf16, const DenseArgs &a, hipStream_t s)
{
    return launch_any<DENSE_LIN>(bf16, a, s);
}

hipError_t launch_skinny_lin(bool bf16, const DenseArgs &a, hipStream_t s)
{
    return bf16 ? launch_skinny<DENSE_LIN, true>(a, s) : launch_skinny<DENSE_LIN, false>(a, s);
}

}  // namespace moe
