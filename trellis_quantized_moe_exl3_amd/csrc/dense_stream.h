// Products whose k is cut over the wavefronts of a block, for few tokens and
// for adapters.
//
// Each wavefront streams its own k shares of both operands through its own
// ring in LDS and needs no barrier until the block's sums meet.  The loads go
// to LDS (16 bytes a lane, eight lanes to a row's 128-byte line) because the
// matrix instruction wants consecutive lanes on different rows: loaded straight
// into its registers, every lane is a memory transaction of its own (64 clocks
// an instruction, measured, against 16 for whole lines).
#pragma once

#include "dense_kernel.h"

namespace moe {

// D[m][n] over NI x NJ blocks of 16 x 16; the block's wavefronts take k shares
// of 64 in turn (share `first`, first + stride, ..), RING shares in flight
// each.  The first NJ loads of Q (8 rows each) go through q[0], the rest
// through q[1].
//
// LDS image of a share: 128-byte rows of eight 16-byte pieces, piece p of row r
// in slot p ^ ((r >> 1) & 7): the 16 rows a fragment reads at one piece hit 16
// distinct 4-bank groups.
template <bool BF16, int NI, int NJ, int RING>
struct Stream {
    static constexpr int kLoads = 2 * (NI + NJ);
    static constexpr int kHalves = 16 * (NI + NJ) * 64;   // of one share
    __amdgpu_buffer_rsrc_t p, q[2];
    uint32_t off[kLoads];   // byte offset of the lane's 16 bytes at k = 0
    int l, kend;

    // Row of load j (P: j < 2 NI, Q: j - 2 NI) that lane l fetches, and its
    // first k.
    MOE_DEV static int row(int l, int j) { return 8 * j + (l >> 3); }
    MOE_DEV static int first_k(int l, int j) { return 8 * ((l & 7) ^ ((4 * j + (l >> 4)) & 7)); }

    // prow(r), qrow(r): memory rows of the tile rows
    template <class FP, class FQ>
    MOE_DEV void init(int lane, int K, int64_t ldp, int64_t ldq, FP prow, FQ qrow)
    {
        l = lane;
        kend = K;
#pragma unroll
        for (int j = 0; j < 2 * NI; ++j)
            off[j] = (uint32_t)((prow(row(l, j)) * ldp + first_k(l, j)) * 2);
#pragma unroll
        for (int j = 0; j < 2 * NJ; ++j)
            off[2 * NI + j] = (uint32_t)((qrow(row(l, j)) * ldq + first_k(l, j)) * 2);
    }
    MOE_DEV void load(int share, LDS_AS uint16_t *lds)
    {
        const int k0 = 64 * share;
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            const bool isq = j >= 2 * NI;
            const int jj = isq ? j - 2 * NI : j;
            const uint32_t o = k0 + first_k(l, jj) < kend ? off[j] + 2u * (uint32_t)k0 : kOutOfRange;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(!isq ? p : jj < NJ ? q[0] : q[1], (LDS_AS void *)(lds + 512 * j),
                                                     16, o, 0, 0, 0);
        }
    }
    // Wait for the share in `cur` (the RING - 1 shares after it stay in
    // flight), read its fragments, refill it, multiply.
    MOE_DEV void step(int refill, LDS_AS uint16_t *cur, f32x4 (&acc)[NI][NJ])
    {
        __builtin_amdgcn_sched_barrier(0);
        wait_vmcnt<(RING - 1) * kLoads>();
        const uint32_t base = (uint32_t)((l & 15) * 128 + (((l >> 4) ^ ((l & 15) >> 1)) << 4));
        u32x4 pf[2][NI], qf[2][NJ];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const LDS_AS char *at = (const LDS_AS char *)cur + (base ^ (64u * h));
#pragma unroll
            for (int i = 0; i < NI; ++i)
                pf[h][i] = *(const LDS_AS u32x4 *)(at + 2048 * i);
#pragma unroll
            for (int j = 0; j < NJ; ++j)
                qf[h][j] = *(const LDS_AS u32x4 *)(at + 2048 * (NI + j));
        }
        __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0): the slot is free
        __builtin_amdgcn_sched_barrier(0);
        load(refill, cur);
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < NI; ++i)
#pragma unroll
                for (int j = 0; j < NJ; ++j)
                    acc[i][j] = dense_mfma<BF16>(qf[h][j], pf[h][i], acc[i][j]);
    }
    MOE_DEV void run(int first, int stride, LDS_AS uint16_t *r0, LDS_AS uint16_t *r1, LDS_AS uint16_t *r2,
                     LDS_AS uint16_t *r3, f32x4 (&acc)[NI][NJ])
    {
        static_assert(RING == 3 || RING == 4, "ring arrays");
        const int shares = (kend + 63) / 64;
        if (first >= shares)
            return;
        load(first, r0);
        load(first + stride, r1);
        load(first + 2 * stride, r2);
        if constexpr (RING == 4)
            load(first + 3 * stride, r3);
        for (int s = first; s < shares; s += RING * stride) {
            step(s + RING * stride, r0, acc);
            step(s + (RING + 1) * stride, r1, acc);
            step(s + (RING + 2) * stride, r2, acc);
            if constexpr (RING == 4)
                step(s + (RING + 3) * stride, r3, acc);
        }
        wait_vmcnt<0>();   // the loads past the end still write LDS
    }
};

// ---- the block and the projection for few tokens

// delta[t][16 columns]: the adapters' rows of tokens t = w, w + XW, .. , four
// at a time: lane l takes column l / 4 and the k octets l % 4 + 0, 4, .. of the
// token's adapter (four lanes to 64 bytes of a row of B), summed in fp32.
template <bool BF16, int XW>
MOE_DEV void skinny_expand(const DenseArgs &a, int n0, int w, int l, float (*delta)[16])
{
    const LoraArgs &lo = a.lora;
    const int c = l >> 2, n = min(n0 + c, a.N - 1);
    constexpr int kBatch = 4;
    for (int t0 = w; t0 < a.M; t0 += kBatch * XW) {
        int rk[kBatch], most = 0;
        const uint16_t *bp[kBatch], *up[kBatch];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int t = min(t0 + b * XW, a.M - 1);
            const int id = lo.ids[t];
            const bool on = id >= 0 && id < lo.n;
            const int e = on ? id : 0;
            rk[b] = on ? (lo.ranks ? min(max(lo.ranks[e], 0), lo.rank) : lo.rank) : 0;
            most = max(most, rk[b]);
            bp[b] = lo.b + ((int64_t)e * a.N + n) * lo.rank;
            up[b] = lo.mid + (int64_t)t * lo.rpad;
        }
        float sum[kBatch] = {};
        for (int k = 8 * (l & 3); k < most; k += 32) {
            u32x4 bv[kBatch], uv[kBatch];
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                bv[b] = *(const u32x4 *)(bp[b] + min(k, lo.rank - 8));
                uv[b] = *(const u32x4 *)(up[b] + k);
            }
#pragma unroll
            for (int b = 0; b < kBatch; ++b)
#pragma unroll
                for (int d = 0; d < 8; ++d) {
                    const float y = act_to_f32<BF16>((uint16_t)(bv[b][d >> 1] >> (16 * (d & 1)))) *
                                    act_to_f32<BF16>((uint16_t)(uv[b][d >> 1] >> (16 * (d & 1))));
                    sum[b] += k + d < rk[b] ? y : 0.0f;
                }
        }
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            sum[b] += __shfl_xor(sum[b], 1);
            sum[b] += __shfl_xor(sum[b], 2);
            if ((l & 3) == 0 && t0 + b * XW < a.M)
                delta[t0 + b * XW][c] = sum[b];
        }
    }
}

// A block owns 16 weight rows (GLU: 8 gate and the same 8 up columns, so that
// a 2048-column block still makes 256 blocks) and all tokens.  NW wavefronts
// stream the weights; LIN blocks have XW more, which work on the adapters
// meanwhile.
template <int MODE, bool BF16, int NI, int NW, int RING, int XW>
__global__ __launch_bounds__(64 * (NW + XW)) void dense_skinny_kernel(DenseArgs a)
{
    using S = Stream<BF16, NI, 1, RING>;
    __shared__ __align__(1024) uint16_t ring0[NW * S::kHalves], ring1[NW * S::kHalves], ring2[NW * S::kHalves],
        ring3[RING == 4 ? NW * S::kHalves : 8];
    __shared__ __align__(16) float delta[MODE == DENSE_LIN ? 16 * NI : 1][16];
    static_assert(NI <= NW && NI * 1024 <= S::kHalves * 2, "sums fit the first ring array");
    const int tid = threadIdx.x, l = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    constexpr int kCols = MODE == DENSE_GLU ? 8 : 16;
    const int n0 = blockIdx.x * kCols;
    LDS_AS f32x4 *red = (LDS_AS f32x4 *)((LDS_AS uint16_t *)ring0);
    constexpr int kStep = S::kHalves / 8;   // f32x4 between the wavefronts' parts
    if (XW == 0 || w < NW) {
        S st;
        st.p = buf_rsrc(a.p[0], a.pbytes);
        st.q[0] = buf_rsrc(a.q[0], a.qbytes);
        st.q[1] = MODE == DENSE_GLU ? buf_rsrc(a.q[1], a.qbytes) : st.q[0];
        st.init(l, a.K, a.ldp, a.ldq, [](int r) { return (int64_t)r; },
                [&](int r) { return (int64_t)(n0 + (MODE == DENSE_GLU ? r & 7 : r)); });
        f32x4 acc[NI][1];
#pragma unroll
        for (int i = 0; i < NI; ++i)
            acc[i][0] = (f32x4){};
        const int at = w * S::kHalves;
        st.run(w, NW, (LDS_AS uint16_t *)ring0 + at, (LDS_AS uint16_t *)ring1 + at, (LDS_AS uint16_t *)ring2 + at,
               (LDS_AS uint16_t *)ring3 + (RING == 4 ? at : 0), acc);
        // the sums of a wavefront in its own part of the first ring array, which
        // only it has used
#pragma unroll
        for (int i = 0; i < NI; ++i)
            red[w * kStep + 64 * i + l] = acc[i][0];
    } else {
        skinny_expand<BF16, XW>(a, n0, w - NW, l, delta);
    }
    __syncthreads();
    if (w >= NI)
        return;
    const int m = 16 * w + (l & 15);
    auto total = [&](int lane) {
        f32x4 v = red[64 * w + lane];
#pragma unroll
        for (int s = 1; s < NW; ++s)
            v += red[s * kStep + 64 * w + lane];
        return v;
    };
    if constexpr (MODE == DENSE_GLU) {
        // lanes 0..31 hold gate columns 4 (l / 16) + 0..3, lanes 32..63 the same
        // columns of up
        if (l < 32 && m < a.M)
            glu_store<BF16>(a, m, n0 + 4 * (l >> 4), total(l), total(l + 32));
    } else if (m < a.M && n0 + 4 * (l >> 4) < a.N) {
        const f32x4 d = *(const f32x4 *)&delta[m][4 * (l >> 4)];
        lin_store<BF16>(a, m, n0 + 4 * (l >> 4), total(l) + d);
    }
}

template <int MODE, bool BF16>
hipError_t launch_skinny(const DenseArgs &a, hipStream_t s)
{
    constexpr int kCols = MODE == DENSE_GLU ? 8 : 16, XW = MODE == DENSE_LIN ? 4 : 0;
    const unsigned grid = (unsigned)((a.N + kCols - 1) / kCols);
    if (a.M <= 16)
        dense_skinny_kernel<MODE, BF16, 1, 8, 4, XW><<<grid, 64 * (8 + XW), 0, s>>>(a);
    else if (a.M <= 32)
        dense_skinny_kernel<MODE, BF16, 2, 8, 3, XW><<<grid, 64 * (8 + XW), 0, s>>>(a);
    else
        dense_skinny_kernel<MODE, BF16, 4, 4, 3, XW><<<grid, 64 * (4 + XW), 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace moe
