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
// of 64 in turn, RING shares in flight each.  The first NJ loads of a KC operand
// Q (8 rows each) go through q[0], the rest through q[1] (GLU: gate, up).  TWO: a
// second pair of tensors p2, q2 follows along k (DX).
//
// LDS image of an operand's share:
//   KC  128-byte rows of eight 16-byte pieces, piece p of row r in slot
//       p ^ ((r >> 1) & 7): the lanes that a 16-byte LDS read serves together
//       (see dense_gemm.h) hit 16 distinct 4-bank groups
//   KS  one 128-byte row of 64 tile rows for each k, the 32-byte chunk c in slot
//       c ^ g(k), g(k) = k / 2 % 2 + 2 (k / 8 % 2): the eight k that 32 lanes
//       of the transposing read touch hit distinct 8-bank groups
template <bool BF16, int NI, int NJ, int RING, int PL = KC, int QL = KC, bool TWO = false>
struct Stream {
    static constexpr int kLoads = 2 * (NI + NJ);
    static constexpr int kHalves = 16 * (NI + NJ) * 64;   // of one share
    static_assert((PL == KC || NI == 4) && (QL == KC || NJ == 4), "KS rows are 128 bytes");
    __amdgpu_buffer_rsrc_t p, q[2], p2, q2;
    uint32_t off[kLoads];   // byte offset of the lane's 16 bytes at k = 0
    uint32_t pstep, qstep;  // bytes from one k to the next
    int l, kend;

    // KC: the row of load j that lane l fetches, and its first k; KS: its k
    MOE_DEV static int row(int l, int j) { return 8 * j + (l >> 3); }
    MOE_DEV static int first_k(int l, int j) { return 8 * ((l & 7) ^ ((4 * j + (l >> 4)) & 7)); }
    MOE_DEV static int ks_chunk(int k) { return ((k >> 1) & 1) | ((k >> 2) & 2); }

    // prow, qrow: memory row of tile row r (KC), or memory column of tile row 0
    // (KS, called with 0)
    template <int L, int N, class F>
    MOE_DEV static void offsets(uint32_t *o, int l, int64_t ld, F row_of)
    {
#pragma unroll
        for (int j = 0; j < 2 * N; ++j) {
            if constexpr (L == KC) {
                o[j] = (uint32_t)((row_of(row(l, j)) * ld + first_k(l, j)) * 2);
            } else {
                const int k = row(l, j);
                const int c = 16 * (((l & 7) >> 1) ^ ks_chunk(k)) + 8 * (l & 1);
                o[j] = (uint32_t)((k * ld + row_of(0) + c) * 2);
            }
        }
    }
    template <class FP, class FQ>
    MOE_DEV void init(int lane, int K, int64_t ldp, int64_t ldq, FP prow, FQ qrow)
    {
        l = lane;
        kend = K;
        pstep = PL == KC ? 2u : (uint32_t)(2 * ldp);
        qstep = QL == KC ? 2u : (uint32_t)(2 * ldq);
        offsets<PL, NI>(off, l, ldp, prow);
        offsets<QL, NJ>(off + 2 * NI, l, ldq, qrow);
    }
    MOE_DEV void load(int share, LDS_AS uint16_t *lds)
    {
        const int most = (kend + 63) / 64;
        const bool second = TWO && share >= most;
        const int k0 = 64 * (second ? share - most : share);
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            const bool isq = j >= 2 * NI;
            const int jj = isq ? j - 2 * NI : j;
            const int k = k0 + ((isq ? QL : PL) == KC ? first_k(l, jj) : row(l, jj));
            const uint32_t o = k < kend ? off[j] + (uint32_t)k0 * (isq ? qstep : pstep) : kOutOfRange;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(!isq ? (second ? p2 : p)
                                                     : second                ? q2
                                                     : QL == KS || jj < NJ   ? q[0]
                                                                             : q[1],
                                                     (LDS_AS void *)(lds + 512 * j), 16, o, 0, 0, 0);
        }
    }
    // Fragments of the half h (32 k) of a share: N blocks of 16 tile rows.
    template <int L, int N>
    MOE_DEV static void read(const LDS_AS uint16_t *lds, int l, int h, u32x4 (&f)[N])
    {
        const LDS_AS char *at = (const LDS_AS char *)lds;
        if constexpr (L == KC) {
            const uint32_t base = (uint32_t)((l & 15) * 128 + (((l >> 4) ^ ((l & 15) >> 1)) << 4)) ^ (64u * h);
#pragma unroll
            for (int i = 0; i < N; ++i)
                f[i] = *(const LDS_AS u32x4 *)(at + base + 2048 * i);
        } else {
            const int k = 32 * h + 8 * (l >> 4) + ((l & 15) >> 2);
            const uint32_t base = (uint32_t)(k * 128 + (ks_chunk(k) << 5) + (l & 3) * 8);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const u32x2 lo = tr_read(at + (base ^ (uint32_t)(i << 5)));
                const u32x2 hi = tr_read(at + (base ^ (uint32_t)(i << 5)) + 512);
                f[i] = (u32x4){lo[0], lo[1], hi[0], hi[1]};
            }
        }
    }
    MOE_DEV static void fragments(const LDS_AS uint16_t *cur, int l, u32x4 (&pf)[2][NI], u32x4 (&qf)[2][NJ])
    {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            read<PL, NI>(cur, l, h, pf[h]);
            read<QL, NJ>(cur + 1024 * NI, l, h, qf[h]);
        }
    }
    // Wait for the share in `cur` (the RING - 1 shares after it stay in
    // flight), read its fragments, refill it, multiply.
    MOE_DEV void step(int refill, LDS_AS uint16_t *cur, f32x4 (&acc)[NI][NJ])
    {
        __builtin_amdgcn_sched_barrier(0);
        wait_vmcnt<(RING - 1) * kLoads>();
        u32x4 pf[2][NI], qf[2][NJ];
        fragments(cur, l, pf, qf);
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
    MOE_DEV int shares() const { return (TWO ? 2 : 1) * ((kend + 63) / 64); }
    // Shares first, first + stride, .. below end of the operands.  (Loads past the
    // operands read zeros; those past an earlier end are never multiplied: RING 1.)
    MOE_DEV void run(int first, int stride, int end, LDS_AS uint16_t *r0, LDS_AS uint16_t *r1, LDS_AS uint16_t *r2,
                     LDS_AS uint16_t *r3, f32x4 (&acc)[NI][NJ])
    {
        static_assert(RING >= 1 && RING <= 4, "ring arrays");
        if (first >= end)
            return;
        load(first, r0);
        if constexpr (RING >= 2)
            load(first + stride, r1);
        if constexpr (RING >= 3)
            load(first + 2 * stride, r2);
        if constexpr (RING >= 4)
            load(first + 3 * stride, r3);
        for (int s = first; s < end; s += RING * stride) {
            step(s + RING * stride, r0, acc);
            if constexpr (RING >= 2)
                step(s + (RING + 1) * stride, r1, acc);
            if constexpr (RING >= 3)
                step(s + (RING + 2) * stride, r2, acc);
            if constexpr (RING >= 4)
                step(s + (RING + 3) * stride, r3, acc);
        }
        wait_vmcnt<0>();   // the loads past the end still write LDS
    }
};

// ---- adapters: x A^T

// The adapter and the rank of token t: -1 and 0 for none.
MOE_DEV void token_adapter(const LoraArgs &lo, int t, int T, int &id, int &rk)
{
    id = t < T ? lo.ids[t] : -1;
    if (id < 0 || id >= lo.n)
        id = -1;
    rk = id < 0 ? 0 : lo.ranks ? min(max(lo.ranks[id], 0), lo.rank) : lo.rank;
}

// The status bits of one token's id and its adapter's rank.
MOE_DEV int id_faults(const LoraArgs &lo, int id)
{
    if (id < 0 || id >= lo.n)
        return id == -1 ? 0 : (int)MOE_EXL3_STATUS_BAD_INDEX;
    if (!lo.ranks)
        return 0;
    const int rank = lo.ranks[id];
    return rank < 0 || rank > lo.rank ? (int)MOE_EXL3_STATUS_BAD_WIDTH : 0;
}

// sum += this wavefront's k share of scales[e] x[t] A_e^T, rows r0 .. r0 + 16 NR
// of A_e, for the 16 tokens of the lanes (lane l: token l % 16 with adapter id
// and rank, -1: none); once per adapter that they name.
template <bool BF16, int NR, int RING, class F>
MOE_DEV void lora_rows(const LoraArgs &lo, int id, int rank, int r0, int l, int w, int nw, int K, int64_t ldx,
                       __amdgpu_buffer_rsrc_t xr, F row, LDS_AS uint16_t *ring0, LDS_AS uint16_t *ring1,
                       LDS_AS uint16_t *ring2, LDS_AS uint16_t *ring3, f32x4 (&sum)[NR])
{
    Stream<BF16, 1, NR, RING> st;
    st.p = xr;
    st.init(l, K, ldx, K, row, [&](int r) { return (int64_t)(r0 + r); });
    uint64_t left = __ballot(rank > r0);   // without rows here there is nothing to add
    while (left) {
        const int at = __ffsll((unsigned long long)left) - 1;
        const int e = __builtin_amdgcn_readlane(id, at), rk = __builtin_amdgcn_readlane(rank, at);
        const bool mine = id == e;
        left &= ~__ballot(mine);
        const float sc = lo.scales ? lo.scales[e] : 1.0f;
        // rows from the adapter's own rank on lie past its buffer: zeros
        st.q[0] = buf_rsrc(lo.a + (int64_t)e * lo.rank * K, (uint32_t)rk * (uint32_t)K * 2u);
        st.q[1] = st.q[0];
        f32x4 acc[1][NR] = {};
        st.run(w, nw, st.shares(), ring0, ring1, ring2, ring3, acc);
        if (mine)
#pragma unroll
            for (int j = 0; j < NR; ++j)
                sum[j] = acc[0][j] * sc;
    }
}

// ---- the block and the projection for few tokens

// Result columns of a block with 16 NJ weight rows.
template <int MODE>
constexpr int skinny_cols(int nj) { return MODE == DENSE_GLU ? 8 * nj : 16 * nj; }

// delta[t][16 columns]: the adapters' rows of tokens t = w, w + XW, .. , kBatch
// at a time with all their loads in flight: lane l takes column l / 4 and the k
// octets l % 4 + 0, 4, .. of the token's adapter (four lanes to 64 bytes of a
// row of B), summed in fp32.  x A^T comes in fp32: 16 bits would round it for
// nothing, and lose values that fp16 does not hold.  Ranks are masked only in the
// 32 that an adapter's own rank ends in (64 tokens, 4096 x 4096, 64 adapters of
// 128: 43.8 us a call with masks everywhere, 39.7).
template <bool BF16, int NI, int XW>
MOE_DEV void skinny_expand(const DenseArgs &a, int n0, int w, int l, float (*delta)[16])
{
    const LoraArgs &lo = a.lora;
    int mine, rank;   // of token l
    token_adapter(lo, l, a.M, mine, rank);
    const int c = l >> 2, n = min(n0 + c, a.N - 1);
    constexpr int kBatch = 16 * NI / XW;   // tokens of a wavefront
    int rk[kBatch], most = 0;
    const uint16_t *bp[kBatch];
    const float *up[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
        const int t = w + b * XW;   // below 16 NI <= 64
        rk[b] = __builtin_amdgcn_readlane(rank, t);
        most = max(most, rk[b]);
        const int e = max(__builtin_amdgcn_readlane(mine, t), 0);
        bp[b] = lo.b + ((int64_t)e * a.N + n) * lo.rank;
        up[b] = (const float *)lo.mid + (int64_t)min(t, a.M - 1) * lo.rpad;
    }
    float sum[kBatch] = {};
    for (int k0 = 0; k0 < most; k0 += 32) {
        const int k = k0 + 8 * (l & 3);
        u32x4 bv[kBatch];
        f32x4 uv[kBatch][2];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            bv[b] = *(const u32x4 *)(bp[b] + min(k, lo.rank - 8));
            uv[b][0] = *(const f32x4 *)(up[b] + k);
            uv[b][1] = *(const f32x4 *)(up[b] + k + 4);
        }
        __builtin_amdgcn_sched_barrier(0);   // all loads first
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            if (k0 >= rk[b])
                continue;
            float y[8];
#pragma unroll
            for (int d = 0; d < 8; ++d)
                y[d] = act_to_f32<BF16>((uint16_t)(bv[b][d >> 1] >> (16 * (d & 1)))) * uv[b][d >> 2][d & 3];
            if (k0 + 32 > rk[b])
#pragma unroll
                for (int d = 0; d < 8; ++d)
                    y[d] = k + d < rk[b] ? y[d] : 0.0f;
#pragma unroll
            for (int d = 0; d < 8; ++d)
                sum[b] += y[d];
        }
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
        sum[b] += __shfl_xor(sum[b], 1);
        sum[b] += __shfl_xor(sum[b], 2);
        if ((l & 3) == 0)
            delta[w + b * XW][c] = sum[b];
    }
}

// skinny_expand of one token of rank at most 32 with x A^T computed here, by the
// XW wavefronts of the block that do not stream weights (one barrier of the
// whole block between the two products).
template <bool BF16, int XW>
MOE_DEV void fused_expand(const DenseArgs &a, int n0, int w, int l, float (*delta)[16])
{
    using S = Stream<BF16, 1, 2, 3>;
    __shared__ __align__(1024) uint16_t ring0[XW * S::kHalves], ring1[XW * S::kHalves], ring2[XW * S::kHalves];
    const LoraArgs &lo = a.lora;
    int id, rank;   // of token l % 16: the one in lanes 0, 16, ..
    token_adapter(lo, l & 15, a.M, id, rank);
    if (blockIdx.x == 0 && w == 0 && l == 0)
        *lo.status = id_faults(lo, lo.ids[0]);
    // B's rows for the second product: lane l takes column l / 4, ranks k .. k + 7
    const int c = l >> 2, n = min(n0 + c, a.N - 1), k = 8 * (l & 3);
    const int e = max(__builtin_amdgcn_readfirstlane(id), 0), rk = __builtin_amdgcn_readfirstlane(rank);
    u32x4 bv = {};
    if (k < rk)
        bv = *(const u32x4 *)(lo.b + ((int64_t)e * a.N + n) * lo.rank + k);
    f32x4 sum[2] = {};
    const int at = w * S::kHalves;
    lora_rows<BF16, 2, 3>(lo, id, rank, 0, l, w, XW, lo.k, a.ldp, buf_rsrc(a.p[0], a.pbytes),
                          [](int r) { return (int64_t)r; }, (LDS_AS uint16_t *)ring0 + at,
                          (LDS_AS uint16_t *)ring1 + at, (LDS_AS uint16_t *)ring2 + at, nullptr, sum);
    LDS_AS f32x4 *red = (LDS_AS f32x4 *)((LDS_AS uint16_t *)ring0);
    constexpr int kStep = S::kHalves / 8;
    red[w * kStep + l] = sum[0];
    red[w * kStep + 64 + l] = sum[1];
    __syncthreads();
    if (w > 0)
        return;
    // ranks k .. k + 3 of token 0 are lane 4 (k % 16)'s of block k / 16, the next
    // four lane 4 (k % 16) + 16's
    f32x4 u0 = {}, u1 = {};
#pragma unroll
    for (int s = 0; s < XW; ++s) {
        u0 += red[s * kStep + 64 * (k >> 4) + 4 * (k & 15)];
        u1 += red[s * kStep + 64 * (k >> 4) + 4 * (k & 15) + 16];
    }
    float y = 0.0f;
#pragma unroll
    for (int d = 0; d < 8; ++d) {
        const float v = act_to_f32<BF16>((uint16_t)(bv[d >> 1] >> (16 * (d & 1)))) * (d < 4 ? u0[d & 3] : u1[d & 3]);
        y += k + d < rk ? v : 0.0f;
    }
    y += __shfl_xor(y, 1);
    y += __shfl_xor(y, 2);
    if ((l & 3) == 0)
        delta[0][c] = y;
}

// Few tokens: bound by the weights' bytes, read once, and at one token by the
// latencies of launch, first loads and the join of the wavefronts (4096 x 2048
// bf16 GLU, 33.6 MB: 8.5 us for 1 to 16 tokens, 3.9 TB/s).
//
// A block owns 16 NJ weight rows (GLU: half of them gate, half the up rows of
// the same columns) and all tokens.  NW wavefronts stream the weights; LIN
// blocks have XW more, which work on the adapters meanwhile.  FUSED: with one
// token's x A^T too (see kFusedRank).
//
// Every block reads all tokens' rows from L2: with 64 tokens, 16 weight rows a
// block move five times the weights' bytes (4096 x 2048: 13.2 us), 32 three times
// (12.4; inter 4096: 26 -> 16.7), where that leaves a block for every other CU.
// A LIN block's adapters are the longer part, and stay with 16 rows (64 tokens,
// 32 adapters of up to 64: 18.0 us, 20.0 with 32).
template <int MODE, bool BF16, int NI, int NJ, int NW, int RING, int XW, bool FUSED = false>
__global__ __launch_bounds__(64 * (NW + XW)) void dense_skinny_kernel(DenseArgs a)
{
    using S = Stream<BF16, NI, NJ, RING>;
    __shared__ __align__(1024) uint16_t ring0[NW * S::kHalves], ring1[NW * S::kHalves],
        ring2[RING >= 3 ? NW * S::kHalves : 8], ring3[RING == 4 ? NW * S::kHalves : 8];
    __shared__ __align__(16) float delta[MODE == DENSE_LIN ? 16 * NI : 1][16];
    static_assert(NI <= NW && NI * NJ * 1024 <= S::kHalves * 2, "sums fit the first ring array");
    const int tid = threadIdx.x, l = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    constexpr int kCols = skinny_cols<MODE>(NJ);
    const int n0 = blockIdx.x * kCols;
    LDS_AS f32x4 *red = (LDS_AS f32x4 *)((LDS_AS uint16_t *)ring0);
    constexpr int kStep = S::kHalves / 8;   // f32x4 between the wavefronts' parts
    if (XW == 0 || w < NW) {
        S st;
        st.p = buf_rsrc(a.p[0], a.pbytes);
        st.q[0] = buf_rsrc(a.q[0], a.qbytes);
        st.q[1] = MODE == DENSE_GLU ? buf_rsrc(a.q[1], a.qbytes) : st.q[0];
        st.init(l, a.K, a.ldp, a.ldq, [](int r) { return (int64_t)r; },
                [&](int r) { return (int64_t)(n0 + (MODE == DENSE_GLU ? r & (kCols - 1) : r)); });
        f32x4 acc[NI][NJ];
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int j = 0; j < NJ; ++j)
                acc[i][j] = (f32x4){};
        const int at = w * S::kHalves;
        st.run(w, NW, st.shares(), (LDS_AS uint16_t *)ring0 + at, (LDS_AS uint16_t *)ring1 + at,
               (LDS_AS uint16_t *)ring2 + (RING >= 3 ? at : 0), (LDS_AS uint16_t *)ring3 + (RING == 4 ? at : 0), acc);
        // the sums of a wavefront in its own part of the first ring array, which
        // only it has used
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int j = 0; j < NJ; ++j)
                red[w * kStep + 64 * (NJ * i + j) + l] = acc[i][j];
        if constexpr (FUSED)
            __syncthreads();
    } else if constexpr (FUSED) {
        fused_expand<BF16, XW>(a, n0, w - NW, l, delta);
    } else if constexpr (XW > 0) {
        skinny_expand<BF16, NI, XW>(a, n0, w - NW, l, delta);
    }
    __syncthreads();
    const int m = 16 * w + (l & 15), c = 4 * (l >> 4);
    if (w >= NI || m >= a.M)
        return;
    auto total = [&](int j, int lane) {
        f32x4 v = red[64 * (NJ * w + j) + lane];
#pragma unroll
        for (int s = 1; s < NW; ++s)
            v += red[s * kStep + 64 * (NJ * w + j) + lane];
        return v;
    };
    if constexpr (MODE == DENSE_GLU && NJ == 1) {
        // lanes 0..31 hold gate columns 4 (l / 16) + 0..3, lanes 32..63 the same
        // columns of up
        if (l < 32)
            glu_store<BF16>(a, m, n0 + c, total(0, l), total(0, l + 32));
    } else if constexpr (MODE == DENSE_GLU) {
        if (n0 + c < a.N)
            glu_store<BF16>(a, m, n0 + c, total(0, l), total(1, l));
    } else {
        static_assert(NJ == 1, "delta holds 16 columns");
        if (n0 + c < a.N)
            lin_store<BF16>(a, m, n0 + c, total(0, l) + *(const f32x4 *)&delta[m][c]);
    }
}

template <int MODE, bool BF16>
hipError_t launch_skinny(const DenseArgs &a, hipStream_t s)
{
    constexpr bool kLin = MODE == DENSE_LIN;
    const unsigned narrow = (unsigned)((a.N + skinny_cols<MODE>(1) - 1) / skinny_cols<MODE>(1));   // blocks
    if constexpr (kLin) {
        if (a.lora.fused) {
            dense_skinny_kernel<MODE, BF16, 1, 1, 8, 2, 4, true><<<narrow, 64 * 12, 0, s>>>(a);
            return hipGetLastError();
        }
    } else if (a.M > 32 && narrow >= 256) {
        dense_skinny_kernel<MODE, BF16, 4, 2, 4, 3, 0><<<(narrow + 1) / 2, 256, 0, s>>>(a);
        return hipGetLastError();
    }
    if (a.M <= 16)
        dense_skinny_kernel<MODE, BF16, 1, 1, 8, 4, kLin ? 4 : 0><<<narrow, 64 * (kLin ? 12 : 8), 0, s>>>(a);
    else if (a.M <= 32)
        dense_skinny_kernel<MODE, BF16, 2, 1, 8, 3, kLin ? 8 : 0><<<narrow, 64 * (kLin ? 16 : 8), 0, s>>>(a);
    else
        dense_skinny_kernel<MODE, BF16, 4, 1, 4, 3, kLin ? 8 : 0><<<narrow, 64 * (kLin ? 12 : 4), 0, s>>>(a);
    return hipGetLastError();
}

// ---- 64 x 64 tiles: all modes, where larger tiles would leave CUs idle

// The adapters' share of a 64 x 64 tile: the adapters that its tokens name are
// dealt to the nw wavefronts of its blocks by their number (so that a token's sum
// is taken in the same order whatever its neighbours), each adding B_a's rows against the
// tokens' s_a x A_a^T to its own part of the sums.
// mine, rank: the adapter of token m0 + l.
template <bool BF16, class S>
MOE_DEV void tile_expand(const DenseArgs &a, int mine, int rank, int m0, int n0, int w, int nw, int l,
                         LDS_AS uint16_t *slot, f32x4 (&acc)[4][4])
{
    const LoraArgs &lo = a.lora;
    uint64_t left = __ballot(mine >= 0);
    if (!left)
        return;
    int id[4];   // of the tokens of this lane's columns
#pragma unroll
    for (int i = 0; i < 4; ++i)
        id[i] = __shfl(mine, 16 * i + (l & 15));
    S st;
    st.p = buf_rsrc(lo.mid, (uint32_t)((int64_t)a.M * lo.rpad * 2));
    st.init(l, 0, lo.rpad, lo.rank, [&](int r) { return (int64_t)(m0 + r); },
            [&](int r) { return (int64_t)(n0 + r); });
    // (e, k0): this wavefront's shares of 64 ranks, one after the other; e < 0
    // past the last
    int e = -1, rk = 0, k0 = 0;
    auto next = [&]() __attribute__((always_inline)) {
        k0 += 64;
        if (k0 < rk)
            return;
        k0 = 0;
        rk = 0;
        e = -1;
        while (left && rk == 0) {
            const int at = __ffsll((unsigned long long)left) - 1;
            const int id0 = __builtin_amdgcn_readlane(mine, at);
            left &= ~__ballot(mine == id0);
            if (id0 % nw == w) {
                e = id0;
                rk = __builtin_amdgcn_readlane(rank, at);
            }
        }
    };
    auto load = [&]() __attribute__((always_inline)) {
        st.kend = rk;   // 0 past the last: the loads read zeros
        st.q[0] = buf_rsrc(lo.b + (int64_t)max(e, 0) * a.N * lo.rank, (uint32_t)((int64_t)a.N * lo.rank * 2));
        st.q[1] = st.q[0];
        st.load(k0 / 64, slot);
    };
    next();
    load();
    while (e >= 0) {
        const int ce = e, crk = rk, ck = k0;
        __builtin_amdgcn_sched_barrier(0);
        wait_vmcnt<0>();
        u32x4 pf[2][4], qf[2][4];
        S::fragments(slot, l, pf, qf);
        __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0): the slot is free
        __builtin_amdgcn_sched_barrier(0);
        next();
        load();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            lora_cut(crk, ck + 32 * h, l, qf[h]);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                lora_products<BF16>(id[i] == ce, pf[h][i], qf[h], acc[i]);
        }
    }
    wait_vmcnt<0>();   // the loads past the end still write LDS
}

// Tile `block` of a launch of NW wavefronts a block; lo, hi: a slot of kTileHalves
// for each of the lower and of the upper half of them, which holds one share at a
// time: a share's fragments are all read before its products, which cover the
// next one's loads.
constexpr int kTileHalves = 16 * 8 * 64;   // of one share of both operands

// Result columns of a tile.
template <int MODE>
constexpr int kTileCols = MODE == DENSE_GLU ? 32 : 64;

template <int MODE, bool BF16, int NW>
MOE_DEV void tile_block(const DenseArgs &a, int block, LDS_AS uint16_t *lo, LDS_AS uint16_t *hi)
{
    using TR = DenseTraits<MODE>;
    using S = Stream<BF16, 4, 4, 1, TR::kPL, TR::kQL, MODE == DENSE_DX>;
    static_assert(S::kHalves == kTileHalves, "ring size");
    const int tid = threadIdx.x, l = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int tiles = a.mt * a.nt, split = block / tiles;
    int m, n;
    dense_tile(block - split * tiles, tiles, a.mt, a.nt, m, n);
    const int half = MODE == DENSE_DW ? a.mt / 2 : a.mt;
    const int z = m >= half ? 1 : 0;
    const int m0 = (m - z * half) * 64, n0 = n * kTileCols<MODE>;
    S st;
    st.p = buf_rsrc(a.p[MODE == DENSE_DW ? z : 0], a.pbytes);
    st.q[0] = buf_rsrc(a.q[0], a.qbytes);
    st.q[1] = MODE == DENSE_GLU ? buf_rsrc(a.q[1], a.qbytes) : st.q[0];
    st.init(l, a.K, a.ldp, a.ldq, [&](int r) { return (int64_t)(m0 + r); },
            [&](int r) { return (int64_t)(n0 + (MODE == DENSE_GLU ? r & 31 : r)); });
    f32x4 acc[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            acc[i][j] = (f32x4){};
    LDS_AS uint16_t *slot = w < NW / 2 ? lo + w * S::kHalves : hi + (w - NW / 2) * S::kHalves;
    int mine = -1, rank = 0;
    if constexpr (MODE == DENSE_LIN)
        token_adapter(a.lora, m0 + l, a.M, mine, rank);
    if constexpr (MODE == DENSE_DX) {
        st.p2 = buf_rsrc(a.p[1], a.pbytes);
        st.q2 = buf_rsrc(a.q[1], a.qbytes);
    }
    st.run(split * a.per + w, NW, min((split + 1) * a.per, st.shares()), slot, nullptr, nullptr, nullptr, acc);
    if constexpr (MODE == DENSE_LIN)
        tile_expand<BF16, S>(a, mine, rank, m0, n0, split * NW + w, a.splits * NW, l, slot, acc);
    // every wavefront's sums in its own slot
    constexpr int kStep = S::kHalves / 8;
    static_assert(kStep >= 16 * 64, "sums fit a slot");
    auto sums = [&](int s) {
        return s < NW / 2 ? (LDS_AS f32x4 *)lo + s * kStep : (LDS_AS f32x4 *)hi + (s - NW / 2) * kStep;
    };
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            ((LDS_AS f32x4 *)slot)[(4 * i + j) * 64 + l] = acc[i][j];
    __syncthreads();
    if (w >= 4)
        return;
    // wavefront i takes the rows i, and its scratch where only it has read
    static_assert(NW >= 4, "a wavefront for each 16 rows");
    f32x4 v[1][4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        v[0][j] = sums(0)[(4 * w + j) * 64 + l];
#pragma unroll
        for (int s = 1; s < NW; ++s)
            v[0][j] += sums(s)[(4 * w + j) * 64 + l];
    }
    if (a.splits > 1) {
        f32x4 *part = (f32x4 *)a.part + (int64_t)block * (16 * 64) + (4 * w) * 64 + l;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            part[64 * j] = v[0][j];
        return;
    }
    dense_store_all<MODE, BF16>(a, z, m0 + 16 * w, n0, l, v, sums(0) + 256 * w);
}

// Grids that 128 x 128 tiles would not fill.  The k of a 64 x 64 tile is cut over
// the wavefronts, so that a block needs a barrier once and short rows of k still
// keep every load in flight; the price is twice the LDS and L2 traffic a product,
// which bounds it (64 KiB into LDS and out of it for each 256 k).  Eight wavefronts
// where a block has its CU to itself, four where two share one (half of them with
// two shares each in flight: 100 tokens, 1032 x 1384: 8.4 us a call, 7.6 like this;
// 200 tokens, 2048 x 2048, 64 adapters: 50.6, 41.3).  333 tokens, 1032 x 1384: 10.5
// us (181 TFLOP/s); 4096 x 2048: 24.6 (454).
template <int MODE, bool BF16, int NW>
__global__ __launch_bounds__(64 * NW, 2) void dense_tile_kernel(DenseArgs a)
{
    __shared__ __align__(1024) uint16_t lds[NW * kTileHalves];
    tile_block<MODE, BF16, NW>(a, blockIdx.x, (LDS_AS uint16_t *)lds, (LDS_AS uint16_t *)lds + NW / 2 * kTileHalves);
}

// Sum of the k splits' partial tiles, in split order, and the epilogue: block
// (tile, i) finishes the 16 rows i.  Bound by what one CU draws of the partial
// tiles, which come from behind the other XCDs' L2, and by their latency: hence
// small blocks with eight splits in flight (32 splits of 16 tiles: 7.1 us; 13.4
// with a block for four of these and one split after the other).
template <int MODE, bool BF16>
__global__ __launch_bounds__(64) void dense_finish_kernel(DenseArgs a)
{
    const int l = threadIdx.x, i = blockIdx.x & 3, tile = blockIdx.x >> 2, tiles = a.mt * a.nt;
    int m, n;
    dense_tile(tile, tiles, a.mt, a.nt, m, n);
    const int half = MODE == DENSE_DW ? a.mt / 2 : a.mt;
    const int z = m >= half ? 1 : 0;
    const f32x4 *part = (const f32x4 *)a.part + (int64_t)tile * (16 * 64) + 4 * i * 64 + l;
    const int64_t step = (int64_t)tiles * (16 * 64);
    f32x4 acc[1][4] = {};
    constexpr int kBatch = 8;   // splits in flight
    for (int k = 0; k < a.splits; k += kBatch) {
        f32x4 v[kBatch][4];
#pragma unroll
        for (int b = 0; b < kBatch; ++b)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                v[b][j] = part[min(k + b, a.splits - 1) * step + 64 * j];
#pragma unroll
        for (int b = 0; b < kBatch; ++b)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                acc[0][j] += k + b < a.splits ? v[b][j] : (f32x4){};
    }
    __shared__ f32x4 lds[256];
    dense_store_all<MODE, BF16>(a, z, (m - z * half) * 64 + 16 * i, n * kTileCols<MODE>, l, acc, (LDS_AS f32x4 *)lds);
}

// Both gradients in one launch: the tiles of dx (64 x 64) and those of dw, 64 x 64
// or (WIDE) 128 x 128, two blocks on a CU.  The longer blocks go first, so that
// the shorter ones fill what they leave (4000 tokens, 512 x 512, dw's twice as
// long: 31.3 us behind dx's, 25.9 before them, when a CU held one).  Bound by
// their number's uneven end and by L2: 509 tokens, 776 x 1304: 16.7 us.
template <bool BF16, bool WIDE>
__global__ __launch_bounds__(256, 2) void dense_grads_kernel(DenseArgs dx, DenseArgs dw, bool dw_first)
{
    static_assert(SmallTile::NW == 4 && SmallTile::RING == 2 && SmallTile::kHalves == 2 * kTileHalves,
                  "the same threads and LDS");
    __shared__ __align__(1024) uint16_t lds0[SmallTile::kHalves], lds1[SmallTile::kHalves];
    LDS_AS uint16_t *r0 = (LDS_AS uint16_t *)lds0, *r1 = (LDS_AS uint16_t *)lds1;
    const int nx = dx.mt * dx.nt, nw = dw.mt * dw.nt, at = blockIdx.x;
    const bool is_dx = dw_first ? at >= nw : at < nx;
    const int block = dw_first == is_dx ? at - (is_dx ? nw : nx) : at;
    if (is_dx) {
        tile_block<DENSE_DX, BF16, 4>(dx, block, r0, r1);
    } else if constexpr (WIDE) {
        dense_block<DENSE_DW, BF16, SmallTile>(dw, block, {r0, r1});
    } else {
        tile_block<DENSE_DW, BF16, 4>(dw, block, r0, r1);
    }
}

template <int MODE, bool BF16>
hipError_t launch_tile(const DenseArgs &a, hipStream_t s)
{
    // eight wavefronts and 128 KiB of LDS while that is one block a CU, two
    // blocks of four wavefronts beyond
    const unsigned grid = (unsigned)(a.mt * a.nt * a.splits);
    if (grid <= 256)
        dense_tile_kernel<MODE, BF16, 8><<<grid, 512, 0, s>>>(a);
    else
        dense_tile_kernel<MODE, BF16, 4><<<grid, 256, 0, s>>>(a);
    if (a.splits > 1)
        dense_finish_kernel<MODE, BF16><<<4 * (unsigned)(a.mt * a.nt), 64, 0, s>>>(a);
    return hipGetLastError();
}

template <int MODE>
hipError_t launch_any(bool bf16, const DenseArgs &a, hipStream_t s)
{
    if (a.bm != kDenseTile)
        return launch_dense_mode<MODE>(bf16, a, s);
    return bf16 ? launch_tile<MODE, true>(a, s) : launch_tile<MODE, false>(a, s);
}

}  // namespace moe
