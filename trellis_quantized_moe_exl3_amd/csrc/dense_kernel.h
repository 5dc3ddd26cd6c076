// The tile kernel of the dense operators and its epilogues (see DenseMode).
#pragma once

#include "dense_gemm.h"

namespace moe {

// act(g) and, for the backward pass, its slope.  GELU's tanh form is written
// through the logistic function, 0.5 (1 + tanh z) = 1 / (1 + e^-2z), which
// keeps the relative accuracy of its small negative tail.
MOE_DEV float logistic(float z) { return __builtin_amdgcn_rcpf(1.0f + __expf(-z)); }

constexpr float kGeluK = 0.7978845608028654f;   // sqrt(2 / pi)
constexpr float kGeluC = 0.044715f;

MOE_DEV float act_value(int act, float g)
{
    if (act == MOE_EXL3_ACT_SILU)
        return silu_f(g);
    return g * logistic(2.0f * kGeluK * (g + kGeluC * g * g * g));
}

MOE_DEV void act_value_slope(int act, float g, float &v, float &d)
{
    if (act == MOE_EXL3_ACT_SILU) {
        const float p = logistic(g);
        v = g * p;
        d = p * (1.0f + g * (1.0f - p));
    } else {
        const float p = logistic(2.0f * kGeluK * (g + kGeluC * g * g * g));
        v = g * p;
        d = p + 2.0f * g * p * (1.0f - p) * kGeluK * (1.0f + 3.0f * kGeluC * g * g);
    }
}

// ---- one tile kernel: shapes per mode

template <int MODE>
struct DenseTraits {
    static constexpr int kPL = MODE == DENSE_DW ? KS : KC;
    static constexpr int kQL = (MODE == DENSE_DX || MODE == DENSE_DW) ? KS : KC;
};

constexpr int kDenseWM = 2, kDenseWN = 2;                     // wavefronts over m and n
constexpr int kDenseNW = kDenseWM * kDenseWN;
constexpr int kDenseTM = kDenseBM / kDenseWM, kDenseTN = kDenseBN / kDenseWN;
constexpr int kDenseNI = kDenseTM / 16, kDenseNJ = kDenseTN / 16;

// Result columns n0 + .. of a tile: GLU tiles hold BN / 2 columns of both
// projections, interleaved by 32 (tile rows 64 s + 0..31 of Q are gate columns
// 32 s + .., the next 32 the same columns of up), so that a wavefront's 64
// tile columns hold gate and up of the same 32 intermediate columns.
template <int MODE>
constexpr int kDenseCols = MODE == DENSE_GLU ? kDenseBN / 2 : kDenseBN;

// Four consecutive columns n of row m: h, and pre where it is kept (in fp32:
// 16-bit pre-activations would add their rounding to every gradient).
template <bool BF16>
MOE_DEV void glu_store(const DenseArgs &a, int m, int n, f32x4 g, f32x4 u)
{
    float h[4];
#pragma unroll
    for (int r = 0; r < 4; ++r)
        h[r] = act_value(a.act, g[r]) * u[r];
    *(u32x2 *)(a.out[0] + (int64_t)m * a.ldo + n) = (u32x2){pack16<BF16>(h[0], h[1]), pack16<BF16>(h[2], h[3])};
    if (a.pre) {
        float *p = a.pre + (int64_t)m * a.N + n;
        *(f32x4 *)p = g;
        *(f32x4 *)(p + (int64_t)a.M * a.N) = u;
    }
}

// Four consecutive columns n of row m of y, with the base added.
template <bool BF16>
MOE_DEV void lin_store(const DenseArgs &a, int m, int n, f32x4 y)
{
    if (a.base) {
        const u32x2 b = *(const u32x2 *)(a.base + (int64_t)m * a.ldbase + n);
        y[0] += act_to_f32<BF16>((uint16_t)b[0]);
        y[1] += act_to_f32<BF16>((uint16_t)(b[0] >> 16));
        y[2] += act_to_f32<BF16>((uint16_t)b[1]);
        y[3] += act_to_f32<BF16>((uint16_t)(b[1] >> 16));
    }
    *(u32x2 *)(a.out[0] + (int64_t)m * a.ldo + n) = (u32x2){pack16<BF16>(y[0], y[1]), pack16<BF16>(y[2], y[3])};
}

// Epilogue of the 16 rows m0 .. of a wavefront's NJ column blocks from n0 on
// (GLU: n0 is the first of its NJ / 2 x 16 intermediate columns).
template <int MODE, bool BF16, int NJ>
MOE_DEV void dense_store(const DenseArgs &a, int z, int m0, int n0, int l, f32x4 (&v)[NJ])
{
    const int m = m0 + (l & 15), nl = 4 * (l >> 4);
    if (m >= a.M)
        return;
    constexpr int kBlocks = MODE == DENSE_GLU ? NJ / 2 : NJ;
#pragma unroll
    for (int j = 0; j < kBlocks; ++j) {
        const int n = n0 + 16 * j + nl;
        if (n >= a.N)
            continue;
        if constexpr (MODE == DENSE_GLU)
            glu_store<BF16>(a, m, n, v[j], v[j + kBlocks]);
        else if constexpr (MODE == DENSE_LIN)
            lin_store<BF16>(a, m, n, v[j]);
        else
            *(u32x2 *)(a.out[MODE == DENSE_DW ? z : 0] + (int64_t)m * a.ldo + n) =
                (u32x2){pack16<BF16>(v[j][0], v[j][1]), pack16<BF16>(v[j][2], v[j][3])};
    }
}

// The adapters' share of a wavefront's NI x NJ blocks: for each adapter that
// some of its tokens name, B_a's rows against s_a x A_a^T of the tokens (the
// shrink's sums, rounded to 16 bits for the matrix cores), added to the
// accumulators of that adapter's tokens only: another token's sum never meets
// a product with this adapter, not even times zero, so one adapter's
// infinities stay with its own tokens.
template <bool BF16, int NI, int NJ>
MOE_DEV void lora_expand(const DenseArgs &a, int m0, int n0, int l, f32x4 (&acc)[NI][NJ])
{
    const LoraArgs &lo = a.lora;
    int id[NI];
    uint32_t left = 0;   // bit i: this lane's token of block i is not done yet
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int t = m0 + 16 * i + (l & 15);
        id[i] = t < a.M ? lo.ids[t] : -1;
        if (id[i] < 0 || id[i] >= lo.n)
            id[i] = -1;
        else
            left |= 1u << i;
    }
    for (;;) {
        const uint64_t any = __ballot(left != 0);
        if (!any)
            break;
        int mine = 0;
#pragma unroll
        for (int i = NI - 1; i >= 0; --i)
            mine = (left >> i) & 1 ? id[i] : mine;
        const int e = __builtin_amdgcn_readlane(mine, __ffsll((unsigned long long)any) - 1);
        const float sc = lo.scales ? lo.scales[e] : 1.0f;
        const int rk = lo.ranks ? min(max(lo.ranks[e], 0), lo.rank) : lo.rank;
        for (int k0 = 0; k0 < rk; k0 += 32) {
            const int k = k0 + 8 * (l >> 4);
            u32x4 q[NJ];
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                const int n = n0 + 16 * j + (l & 15);
                q[j] = (u32x4){};
                if (n < a.N && k < rk) {
                    q[j] = *(const u32x4 *)(lo.b + ((int64_t)e * a.N + n) * lo.rank + k);
                    // columns from the adapter's own rank on are not part of it
#pragma unroll
                    for (int d = 0; d < 4; ++d)
                        q[j][d] &= (k + 2 * d < rk ? 0xFFFFu : 0u) | (k + 2 * d + 1 < rk ? 0xFFFF0000u : 0u);
                }
            }
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const bool hit = id[i] == e;
                if (!__ballot(hit))
                    continue;
                float u[8] = {};
                if (hit && k < rk) {
                    const int64_t t = m0 + 16 * i + (l & 15);
                    for (int z = 0; z < lo.splits; ++z) {
                        const f32x4 *p = (const f32x4 *)(lo.mid + ((int64_t)z * a.M + t) * lo.rpad + k);
                        const f32x4 x0 = p[0], x1 = p[1];
#pragma unroll
                        for (int d = 0; d < 4; ++d) {
                            u[d] += x0[d];
                            u[4 + d] += x1[d];
                        }
                    }
                }
                u32x4 p;
#pragma unroll
                for (int d = 0; d < 4; ++d)
                    p[d] = pack16<BF16>(u[2 * d] * sc, u[2 * d + 1] * sc);
#pragma unroll
                for (int j = 0; j < NJ; ++j) {
                    const f32x4 y = dense_mfma<BF16>(q[j], p, (f32x4){});
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        acc[i][j][r] = hit ? acc[i][j][r] + y[r] : acc[i][j][r];
                }
            }
        }
#pragma unroll
        for (int i = 0; i < NI; ++i)
            if (id[i] == e)
                left &= ~(1u << i);
    }
}

// Fragments of one stage: NI row blocks of P and NJ of Q.
struct DenseFrags {
    u32x4 p[kDenseNI], q[kDenseNJ];
};

template <int MODE, bool BF16>
struct DenseTile {
    using TR = DenseTraits<MODE>;
    using OP = Operand<kDenseBM, TR::kPL, kDenseNW>;
    using OQ = Operand<kDenseBN, TR::kQL, kDenseNW>;
    static constexpr int kLoads = OP::kLoads + OQ::kLoads;
    OP po;
    OQ qo;
    __amdgpu_buffer_rsrc_t pr[2], qr[2];
    int w, nsk, send, kend;   // stages per segment, first stage past this block's share, K
    uint32_t pstep, qstep;
    uint32_t pbase, qbase;

    MOE_DEV void load(int s, LDS_AS uint16_t *ring)
    {
        const bool second = MODE == DENSE_DX && s >= nsk;
        const int k0 = kDenseBK * (second ? s - nsk : s);
        const int end = s < send ? kend : 0;
        po.issue(second ? pr[1] : pr[0], ring, w, k0, end, pstep);
        qo.issue(second ? qr[1] : qr[0], ring + kDenseBM * kDenseBK, w, k0, end, qstep);
    }
    MOE_DEV void read(const LDS_AS uint16_t *ring, DenseFrags &f)
    {
#pragma unroll
        for (int i = 0; i < kDenseNI; ++i)
            f.p[i] = OP::frag(ring, pbase, i);
#pragma unroll
        for (int j = 0; j < kDenseNJ; ++j)
            f.q[j] = OQ::frag(ring + kDenseBM * kDenseBK, qbase, j);
    }
    // Stage s in ring slot `cur`, whose fragments `f` were read during stage
    // s - 1.  "At most 2 loads' worth outstanding" (stages s + 2 and s + 3)
    // proves that this wavefront's loads of stage s + 1 have landed; past the
    // barrier every wavefront's have, and every wavefront has read slot `cur`,
    // which stage s + 4 refills.
    MOE_DEV void stage(int s, LDS_AS uint16_t *cur, const LDS_AS uint16_t *next, const DenseFrags &f, DenseFrags &fn,
                       f32x4 (&acc)[kDenseNI][kDenseNJ])
    {
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0)
        wait_vmcnt<2 * kLoads>();
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
        load(s + 4, cur);
        read(next, fn);
#pragma unroll
        for (int i = 0; i < kDenseNI; ++i)
#pragma unroll
            for (int j = 0; j < kDenseNJ; ++j)
                acc[i][j] = dense_mfma<BF16>(f.q[j], f.p[i], acc[i][j]);
    }
    MOE_DEV void run(int s0, LDS_AS uint16_t *r0, LDS_AS uint16_t *r1, LDS_AS uint16_t *r2, LDS_AS uint16_t *r3,
                     f32x4 (&acc)[kDenseNI][kDenseNJ])
    {
        if (s0 >= send)
            return;
        load(s0, r0);
        load(s0 + 1, r1);
        load(s0 + 2, r2);
        load(s0 + 3, r3);
        __builtin_amdgcn_sched_barrier(0);
        wait_vmcnt<3 * kLoads>();
        __builtin_amdgcn_s_barrier();
        DenseFrags f0, f1;
        read(r0, f0);
        for (int s = s0; s < send; s += 4) {
            stage(s, r0, r1, f0, f1, acc);
            stage(s + 1, r1, r2, f1, f0, acc);
            stage(s + 2, r2, r3, f0, f1, acc);
            stage(s + 3, r3, r0, f1, f0, acc);
        }
        wait_vmcnt<0>();   // the loads past the end still write LDS
    }
};

template <int MODE, bool BF16>
__global__ __launch_bounds__(64 * kDenseNW, 2) void dense_kernel(DenseArgs a)
{
    using T = DenseTile<MODE, BF16>;
    constexpr int kHalves = (kDenseBM + kDenseBN) * kDenseBK;
    __shared__ __align__(1024) uint16_t ring0[kHalves], ring1[kHalves], ring2[kHalves], ring3[kHalves];
    const int tid = threadIdx.x, l = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = w / kDenseWN, wn = w % kDenseWN;
    const int tiles = a.mt * a.nt;
    const int split = blockIdx.x / tiles;
    int m, n;
    dense_tile(blockIdx.x - split * tiles, tiles, a.mt, a.nt, m, n);
    // DW: the row tiles of the second tensor follow those of the first
    const int half = MODE == DENSE_DW ? a.mt / 2 : a.mt;
    const int z = m >= half ? 1 : 0;
    const int m0 = (m - z * half) * kDenseBM, n0 = n * kDenseCols<MODE>;

    T t;
    t.w = w;
    t.kend = a.K;
    t.nsk = (a.K + kDenseBK - 1) / kDenseBK;
    const int s0 = split * a.per;
    t.send = min(s0 + a.per, MODE == DENSE_DX ? 2 * t.nsk : t.nsk);
    const int ztensor = MODE == DENSE_DW ? z : 0;
    t.pr[0] = buf_rsrc(a.p[ztensor], a.pbytes);
    t.pr[1] = MODE == DENSE_DX ? buf_rsrc(a.p[1], a.pbytes) : t.pr[0];
    if constexpr (MODE == DENSE_GLU) {
        // a wavefront's loads (16 tile rows each) all lie in one projection
        static_assert(kDenseNW % 4 == 0, "projection of a wavefront's loads");
        t.qr[0] = buf_rsrc(a.q[(w >> 1) & 1], a.qbytes);
        t.qr[1] = t.qr[0];
    } else {
        t.qr[0] = buf_rsrc(a.q[0], a.qbytes);
        t.qr[1] = MODE == DENSE_DX ? buf_rsrc(a.q[1], a.qbytes) : t.qr[0];
    }
    if constexpr (T::TR::kPL == KC) {
        t.po.init_kc(w, l, a.ldp, [&](int r) { return (int64_t)(m0 + r); });
        t.pstep = 2;
    } else {
        t.po.init_ks(w, l, a.ldp, m0);
        t.pstep = (uint32_t)(2 * a.ldp);
    }
    if constexpr (T::TR::kQL == KC) {
        t.qo.init_kc(w, l, a.ldq, [&](int r) {
            return (int64_t)(n0 + (MODE == DENSE_GLU ? 32 * (r >> 6) + (r & 31) : r));
        });
        t.qstep = 2;
    } else {
        t.qo.init_ks(w, l, a.ldq, n0);
        t.qstep = (uint32_t)(2 * a.ldq);
    }
    t.pbase = T::OP::frag_base(l, wm * kDenseTM);
    t.qbase = T::OQ::frag_base(l, wn * kDenseTN);

    f32x4 acc[kDenseNI][kDenseNJ];
#pragma unroll
    for (int i = 0; i < kDenseNI; ++i)
#pragma unroll
        for (int j = 0; j < kDenseNJ; ++j)
            acc[i][j] = (f32x4){};
    t.run(s0, (LDS_AS uint16_t *)ring0, (LDS_AS uint16_t *)ring1, (LDS_AS uint16_t *)ring2, (LDS_AS uint16_t *)ring3,
          acc);

    if (a.splits > 1) {
        f32x4 *part = (f32x4 *)a.part + ((int64_t)blockIdx.x * kDenseNI * kDenseNJ) * (64 * kDenseNW) + tid;
#pragma unroll
        for (int i = 0; i < kDenseNI; ++i)
#pragma unroll
            for (int j = 0; j < kDenseNJ; ++j)
                part[(i * kDenseNJ + j) * (64 * kDenseNW)] = acc[i][j];
        return;
    }
    const int mw = m0 + wm * kDenseTM, nw = n0 + wn * (kDenseCols<MODE> / kDenseWN);
    if constexpr (MODE == DENSE_LIN)
        if (a.lora.rank > 0)
            lora_expand<BF16, kDenseNI, kDenseNJ>(a, mw, nw, l, acc);
#pragma unroll
    for (int i = 0; i < kDenseNI; ++i)
        dense_store<MODE, BF16, kDenseNJ>(a, z, mw + 16 * i, nw, l, acc[i]);
}

// Sum of the k splits' partial tiles, in split order, and the epilogue: block
// (tile, i) finishes the 16-row blocks i of the tile's wavefronts.
template <int MODE, bool BF16>
__global__ __launch_bounds__(64 * kDenseNW) void dense_finish_kernel(DenseArgs a)
{
    const int tid = threadIdx.x, l = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = w / kDenseWN, wn = w % kDenseWN;
    const int tiles = a.mt * a.nt;
    const int L = blockIdx.x / kDenseNI, i = blockIdx.x % kDenseNI;
    int m, n;
    dense_tile(L, tiles, a.mt, a.nt, m, n);
    const int half = MODE == DENSE_DW ? a.mt / 2 : a.mt;
    const int z = m >= half ? 1 : 0;
    const int m0 = (m - z * half) * kDenseBM, n0 = n * kDenseCols<MODE>;
    const f32x4 *part = (const f32x4 *)a.part + ((int64_t)L * kDenseNI + i) * kDenseNJ * (64 * kDenseNW) + tid;
    const int64_t step = (int64_t)tiles * kDenseNI * kDenseNJ * (64 * kDenseNW);
    f32x4 acc[1][kDenseNJ];
#pragma unroll
    for (int j = 0; j < kDenseNJ; ++j)
        acc[0][j] = part[j * (64 * kDenseNW)];
    for (int k = 1; k < a.splits; ++k)
#pragma unroll
        for (int j = 0; j < kDenseNJ; ++j)
            acc[0][j] += part[k * step + j * (64 * kDenseNW)];
    const int mw = m0 + wm * kDenseTM + 16 * i, nw = n0 + wn * (kDenseCols<MODE> / kDenseWN);
    if constexpr (MODE == DENSE_LIN)
        if (a.lora.rank > 0)
            lora_expand<BF16, 1, kDenseNJ>(a, mw, nw, l, acc);
    dense_store<MODE, BF16, kDenseNJ>(a, z, mw, nw, l, acc[0]);
}

template <int MODE>
hipError_t launch_dense_mode(bool bf16, const DenseArgs &a, hipStream_t s)
{
    const dim3 grid((unsigned)(a.mt * a.nt * a.splits)), block(64 * kDenseNW);
    if (bf16)
        dense_kernel<MODE, true><<<grid, block, 0, s>>>(a);
    else
        dense_kernel<MODE, false><<<grid, block, 0, s>>>(a);
    if (a.splits > 1) {
        const dim3 fin((unsigned)(a.mt * a.nt * kDenseNI));
        if (bf16)
            dense_finish_kernel<MODE, true><<<fin, block, 0, s>>>(a);
        else
            dense_finish_kernel<MODE, false><<<fin, block, 0, s>>>(a);
    }
    return hipGetLastError();
}

}  // namespace moe
