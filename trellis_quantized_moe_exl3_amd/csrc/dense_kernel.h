// The tile kernel of the dense operators and its epilogues (see DenseMode).
#pragma once

#include <type_traits>

#include "dense_gemm.h"

namespace moe {

// act(g) and, for the backward pass, its slope.  GELU's tanh form is written
// through the logistic function, 0.5 (1 + tanh z) = 1 / (1 + e^-2z), which
// keeps the relative accuracy of its small negative tail.
MOE_DEV float logistic(float z) { return __builtin_amdgcn_rcpf(1.0f + __expf(-z)); }

constexpr float kGeluK = 0.7978845608028654f;   // sqrt(2 / pi)
constexpr float kGeluC = 0.044715f;

template <int ACT>
MOE_DEV float act_value(float g)
{
    if constexpr (ACT == MOE_EXL3_ACT_SILU)
        return silu_f(g);
    else
        return g * logistic(2.0f * kGeluK * (g + kGeluC * g * g * g));
}

MOE_DEV void act_value_slope(int act, float g, float &v, float &d)
{
    if (act == MOE_EXL3_ACT_SILU) {
        const float p = logistic(g);
        v = g * p;
        d = p * (1.0f + g * (1.0f - p));
    } else {
        // past 16 the logistic is 0 or 1 and the slope no longer moves: the cube
        // of a larger gate would overflow against that zero
        const float z = g > 16.0f ? 16.0f : g < -16.0f ? -16.0f : g;
        const float p = logistic(2.0f * kGeluK * (z + kGeluC * z * z * z));
        v = g * p;
        d = p + 2.0f * z * p * (1.0f - p) * kGeluK * (1.0f + 3.0f * kGeluC * z * z);
    }
}

// ---- one tile kernel: shapes per mode

template <int MODE>
struct DenseTraits {
    static constexpr int kPL = MODE == DENSE_DW ? KS : KC;
    static constexpr int kQL = (MODE == DENSE_DX || MODE == DENSE_DW) ? KS : KC;
};

// Tile shapes: WM x WN wavefronts of TM x TN outputs each, RING stages of BK k in
// LDS.  TN = 64 in all of them (see kDenseCols).
template <int BM_, int BN_, int WM_, int WN_, int BK_, int RING_>
struct DenseShape {
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, NW = WM * WN, BK = BK_, RING = RING_;
    static constexpr int kHalves = (BM + BN) * BK;   // of a stage of both operands
    static constexpr int TM = BM / WM, TN = BN / WN, NI = TM / 16, NJ = TN / 16;
    static_assert(TN == 64 && NW % 4 == 0, "GLU column interleave");
    static_assert(BM % 64 == 0 && 64 * NW >= BM, "a thread for each row");
};
using SmallTile = DenseShape<kDenseSmall, kDenseSmall, 2, 2, 64, 2>;   // two on a CU
using AloneTile = DenseShape<kDenseSmall, kDenseSmall, 2, 2, 64, 4>;   // one on a CU
using LargeTile = DenseShape<kDenseLarge, kDenseLarge, 2, 4, 32, 4>;

// Result columns n0 + .. of a tile: GLU tiles hold BN / 2 columns of both
// projections, interleaved by 32 (tile rows 64 s + 0..31 of Q are gate columns
// 32 s + .., the next 32 the same columns of up), so that a wavefront's 64
// tile columns hold gate and up of the same 32 intermediate columns.
template <int MODE, class S>
constexpr int kDenseCols = MODE == DENSE_GLU ? S::BN / 2 : S::BN;

// Four consecutive columns n of row m: h, and pre where it is kept (in fp32:
// 16-bit pre-activations would add their rounding to every gradient).
template <bool BF16>
MOE_DEV void glu_store(const DenseArgs &a, int m, int n, f32x4 g, f32x4 u)
{
    float h[4];
#pragma unroll
    for (int r = 0; r < 4; ++r)
        h[r] = (a.act == MOE_EXL3_ACT_SILU ? act_value<MOE_EXL3_ACT_SILU>(g[r])
                                           : act_value<MOE_EXL3_ACT_GELU_TANH>(g[r])) * u[r];
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

// Eight consecutive values in 16 bits.
template <bool BF16>
MOE_DEV u32x4 pack8(f32x4 a, f32x4 b)
{
    return (u32x4){pack16<BF16>(a[0], a[1]), pack16<BF16>(a[2], a[3]), pack16<BF16>(b[0], b[1]),
                   pack16<BF16>(b[2], b[3])};
}

// Epilogue of the 16 rows m0 .. of a wavefront's 64 tile columns (n0: the first
// result column; GLU: of its 32; ACT: its activation).  The accumulators hold
// four columns of row l % 16: stored as they are, neighbouring lanes would
// write to different rows and every lane be a memory transaction of its own.
// They pass through 4 KiB of LDS that only this wavefront uses (16-byte unit c
// of row r in place c ^ r), so that eight lanes write the 128 bytes of a row
// (GLU: four lanes 64) (2048 tokens, adapters alone, 4096 columns: tile kernel
// 14.2 -> 12.2 us; 10.6 since its stages are 64 ranks).
template <int MODE, bool BF16, int ACT>
MOE_DEV void dense_store(const DenseArgs &a, int z, int m0, int n0, int l, const f32x4 (&v)[4],
                         const u32x4 (&base)[2], LDS_AS f32x4 *lds)
{
    const int r = l & 15;
    wave_lds_fence();   // the rows before these, or the sums, are read
#pragma unroll
    for (int j = 0; j < 4; ++j)
        lds[16 * r + ((4 * j + (l >> 4)) ^ r)] = v[j];
    wave_lds_fence();
    auto at = [&](int row, int unit) { return lds[16 * row + (unit ^ row)]; };
    // one 64-bit address for the 16 rows, 32-bit offsets in them
    uint16_t *out = a.out[MODE == DENSE_DW ? z : 0] + (int64_t)m0 * a.ldo + n0;
    const int left = a.M - m0, ldo = (int)a.ldo;
    if constexpr (MODE == DENSE_GLU) {
        if (a.pre) {
            // eight lanes to the 128 bytes of a row of 32 columns
            float *pg = a.pre + (int64_t)m0 * a.N + n0, *pu = pg + (int64_t)a.M * a.N;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int row = 8 * h + (l >> 3), c = l & 7;
                const f32x4 g = at(row, c), u = at(row, 8 + c);
                if (row < left && n0 + 4 * c < a.N) {
                    *(f32x4 *)(pg + (uint32_t)(row * a.N + 4 * c)) = g;
                    *(f32x4 *)(pu + (uint32_t)(row * a.N + 4 * c)) = u;
                }
            }
        }
        const int row = l >> 2, c = 2 * (l & 3);
        const f32x4 g[2] = {at(row, c), at(row, c + 1)}, u[2] = {at(row, 8 + c), at(row, 9 + c)};
        if (row >= left || n0 + 4 * c >= a.N)
            return;
        f32x4 h[2];
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int d = 0; d < 4; ++d)
                h[q][d] = act_value<ACT>(g[q][d]) * u[q][d];
        *(u32x4 *)(out + (uint32_t)(row * ldo + 4 * c)) = pack8<BF16>(h[0], h[1]);
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int row = 8 * h + (l >> 3), c = 2 * (l & 7);
            f32x4 y[2] = {at(row, c), at(row, c + 1)};
            if (row >= left || n0 + 4 * c >= a.N)
                continue;
            if constexpr (MODE == DENSE_LIN) {
                if (a.base)
#pragma unroll
                    for (int d = 0; d < 8; ++d)
                        y[d >> 2][d & 3] += act_to_f32<BF16>((uint16_t)(base[h][d >> 1] >> (16 * (d & 1))));
            }
            *(u32x4 *)(out + (uint32_t)(row * ldo + 4 * c)) = pack8<BF16>(y[0], y[1]);
        }
    }
}

// The same for N blocks of 16 rows, up to four at a time with the loads of
// their base (LIN) all in flight.
template <int MODE, bool BF16, int N>
MOE_DEV void dense_store_all(const DenseArgs &a, int z, int m0, int n0, int l, const f32x4 (&v)[N][4],
                             LDS_AS f32x4 *lds)
{
#pragma unroll
    for (int i0 = 0; i0 < N; i0 += 4) {
        u32x4 base[4][2] = {};
        if constexpr (MODE == DENSE_LIN)
            if (a.base)
#pragma unroll
                for (int i = i0; i < i0 + 4 && i < N; ++i)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int m = m0 + 16 * i + 8 * h + (l >> 3), n = n0 + 8 * (l & 7);
                        if (m < a.M && n < a.N)
                            base[i - i0][h] = *(const u32x4 *)(a.base + (int64_t)m * a.ldbase + n);
                    }
        if (MODE != DENSE_GLU || a.act == MOE_EXL3_ACT_SILU) {
#pragma unroll
            for (int i = i0; i < i0 + 4 && i < N; ++i)
                dense_store<MODE, BF16, MOE_EXL3_ACT_SILU>(a, z, m0 + 16 * i, n0, l, v[i], base[i - i0], lds);
        } else {
#pragma unroll
            for (int i = i0; i < i0 + 4 && i < N; ++i)
                dense_store<MODE, BF16, MOE_EXL3_ACT_GELU_TANH>(a, z, m0 + 16 * i, n0, l, v[i], base[i - i0], lds);
        }
    }
}

// Fragments of 32 k: NI row blocks of P and NJ of Q.
template <class S>
struct DenseFrags {
    u32x4 p[S::NI], q[S::NJ];
};

template <bool BF16, class S>
MOE_DEV void multiply(const DenseFrags<S> &f, f32x4 (&acc)[S::NI][S::NJ])
{
#pragma unroll
    for (int i = 0; i < S::NI; ++i)
#pragma unroll
        for (int j = 0; j < S::NJ; ++j)
            acc[i][j] = dense_mfma<BF16>(f.q[j], f.p[i], acc[i][j]);
}

// The order of 32 k: the L loads between the first MFMAs, the next fragments'
// reads between the others (7168 tokens, 4096 x 2048: 196.7 -> 193.7 us; reads
// before loads leave too many fragments in registers and spill: 237).  The
// transposing reads' two halves a fragment leave no registers for any order: they
// spill and halve the rate.
template <int MODE, class S, int L>
MOE_DEV void spread()
{
    if constexpr (DenseTraits<MODE>::kPL == KC && DenseTraits<MODE>::kQL == KC) {
        constexpr int kPer = (S::NI * S::NJ - L) / (S::NI + S::NJ);
#pragma unroll
        for (int r = 0; r < L; ++r) {
            __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        }
#pragma unroll
        for (int r = 0; r < S::NI + S::NJ; ++r) {
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x008, kPer, 0);
        }
    }
}

template <int MODE, bool BF16, class S>
struct DenseTile {
    static constexpr int NI = S::NI, NJ = S::NJ;
    using Frags = DenseFrags<S>;
    using TR = DenseTraits<MODE>;
    using OP = Operand<S::BM, TR::kPL, S::NW, S::BK>;
    using OQ = Operand<S::BN, TR::kQL, S::NW, S::BK>;
    static constexpr int kLoads = OP::kLoads + OQ::kLoads;
    static constexpr int kRing = S::RING, kStep = S::BK, kPer = 1;
    OP po;
    OQ qo;
    __amdgpu_buffer_rsrc_t pr[2], qr[2];
    int w, nsk, send, kend;   // stages per segment, all of them, K
    uint32_t pstep, qstep;
    uint32_t pbase, qbase;

    MOE_DEV void load(int s, LDS_AS uint16_t *ring)
    {
        const bool second = MODE == DENSE_DX && s >= nsk;
        const int k0 = S::BK * (second ? s - nsk : s);
        const int end = s < send ? kend : 0;
        po.issue(second ? pr[1] : pr[0], ring, w, k0, end, pstep);
        qo.issue(second ? qr[1] : qr[0], ring + S::BM * S::BK, w, k0, end, qstep);
    }
    MOE_DEV void read(const LDS_AS uint16_t *ring, int h, Frags &f)
    {
#pragma unroll
        for (int i = 0; i < S::NI; ++i)
            f.p[i] = OP::frag(ring, pbase, i, h);
#pragma unroll
        for (int j = 0; j < S::NJ; ++j)
            f.q[j] = OQ::frag(ring + S::BM * S::BK, qbase, j, h);
    }
    // Stage s in ring slot `cur`, whose first fragments f0 were read during stage
    // s - 1; f0 and f1 change places from one 32 k to the next.  "At most RING - 2
    // stages' loads outstanding" (s + 2 .. s + RING - 1) proves that this
    // wavefront's loads of stage s + 1 have landed; past the barrier every
    // wavefront's have, and every wavefront has read slot `cur`, which stage s +
    // RING refills.
    MOE_DEV void stage(int s, LDS_AS uint16_t *cur, const LDS_AS uint16_t *next, Frags &f0, Frags &f1,
                       f32x4 (&acc)[NI][NJ])
    {
        if constexpr (S::BK == 64) {
            read(cur, 1, f1);
            multiply<BF16, S>(f0, acc);
            spread<MODE, S, 0>();
        }
        Frags &last = S::BK == 64 ? f1 : f0, &first = S::BK == 64 ? f0 : f1;
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0)
        wait_vmcnt<(S::RING - 2) * kLoads>();
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
        load(s + S::RING, cur);
        read(next, 0, first);
        multiply<BF16, S>(last, acc);
        spread<MODE, S, kLoads>();
    }
    // `meanwhile` runs once, while the first loads are on their way.
    template <class F>
    MOE_DEV void run(LDS_AS uint16_t *const (&ring)[S::RING], f32x4 (&acc)[NI][NJ], F meanwhile)
    {
        if (send == 0) {
            meanwhile();
            return;
        }
#pragma unroll
        for (int r = 0; r < S::RING; ++r)
            load(r, ring[r]);
        meanwhile();
        __builtin_amdgcn_sched_barrier(0);
        wait_vmcnt<(S::RING - 1) * kLoads>();
        __builtin_amdgcn_s_barrier();
        Frags f0, f1;
        read(ring[0], 0, f0);
        constexpr bool kSwap = S::BK == 32;
        for (int s = 0; s < send; s += S::RING)
#pragma unroll
            for (int r = 0; r < S::RING; r += 2) {
                stage(s + r, ring[r], ring[r + 1], f0, f1, acc);
                stage(s + r + 1, ring[r + 1], ring[(r + 2) % S::RING], kSwap ? f1 : f0, kSwap ? f0 : f1, acc);
            }
        wait_vmcnt<0>();   // the loads past the end still write LDS
    }
};

// The same for 256 x 256 tiles whose P is KC: P in two stages of 64 k (whole
// lines, see dense_kernel), Q in four of 32.
template <int MODE, bool BF16, class S>
struct PairTile {
    static constexpr int NI = S::NI, NJ = S::NJ, kRing = 6;   // slots: P's two, then Q's four
    static constexpr int kPHalves = S::BM * 64, kQHalves = S::BN * 32;
    static constexpr int kStep = 32, kPer = 2;   // k of a stage; stages come in pairs
    using Frags = DenseFrags<S>;
    using TR = DenseTraits<MODE>;
    using OP = Operand<S::BM, KC, S::NW, 64>;
    using OQ = Operand<S::BN, TR::kQL, S::NW, 32>;
    OP po;
    OQ qo;
    __amdgpu_buffer_rsrc_t pr[2], qr[2];
    int w, nsk, send, kend;   // stages per segment (even), all of them, K
    uint32_t pstep, qstep;
    uint32_t pbase, qbase;

    // Stages s and s + 1, s even, of P; stage s of Q.
    MOE_DEV void load_p(int s, LDS_AS uint16_t *slot)
    {
        const bool second = MODE == DENSE_DX && s >= nsk;
        po.issue(second ? pr[1] : pr[0], slot, w, 32 * (second ? s - nsk : s), s < send ? kend : 0, pstep);
    }
    MOE_DEV void load_q(int s, LDS_AS uint16_t *slot)
    {
        const bool second = MODE == DENSE_DX && s >= nsk;
        qo.issue(second ? qr[1] : qr[0], slot, w, 32 * (second ? s - nsk : s), s < send ? kend : 0, qstep);
    }
    MOE_DEV void read(const LDS_AS uint16_t *p, int h, const LDS_AS uint16_t *q, Frags &f)
    {
#pragma unroll
        for (int i = 0; i < NI; ++i)
            f.p[i] = OP::frag(p, pbase, i, h);
#pragma unroll
        for (int j = 0; j < NJ; ++j)
            f.q[j] = OQ::frag(q, qbase, j, 0);
    }
    // Stage s, R = s % 4, whose fragments f were read during stage s - 1.  Odd
    // stages load P for s + 3 and s + 4, every stage then Q for s + 4: younger than
    // the loads of stage s + 1 are those of Q for s + 2 and s + 3, and in even
    // stages of P for s + 2.  Past the barrier every wavefront has read stage s:
    // Q's slot is free, and in odd stages P's.
    template <int R>
    MOE_DEV void stage(int s, LDS_AS uint16_t *const (&ring)[kRing], const Frags &f, Frags &fn, f32x4 (&acc)[NI][NJ])
    {
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0)
        wait_vmcnt<R & 1 ? 2 * OQ::kLoads : OP::kLoads + 2 * OQ::kLoads>();
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (R & 1)
            load_p(s + 3, ring[R / 2 % 2]);
        load_q(s + 4, ring[2 + R % 4]);
        read(ring[(R + 1) / 2 % 2], (R + 1) & 1, ring[2 + (R + 1) % 4], fn);
        multiply<BF16, S>(f, acc);
        spread<MODE, S, OQ::kLoads + (R & 1) * OP::kLoads>();
    }
    template <class F>
    MOE_DEV void run(LDS_AS uint16_t *const (&ring)[kRing], f32x4 (&acc)[NI][NJ], F meanwhile)
    {
        if (send == 0) {
            meanwhile();
            return;
        }
        load_q(0, ring[2]);
        load_p(0, ring[0]);
        load_q(1, ring[3]);
        load_q(2, ring[4]);
        load_p(2, ring[1]);
        load_q(3, ring[5]);
        meanwhile();
        __builtin_amdgcn_sched_barrier(0);
        wait_vmcnt<OP::kLoads + 3 * OQ::kLoads>();
        __builtin_amdgcn_s_barrier();
        Frags f0, f1;
        read(ring[0], 0, ring[2], f0);
        for (int s = 0; s < send; s += 4) {
            stage<0>(s, ring, f0, f1, acc);
            stage<1>(s + 1, ring, f1, f0, acc);
            stage<2>(s + 2, ring, f0, f1, acc);
            stage<3>(s + 3, ring, f1, f0, acc);
        }
        wait_vmcnt<0>();   // the loads past the end still write LDS
    }
};

template <int MODE, class S>
constexpr bool kPairs = S::BM == kDenseLarge && DenseTraits<MODE>::kPL == KC;

template <int MODE, bool BF16, class S>
using TileOf = std::conditional_t<kPairs<MODE, S>, PairTile<MODE, BF16, S>, DenseTile<MODE, BF16, S>>;

// B_a's rows for 32 ranks from k0 on, without what follows the adapter's own
// rank inside an octet (whole octets past it were read as zeros).
template <int NJ>
MOE_DEV void lora_cut(int rk, int k0, int l, u32x4 (&q)[NJ])
{
    if (k0 + 32 <= rk || !(rk & 7))
        return;
    const int k = k0 + 8 * (l >> 4);
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int d = 0; d < 4; ++d)
            q[j][d] &= (k + 2 * d < rk ? 0xFFFFu : 0u) | (k + 2 * d + 1 < rk ? 0xFFFF0000u : 0u);
}

// An adapter's products, q = B_a's rows, p = s_a x A_a^T of 16 tokens, taken
// into the sums of its own tokens (hit) only: another token's sum never meets
// them, not even times zero, so one adapter's infinities stay with its own
// tokens.
template <bool BF16, int NJ>
MOE_DEV void lora_products(bool hit, u32x4 p, const u32x4 (&q)[NJ], f32x4 (&acc)[NJ])
{
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
        const f32x4 y = dense_mfma<BF16>(q[j], p, acc[j]);
#pragma unroll
        for (int r = 0; r < 4; ++r)
            acc[j][r] = hit ? y[r] : acc[j][r];
    }
}

// The adapters of a tile's tokens as a list of stages of BK ranks.
template <int BM, int BK>
struct AdapterJobs {
    int id[BM];                         // adapter of each token, -1: none
    int count;
    uint32_t job[BM * (kMaxRank / BK)]; // adapter | stage << 16 | its rank << 20

    // The tokens' ids, by all threads.
    MOE_DEV void ids_of(const LoraArgs &lo, int m0, int T, int tid)
    {
        if (tid < BM) {
            const int t = m0 + tid, e = t < T ? lo.ids[t] : -1;
            id[tid] = e >= 0 && e < lo.n ? e : -1;
        }
    }
    // One wavefront, the ids being visible: the list, adapters in the order of
    // their first tokens.
    MOE_DEV void build(const LoraArgs &lo, int l)
    {
        int n = 0;
        uint64_t left[BM / 64];
        int mine[BM / 64], rank[BM / 64];
#pragma unroll
        for (int g = 0; g < BM / 64; ++g) {
            mine[g] = id[64 * g + l];
            left[g] = __ballot(mine[g] >= 0);
            rank[g] = lo.rank;
        }
        if (lo.ranks)
#pragma unroll
            for (int g = 0; g < BM / 64; ++g)
                rank[g] = min(max(lo.ranks[max(mine[g], 0)], 0), lo.rank);
#pragma unroll
        for (int g = 0; g < BM / 64; ++g)
            while (left[g]) {
                const int at = __ffsll((unsigned long long)left[g]) - 1;
                const int e = __builtin_amdgcn_readlane(mine[g], at), rk = __builtin_amdgcn_readlane(rank[g], at);
#pragma unroll
                for (int h = g; h < BM / 64; ++h)
                    left[h] &= ~__ballot(mine[h] == e);
                const int stages = (rk + BK - 1) / BK;
                if (l < stages)
                    job[n + l] = (uint32_t)e | (uint32_t)l << 16 | (uint32_t)rk << 20;
                n += stages;
            }
        if (l == 0)
            count = n;
    }
};

// The adapters' share of a tile, added to its accumulators: stages like those
// of the k loop, one for every BK ranks of every adapter that a token of the
// tile names, P = the tokens' s_a x A_a^T, Q = B_a's rows, through the same
// ring.
template <bool BF16, class S, int RING>
MOE_DEV void lora_expand(const DenseArgs &a, int m0, int n0, int tid, const AdapterJobs<S::BM, S::BK> &jobs,
                         LDS_AS uint16_t *const (&pring)[RING], LDS_AS uint16_t *const (&qring)[RING],
                         f32x4 (&acc)[S::NI][S::NJ])
{
    using OP = Operand<S::BM, KC, S::NW, S::BK>;
    using OQ = Operand<S::BN, KC, S::NW, S::BK>;
    constexpr int kLoads = OP::kLoads + OQ::kLoads;
    const LoraArgs &lo = a.lora;
    const int l = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = w / S::WN, wn = w % S::WN;
    __syncthreads();   // the list, and the end of the k loop's reads of the ring
    const int count = __builtin_amdgcn_readfirstlane(jobs.count);
    if (count == 0)
        return;
    OP po;
    OQ qo;
    po.init_kc(w, l, lo.rpad, [&](int r) { return (int64_t)(m0 + r); });
    qo.init_kc(w, l, lo.rank, [&](int r) { return (int64_t)(n0 + r); });
    const __amdgpu_buffer_rsrc_t pr = buf_rsrc(lo.mid, (uint32_t)((int64_t)a.M * lo.rpad * 2));
    const uint32_t bbytes = (uint32_t)((int64_t)a.N * lo.rank * 2);
    const uint32_t pbase = OP::frag_base(l, wm * S::TM), qbase = OQ::frag_base(l, wn * S::TN);
    const int *ids = jobs.id + wm * S::TM + (l & 15);

    auto job_of = [&](int t) __attribute__((always_inline)) {
        return (uint32_t)__builtin_amdgcn_readfirstlane((int)jobs.job[min(t, count - 1)]);
    };
    auto load = [&](int t, LDS_AS uint16_t *pslot, LDS_AS uint16_t *qslot) __attribute__((always_inline)) {
        const uint32_t job = job_of(t);
        const int e = job & 0xFFFF, k0 = S::BK * ((job >> 16) & 15), rk = t < count ? (int)(job >> 20) : 0;
        po.issue(pr, pslot, w, k0, rk, 2);
        qo.issue(buf_rsrc(lo.b + (int64_t)e * a.N * lo.rank, bbytes), qslot, w, k0, rk, 2);
    };
    LDS_AS uint16_t *ps[RING], *qs[RING];   // slots of stages t, t + 1, ..
#pragma unroll
    for (int r = 0; r < RING; ++r) {
        ps[r] = pring[r];
        qs[r] = qring[r];
        if (r < RING - 1)
            load(r, ps[r], qs[r]);
    }
#pragma unroll 1
    for (int t = 0; t < count; ++t) {
        __builtin_amdgcn_sched_barrier(0);
        wait_vmcnt<(RING - 2) * kLoads>();   // the stages after t stay in flight
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
        load(t + RING - 1, ps[RING - 1], qs[RING - 1]);
        const uint32_t job = job_of(t);
        const int e = job & 0xFFFF, k0 = S::BK * ((job >> 16) & 15), rk = job >> 20;
#pragma unroll
        for (int h = 0; h < S::BK / 32; ++h) {
            if (k0 + 32 * h >= rk)
                break;
            u32x4 q[S::NJ];
#pragma unroll
            for (int j = 0; j < S::NJ; ++j)
                q[j] = OQ::frag(qs[0], qbase, j, h);
            lora_cut(rk, k0 + 32 * h, l, q);
#pragma unroll
            for (int i = 0; i < S::NI; i += 2) {
                const u32x4 p0 = OP::frag(ps[0], pbase, i, h), p1 = OP::frag(ps[0], pbase, i + 1, h);
                lora_products<BF16>(ids[16 * i] == e, p0, q, acc[i]);
                lora_products<BF16>(ids[16 * i + 16] == e, p1, q, acc[i + 1]);
                __builtin_amdgcn_sched_barrier(0);   // fragments of two blocks at a time: registers
            }
        }
        __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0): reads done before the next barrier
        LDS_AS uint16_t *p0 = ps[0], *q0 = qs[0];
#pragma unroll
        for (int r = 0; r < RING - 1; ++r) {
            ps[r] = ps[r + 1];
            qs[r] = qs[r + 1];
        }
        ps[RING - 1] = p0;
        qs[RING - 1] = q0;
    }
    wait_vmcnt<0>();   // the loads past the end still write LDS
}

// Tile `block` of a launch.  The ring's slots are arrays apart: of loads into one
// array the compiler waits for all before it reads any.
template <int MODE, bool BF16, class S>
MOE_DEV void dense_block(const DenseArgs &a, int block, LDS_AS uint16_t *const (&ring)[TileOf<MODE, BF16, S>::kRing])
{
    using T = TileOf<MODE, BF16, S>;
    const int tid = threadIdx.x, l = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = w / S::WN, wn = w % S::WN;
    int m, n;
    dense_tile(block, a.mt * a.nt, a.mt, a.nt, m, n);
    // DW: the row tiles of the second tensor follow those of the first
    const int half = MODE == DENSE_DW ? a.mt / 2 : a.mt;
    const int z = m >= half ? 1 : 0;
    const int m0 = (m - z * half) * S::BM, n0 = n * (kDenseCols<MODE, S>);

    T t;
    t.w = w;
    t.kend = a.K;
    t.nsk = (a.K + T::kStep * T::kPer - 1) / (T::kStep * T::kPer) * T::kPer;
    t.send = MODE == DENSE_DX ? 2 * t.nsk : t.nsk;
    const int ztensor = MODE == DENSE_DW ? z : 0;
    t.pr[0] = buf_rsrc(a.p[ztensor], a.pbytes);
    t.pr[1] = MODE == DENSE_DX ? buf_rsrc(a.p[1], a.pbytes) : t.pr[0];
    if constexpr (MODE == DENSE_GLU) {
        // a wavefront's loads all lie in one projection: 32 rows next to each
        // other, or 16 rows and those 16 NW further on
        static_assert(S::BK == 64 ? 8 * T::OQ::kLoads == 32 : S::NW % 4 == 0, "projection of a wavefront's loads");
        t.qr[0] = buf_rsrc(a.q[S::BK == 64 ? w & 1 : (w >> 1) & 1], a.qbytes);
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
    t.pbase = T::OP::frag_base(l, wm * S::TM);
    t.qbase = T::OQ::frag_base(l, wn * S::TN);

    f32x4 acc[S::NI][S::NJ];
#pragma unroll
    for (int i = 0; i < S::NI; ++i)
#pragma unroll
        for (int j = 0; j < S::NJ; ++j)
            acc[i][j] = (f32x4){};
    if constexpr (MODE == DENSE_LIN) {
        __shared__ AdapterJobs<S::BM, S::BK> jobs;
        t.run(ring, acc, [&]() __attribute__((always_inline)) {
            jobs.ids_of(a.lora, m0, a.M, tid);
            __syncthreads();
            if (w == 0)
                jobs.build(a.lora, l);
        });
        if constexpr (kPairs<MODE, S>) {
            lora_expand<BF16, S, 2>(a, m0, n0, tid, jobs, {ring[0], ring[1]}, {ring[2], ring[3]}, acc);
        } else {
            LDS_AS uint16_t *qring[S::RING];
#pragma unroll
            for (int r = 0; r < S::RING; ++r)
                qring[r] = ring[r] + S::BM * S::BK;
            lora_expand<BF16, S, S::RING>(a, m0, n0, tid, jobs, ring, qring, acc);
        }
    } else {
        t.run(ring, acc, [] {});
    }

    const int mw = m0 + wm * S::TM, nw = n0 + wn * ((kDenseCols<MODE, S>) / S::WN);
    __syncthreads();   // the ring is free
    static_assert(S::NW * 4096 <= S::kHalves * 2, "a wavefront's share of the first ring array");
    dense_store_all<MODE, BF16>(a, z, mw, nw, l, acc, (LDS_AS f32x4 *)ring[0] + 256 * w);
}

// The large products.  A tile of BM x BN reads BM + BN rows of each k for BM x BN
// multiply-adds, so the larger the tile the less it asks of L2 and LDS: 256 x 256
// (eight wavefronts of 128 x 64) where they fill the CUs, 128 x 128 (four of 64 x
// 64) below that, with four stages of 64 k where it has a CU to itself and two
// where two share one.  A load of a 64-k stage takes eight whole 128-byte pieces
// of rows; those of 32 k are twice as many, and where rows do not begin on a
// 128-byte line they touch up to two lines each (198 tokens, 7528 x 6144, 128 x 128
// tiles: 130 us in four stages of 32 k, 95 in four of 64; 1024 tokens, 4096 x 2048:
// 37.5, 35.3).  256 x 256 tiles have room for one operand's: x or dg in two stages
// of 64 k, the weights in four of 32 (7168 tokens, 4104 x 2048: 255 us with both in
// 32, 223; 4096 x 2048: 197, 194; with both in two of 64 they wait for the loads:
// 304).  The gradients of the weights read both operands along their rows.
//
// The matrix cores are busy 62 to 72% of the CUs' time; the rest are waits at the
// stages' barriers, first loads and epilogues, which no other block covers, and
// rounds that do not come out even (448 tiles on 256 CUs: 1.75 as 2).  4096 x 2048
// bf16, forward 7168 tokens 190 to 200 us on different cards (1.20 to 1.27 PFLOP/s;
// 4104 x 2048: 225); 16384 tokens with pre 452 to 463 us (1.19 to 1.22), dx 433 to
// 455 (1.21 to 1.27), dw 405 to 426 (1.29 to 1.36).  The library's bare products of
// these sizes: 193, 367, 446 and 490 us, and 1.55 PFLOP/s for 8192^3.
template <int MODE, bool BF16, class S>
__global__ __launch_bounds__(64 * S::NW, 2) void dense_kernel(DenseArgs a)
{
    if constexpr (kPairs<MODE, S>) {
        using T = TileOf<MODE, BF16, S>;
        __shared__ __align__(1024) uint16_t p0[T::kPHalves], p1[T::kPHalves];
        __shared__ __align__(1024) uint16_t q0[T::kQHalves], q1[T::kQHalves], q2[T::kQHalves], q3[T::kQHalves];
        dense_block<MODE, BF16, S>(a, blockIdx.x, {(LDS_AS uint16_t *)p0, (LDS_AS uint16_t *)p1,
                                                   (LDS_AS uint16_t *)q0, (LDS_AS uint16_t *)q1, (LDS_AS uint16_t *)q2,
                                                   (LDS_AS uint16_t *)q3});
    } else {
        __shared__ __align__(1024) uint16_t r0[S::kHalves], r1[S::kHalves];
        if constexpr (S::RING == 2) {
            dense_block<MODE, BF16, S>(a, blockIdx.x, {(LDS_AS uint16_t *)r0, (LDS_AS uint16_t *)r1});
        } else {
            __shared__ __align__(1024) uint16_t r2[S::kHalves], r3[S::kHalves];
            dense_block<MODE, BF16, S>(a, blockIdx.x, {(LDS_AS uint16_t *)r0, (LDS_AS uint16_t *)r1,
                                                       (LDS_AS uint16_t *)r2, (LDS_AS uint16_t *)r3});
        }
    }
}

template <int MODE, bool BF16, class S>
hipError_t launch_dense_shape(const DenseArgs &a, hipStream_t s)
{
    dense_kernel<MODE, BF16, S><<<(unsigned)(a.mt * a.nt), 64 * S::NW, 0, s>>>(a);
    return hipGetLastError();
}

template <int MODE>
hipError_t launch_dense_mode(bool bf16, const DenseArgs &a, hipStream_t s)
{
    if (a.bm == kDenseLarge)
        return bf16 ? launch_dense_shape<MODE, true, LargeTile>(a, s) : launch_dense_shape<MODE, false, LargeTile>(a, s);
    if (a.mt * a.nt <= 256)
        return bf16 ? launch_dense_shape<MODE, true, AloneTile>(a, s) : launch_dense_shape<MODE, false, AloneTile>(a, s);
    return bf16 ? launch_dense_shape<MODE, true, SmallTile>(a, s) : launch_dense_shape<MODE, false, SmallTile>(a, s);
}

}  // namespace moe
