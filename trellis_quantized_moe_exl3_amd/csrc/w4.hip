// Products with 4-bit weights and group scales, dense or by expert.
//
//   y[r][n] = sum_g s[n][g] sum_{k in g} x[r][k] (q[n][k] - z[n][g])
//
// on v_mfma_f32_16x16x32 with the rows of x as its row operand and sixteen
// columns n beside them: lane l holds the code dword of column l % 16, k = 8 (l
// / 16) + 0..7 of 32 k.  A code becomes the 16-bit number 16 + q by shift and
// bits alone (one exponent, q in the leading mantissa bits; exact), two to an
// instruction, and a second product of the same rows with ones gives sum x, so
// that with fp32 sums per group
//   acc += s (sum x (16 + q) - (16 + z) sum x).
// The weights themselves are never rounded.  The price of the 16 is two to three
// of the sums' 24 bits.
#include "dense_kernel.h"
#include "w4.h"

namespace moe {

// Eight codes -> eight 16-bit numbers 16 + q, in the order of permute8().
// sixteen: sixteen<BF16>(), in a register.
template <bool BF16>
MOE_DEV u32x4 expand8(uint32_t c, uint32_t sixteen)
{
    if constexpr (BF16)   // steps of 1 at bit 3
        return (u32x4){((c << 3) & 0x00780078u) | sixteen, ((c >> 1) & 0x00780078u) | sixteen,
                       ((c >> 5) & 0x00780078u) | sixteen, ((c >> 9) & 0x00780078u) | sixteen};
    else                  // at bit 6
        return (u32x4){((c << 6) & 0x03C003C0u) | sixteen, ((c << 2) & 0x03C003C0u) | sixteen,
                       ((c >> 2) & 0x03C003C0u) | sixteen, ((c >> 6) & 0x03C003C0u) | sixteen};
}

// 16 twice.  Hidden from the compiler in a vector register: with both constants
// known it takes an instruction each for and and or, as one may hold one of them.
template <bool BF16>
MOE_DEV uint32_t sixteen()
{
    uint32_t v = BF16 ? 0x41804180u : 0x4C004C00u;
    asm("" : "+v"(v));
    return v;
}

// k 0..7 -> 0 4 1 5 2 6 3 7: what the two halves of a code dword give in turn.
MOE_DEV u32x4 permute8(u32x4 x)
{
    return (u32x4){__builtin_amdgcn_perm(x[2], x[0], 0x05040100u), __builtin_amdgcn_perm(x[2], x[0], 0x07060302u),
                   __builtin_amdgcn_perm(x[3], x[1], 0x05040100u), __builtin_amdgcn_perm(x[3], x[1], 0x07060302u)};
}

// The tile number `c` of a launch: its expert and rows (n = 0: past the last one).
// Every thread of the block calls it.
struct W4Tile {
    int e, row, n;
};

// Rows of expert e, clamped into the call's.
MOE_DEV void w4_rows(const W4Args &a, int e, int &lo, int &hi)
{
    lo = hi = 0;
    if (e < a.E) {
        lo = min(max(a.offsets[e], 0), a.R);
        hi = min(max(a.offsets[e + 1], lo), a.R);
    }
}

template <int NW>
MOE_DEV W4Tile w4_tile(const W4Args &a, int c, int tile_rows)
{
    if (a.list) {
        // (an entry past the last one may be read: the list has room for one)
        const int4 t = a.list[min(c, a.most)];
        const int n = __builtin_amdgcn_readfirstlane(*a.count);
        return {__builtin_amdgcn_readfirstlane(t.x), __builtin_amdgcn_readfirstlane(t.y),
                c < n ? __builtin_amdgcn_readfirstlane(t.z) : 0};
    }
    if (!a.offsets) {
        const int row = c * tile_rows;
        return {0, row, row < a.R ? min(tile_rows, a.R - row) : 0};
    }
    __shared__ int found[3], wsum[NW];
    const int tid = threadIdx.x, w = tid >> 6, l = tid & 63;
    if (tid == 0)
        found[2] = 0;
    int before = 0;
    for (int e0 = 0; e0 < a.E; e0 += 64 * NW) {
        __syncthreads();
        const int e = e0 + tid;
        int lo, hi;
        w4_rows(a, e, lo, hi);
        const int tiles = (hi - lo + tile_rows - 1) / tile_rows;
        int v = tiles;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int o = __shfl_up(v, d, 64);
            v += l >= d ? o : 0;
        }
        if (l == 63)
            wsum[w] = v;
        __syncthreads();
        int first = before + v - tiles;
        for (int i = 0; i < NW; ++i) {
            first += i < w ? wsum[i] : 0;
            before += wsum[i];
        }
        if (c >= first && c < first + tiles) {
            found[0] = e;
            found[1] = lo + (c - first) * tile_rows;
            found[2] = min(tile_rows, hi - found[1]);
        }
    }
    __syncthreads();
    return {__builtin_amdgcn_readfirstlane(found[0]), __builtin_amdgcn_readfirstlane(found[1]),
            __builtin_amdgcn_readfirstlane(found[2])};
}

// Offsets that are not ascending within the rows.
MOE_DEV void w4_status(const W4Args &a)
{   // (every thread of a block)
    __shared__ int bad;
    if (threadIdx.x == 0)
        bad = 0;
    __syncthreads();
    if (a.offsets)
        for (int e = threadIdx.x; e <= a.E; e += blockDim.x) {
            const int o = a.offsets[e];
            if (o < 0 || o > a.R || (e > 0 && o < a.offsets[e - 1]))
                bad = 1;
        }
    __syncthreads();
    if (threadIdx.x == 0)
        *a.status = bad ? MOE_EXL3_STATUS_BAD_INDEX : 0;
}

// The tiles of a call's two launches, each an expert, its first row and their
// number, from the offsets, in one block.  Experts of more than `limit` rows make up
// the second list if their tiles take the first variant half as long again as the
// second at least.  Bound by latency (two reads of the offsets, four barriers).
__global__ __launch_bounds__(1024) void w4_list_kernel(W4Args a, W4Lists lists)
{
    __shared__ int first[2][1024], last[1024];   // of an expert's tiles in either list; its last row
    __shared__ int wsum[2][16], crowd[2][16];
    const int e = threadIdx.x, w = e >> 6, l = e & 63;
    w4_status(a);
    int lo, hi;
    w4_rows(a, e, lo, hi);
    const int rows = hi - lo;
    const bool many = rows > lists.limit;
    int t[2], v[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        t[i] = (rows + lists.rows[i] - 1) / lists.rows[i];
        v[i] = many ? t[i] : 0;
#pragma unroll
        for (int d = 32; d > 0; d >>= 1)
            v[i] += __shfl_xor(v[i], d, 64);
        if (l == 0)
            crowd[i][w] = v[i];
    }
    __syncthreads();
    v[0] = v[1] = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        v[0] += crowd[0][i];
        v[1] += crowd[1][i];
    }
    const bool two = (float)v[0] * lists.us[0] > 1.5f * fmaxf((float)v[1] * lists.us[1], lists.least_us);
    t[0] = two && many ? 0 : t[0];
    t[1] = two && many ? t[1] : 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        v[i] = t[i];
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int o = __shfl_up(v[i], d, 64);
            v[i] += l >= d ? o : 0;
        }
        if (l == 63)
            wsum[i][w] = v[i];
    }
    __syncthreads();
    int total[2] = {};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        int before = v[i] - t[i];
#pragma unroll
        for (int s = 0; s < 16; ++s) {
            before += s < w ? wsum[i][s] : 0;
            total[i] += wsum[i][s];
        }
        // (offsets that descend may make more tiles than the rows have)
        total[i] = min(total[i], lists.most[i]);
        first[i][e] = before;
        if (e == 0)
            *lists.count[i] = total[i];
    }
    last[e] = hi;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i)
        for (int c = e; c < total[i]; c += 1024) {
            // the last expert whose tiles begin at c or before (those without tiles
            // begin where the next one's do)
            int at = 0;
#pragma unroll
            for (int step = 512; step > 0; step >>= 1)
                if (first[i][at + step] <= c)
                    at += step;
            const int row = min(max(a.offsets[at], 0), a.R) + (c - first[i][at]) * lists.rows[i];
            lists.list[i][c] = make_int4(at, row, min(lists.rows[i], last[at] - row), 0);
        }
}

// ---- tiles of few rows, k cut over the wavefronts of a block
//
// A wavefront takes the k in shares of 256 (a 128-byte line of each code row) in
// turn and streams its own codes and rows of x through its own slots in LDS, with
// no barrier until the block's sums meet.  16-byte loads straight to LDS, eight lanes
// a line: in registers, with a row for every lane, each lane would be a
// memory transaction.
//   codes  NJ x 16 rows (columns n) of 128 bytes, two slots.  Piece p of 16 bytes
//          (32 k) of row r lies in place p ^ (r / 2 % 8): the 64 lanes that read a
//          dword each (16 rows, one piece) hit 64 banks
//   x      ROWS rows of XK = 256 / XS k, two slots.  Piece p (8 k) of row r lies in
//          place p ^ swizzle(r)
//   scales, zeros   one element a lane in registers, a share ahead; a lane takes
//          its column's from the lane that has it
// Where the rows are few the codes bound it: 64 rows at 58 experts' pairs of 4096 x
// 2048 take 103 us, 502 MB at 4.9 TB/s (a 1 GiB copy reaches 5.1).  A small matrix
// ends before its stream is at full rate (1 row, 2048 x 4096: 4.0 us, of which 2.2 are
// those of an empty launch), and 32 rows a tile are bound by what a tile costs
// alone: its start, the loads of its share of k in turn (of 32 rows a slot of x holds
// 64 k, so the 512 k of a wavefront are eight of them, two in flight), the meeting
// (64 rows, 4096 x 4096: 9.3 us).
template <bool BF16, int GLOG, int ROWS, int NJ, bool GLU>
struct W4Stream {
    static constexpr int MR = (ROWS + 15) / 16;                  // blocks of 16 rows
    static constexpr int XS = ROWS <= 4 ? 1 : ROWS <= 16 ? 2 : 4; // x slots of a share
    static constexpr int XK = 256 / XS;
    static constexpr int kPieces = XK / 8;                       // of a row of x
    static constexpr int kXLoads = ROWS * XK / 512, kCLoads = 2 * NJ;
    static constexpr int kXHalves = ROWS * XK, kCHalves = NJ * 1024;   // of a slot
    static constexpr int kCols = 16 * (GLU ? NJ / 2 : NJ);      // columns of a tile
    static constexpr int kSteps = 8 / XS;                        // of 32 k, a slot of x
    static constexpr int GS = 256 >> GLOG;                       // groups of a share
    static constexpr int kGroupSteps = 8 / GS;
    static constexpr int kScales = GS == 2 ? (NJ + 1) / 2 : NJ * GS / 4;
    static_assert(kXLoads * 512 == kXHalves, "whole loads");

    __amdgpu_buffer_rsrc_t x, c[2];
    uint32_t xoff[kXLoads], coff[kCLoads];
    const uint16_t *sp[kScales];
    const uint8_t *zp[kScales];
    int scol[kScales];
    int l, K, G, N;
    uint32_t base16;
    uint16_t snext[kScales];
    uint8_t znext[kScales];
    uint32_t now[kScales], zmask[kScales];   // scale | zero << 16
    uint32_t xat, cat;   // byte addresses in the slots of the lane's fragments of step 0
    f32x4 acc[MR][NJ], tmp[MR][NJ], sum[MR];

    MOE_DEV static int swizzle(int r) { return XS == 1 ? (r & 3) << 2 : XS == 2 ? r & 15 : (r >> 1) & 7; }

    MOE_DEV void init(const W4Args &a, const W4Tile &t, int n0, int lane)
    {
        l = lane;
        K = a.K;
        G = K >> GLOG;
        N = a.N;
        const int r = ROWS < 16 ? l & (ROWS - 1) : l & 15;
        xat = (uint32_t)(r * 2 * XK + 16 * ((l >> 4) ^ swizzle(r)));
        cat = (uint32_t)((l & 15) * 128 + 16 * ((l & 15) >> 1) + 4 * (l >> 4));
        const int64_t matrix = (int64_t)t.e * a.N;
        x = buf_rsrc(a.x + (int64_t)t.row * a.ldx, (uint32_t)(((t.n - 1) * a.ldx + K) * 2));
#pragma unroll
        for (int i = 0; i < (GLU ? 2 : 1); ++i)
            c[i] = buf_rsrc(a.codes[i] + matrix * (K / 2), (uint32_t)a.N * (uint32_t)(K / 2));
#pragma unroll
        for (int i = 0; i < kXLoads; ++i) {
            const int s = 64 * i + l, r = s / kPieces, k = 8 * ((s % kPieces) ^ swizzle(r));
            xoff[i] = r < t.n ? (uint32_t)((r * a.ldx + k) * 2) : kOutOfRange;
        }
#pragma unroll
        for (int i = 0; i < kCLoads; ++i) {
            const int r = 8 * i + (l >> 3), p = (l & 7) ^ ((r >> 1) & 7);
            coff[i] = (uint32_t)column(n0, r) * (uint32_t)(K / 2) + 16 * p;
        }
        base16 = sixteen<BF16>();
#pragma unroll
        for (int i = 0; i < kScales; ++i) {
            const int r = min(GS == 2 ? 32 * i + (l >> 1) : 16 * (i / (GS / 4)) + (l >> 2), 16 * NJ - 1);
            const int m = GLU && r >= 8 * NJ;
            const int64_t row = matrix * G;
            scol[i] = column(n0, r);
            sp[i] = (m ? a.scales[1] : a.scales[0]) + row;
            const uint8_t *z = m ? a.zeros[1] : a.zeros[0];
            zmask[i] = z ? 0xFF0000u : 0u;
            // (without zeros some bytes of the scales are read and masked off)
            zp[i] = (z ? z : (const uint8_t *)(m ? a.scales[1] : a.scales[0])) + row;
        }
    }
    // Column of the matrix that row r of the codes' tile is.
    MOE_DEV static int column(int n0, int r) { return n0 + (GLU ? r % (8 * NJ) : r); }

    // What a wavefront's share is: its first k (K: none) and its tile of columns.
    struct Pos {
        int k, tile;
    };

    MOE_DEV void load_x(int k0, LDS_AS uint16_t *lds)
    {
#pragma unroll
        for (int i = 0; i < kXLoads; ++i) {
            const int s = 64 * i + l, k = k0 + 8 * ((s % kPieces) ^ swizzle(s / kPieces));
            __builtin_amdgcn_raw_ptr_buffer_load_lds(x, (LDS_AS void *)(lds + 512 * i), 16,
                                                     k < K ? xoff[i] + 2 * (uint32_t)k0 : kOutOfRange, 0, 0, 0);
        }
    }
    MOE_DEV void load_codes(const Pos &at, LDS_AS uint16_t *lds)
    {
        const uint32_t o = (uint32_t)(at.tile * kCols) * (uint32_t)(K / 2) + (uint32_t)(at.k / 2);
#pragma unroll
        for (int i = 0; i < kCLoads; ++i) {
            const int r = 8 * i + (l >> 3), k = at.k + 32 * ((l & 7) ^ ((r >> 1) & 7));
            __builtin_amdgcn_raw_ptr_buffer_load_lds(c[GLU && i >= NJ], (LDS_AS void *)(lds + 512 * i), 16,
                                                     k < K ? coff[i] + o : kOutOfRange, 0, 0, 0);
        }
    }
    // (Groups past the last one read it again: their x and codes are zeros.)
    MOE_DEV void load_scales(const Pos &at)
    {
#pragma unroll
        for (int i = 0; i < kScales; ++i) {
            const int g = min((at.k >> GLOG) + (GS == 2 ? l & 1 : (l & 3) + 4 * (i % (GS / 4))), G - 1);
            const uint32_t o = (uint32_t)min(scol[i] + at.tile * kCols, N - 1) * (uint32_t)G + (uint32_t)g;
            snext[i] = sp[i][o];
            znext[i] = zp[i][o];
        }
    }
    // The k of a slot of x, number j of its share.
    MOE_DEV void slot(int j, const u32x4 (&xf)[kSteps][MR], const uint32_t (&cf)[kSteps][NJ])
    {
        const uint32_t one = BF16 ? 0x3F803F80u : 0x3C003C00u;
        const u32x4 ones = {one, one, one, one};
#pragma unroll
        for (int h = 0; h < kSteps; ++h) {
            const int step = kSteps * j + h;
            const bool first = step % kGroupSteps == 0;
            u32x4 xp[MR];
#pragma unroll
            for (int i = 0; i < MR; ++i) {
                xp[i] = permute8(xf[h][i]);
                sum[i] = dense_mfma<BF16>(xp[i], ones, first ? (f32x4){} : sum[i]);
            }
#pragma unroll
            for (int q = 0; q < NJ; ++q) {
                const u32x4 w = expand8<BF16>(cf[h][q], base16);
#pragma unroll
                for (int i = 0; i < MR; ++i)
                    tmp[i][q] = dense_mfma<BF16>(xp[i], w, first ? (f32x4){} : tmp[i][q]);
            }
            if (step % kGroupSteps != kGroupSteps - 1)
                continue;
            const int g = step / kGroupSteps;
#pragma unroll
            for (int q = 0; q < NJ; ++q) {
                const int from = GS == 2 ? (16 * (q & 1) + (l & 15)) * 2 + g : (l & 15) * 4 + (g & 3);
                const uint32_t v = __builtin_amdgcn_ds_bpermute(4 * from, now[GS == 2 ? q >> 1 : q * (GS / 4) + (g >> 2)]);
                const float s = act_to_f32<BF16>((uint16_t)v), z = 16.0f + (float)(v >> 16);
#pragma unroll
                for (int i = 0; i < MR; ++i)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        acc[i][q][r] = fmaf(s, fmaf(-z, sum[i][r], tmp[i][q][r]), acc[i][q][r]);
            }
            // here, not after the share: the compiler would hold every group's sums
            // until then
#pragma unroll
            for (int q = 0; q < NJ; ++q)
#pragma unroll
                for (int i = 0; i < MR; ++i)
                    asm volatile("" : "+v"(acc[i][q]));
        }
    }
    // Slot J of the share at[0]; what is loaded next: the slot of x two on, after the
    // last one the codes of the share two on, before the first the scales of the
    // next.  (The loads that may stay in flight are the slot and the codes issued
    // after the ones needed here.)
    template <int J>
    MOE_DEV void run_slot(const Pos (&at)[3], LDS_AS uint16_t *xs, LDS_AS uint16_t *cs)
    {
        __builtin_amdgcn_sched_barrier(0);
        wait_vmcnt<kXLoads + (J == 0 ? kCLoads : 0)>();
        u32x4 xf[kSteps][MR];
        uint32_t cf[kSteps][NJ];
#pragma unroll
        for (int h = 0; h < kSteps; ++h) {
#pragma unroll
            for (int i = 0; i < MR; ++i)
                xf[h][i] = *(const LDS_AS u32x4 *)((const LDS_AS char *)xs + (xat ^ (64u * h)) + 32 * XK * i);
#pragma unroll
            for (int q = 0; q < NJ; ++q)
                cf[h][q] = *(const LDS_AS uint32_t *)((const LDS_AS char *)cs + (cat ^ (16u * (kSteps * J + h))) + 2048 * q);
        }
        __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0): the slots are free
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (J == 0) {
#pragma unroll
            for (int i = 0; i < kScales; ++i)
                now[i] = snext[i] | (((uint32_t)znext[i] << 16) & zmask[i]) | (zmask[i] ? 0u : 8u << 16);
            load_scales(at[1]);
        }
        if constexpr (J == XS - 1)
            load_codes(at[2], cs);
        load_x(at[(J + 2) / XS].k + XK * ((J + 2) % XS), xs);
        __builtin_amdgcn_sched_barrier(0);
        slot(J, xf, cf);
    }
    MOE_DEV void share(const Pos (&at)[3], LDS_AS uint16_t *x0, LDS_AS uint16_t *x1, LDS_AS uint16_t *cs)
    {
        run_slot<0>(at, x0, cs);
        if constexpr (XS >= 2)
            run_slot<1>(at, x1, cs);
        if constexpr (XS == 4) {
            run_slot<2>(at, x0, cs);
            run_slot<3>(at, x1, cs);
        }
    }
    MOE_DEV void clear()
    {
#pragma unroll
        for (int i = 0; i < MR; ++i)
#pragma unroll
            for (int q = 0; q < NJ; ++q)
                acc[i][q] = (f32x4){};
    }
    // Of each of the block's tiles of columns the shares first, first + stride, ..;
    // the same number for every wavefront, some past the end (zeros).  `flush` takes
    // the sums of a tile while the next one's shares are on their way.
    template <class F>
    MOE_DEV void run(int first, int stride, int tiles, LDS_AS uint16_t *x0, LDS_AS uint16_t *x1, LDS_AS uint16_t *c0,
                     LDS_AS uint16_t *c1, F flush)
    {
        const int per = (K + 256 * stride - 1) / (256 * stride);
        auto after = [&](const Pos &p) {
            Pos n = {p.k + 256 * stride, p.tile};
            if (n.k >= 256 * stride * per)
                n = {256 * first, p.tile + 1};
            if (n.tile >= tiles)
                n.k = K;   // (and no further: its columns may not exist)
            return n;
        };
        Pos at[3] = {{256 * first, 0}, {}, {}};
        at[1] = after(at[0]);
        at[2] = after(at[1]);
        load_scales(at[0]);
        load_codes(at[0], c0);
        load_x(at[0].k, x0);
        load_codes(at[1], c1);
        load_x(XS == 1 ? at[1].k : at[0].k + XK, x1);
        clear();
        int left = per;
        auto done = [&] {   // of a share: the next one, and whether there is one
            if (--left == 0) {
                flush(at[0].tile);
                left = per;
                clear();
                if (at[0].tile + 1 >= tiles)
                    return true;
            }
            at[0] = at[1];
            at[1] = at[2];
            at[2] = after(at[2]);
            return false;
        };
        for (;;) {
            share(at, x0, x1, c0);
            if (done())
                break;
            if constexpr (XS == 1)
                share(at, x1, x0, c1);
            else
                share(at, x0, x1, c1);
            if (done())
                break;
        }
        wait_vmcnt<0>();   // the loads past the end still write LDS
    }
};

template <bool BF16, bool GLU>
MOE_DEV void w4_store(const W4Args &a, int64_t row, int n, float g, float u)
{
    float y = g;
    if constexpr (GLU)
        y = (a.act == MOE_EXL3_ACT_SILU ? act_value<MOE_EXL3_ACT_SILU>(g) : act_value<MOE_EXL3_ACT_GELU_TANH>(g)) * u;
    if (a.base)
        y += act_to_f32<BF16>(a.base[row * a.ldbase + n]);
    a.y[row * a.ldy + n] = BF16 ? f32_to_bf16_bits(y) : f32_to_f16_bits(y);
}

// A block takes `a.tiles` tiles of columns in turn, so that its start (the
// offsets, the first loads) is paid once for them.  Its wavefronts' sums meet in LDS
// in their order, so that the same rows give the same bits.
template <bool BF16, bool GLU, int GLOG, int ROWS, int NJ, int NW>
__global__ __launch_bounds__(64 * NW, ROWS <= 4 && NW == 4 ? 3 : 2) void w4_split_kernel(W4Args a)
{
    using S = W4Stream<BF16, GLOG, ROWS, NJ, GLU>;
    constexpr bool kApart = ROWS <= 16;          // the sums have LDS of their own
    constexpr int kLanes = ROWS <= 4 ? 16 : 64;  // that hold rows of the tile
    constexpr int kBlocks = S::MR * NJ;
    __shared__ __align__(1024) uint16_t x0[NW * S::kXHalves], x1[NW * S::kXHalves], c0[NW * S::kCHalves],
        c1[NW * S::kCHalves];
    __shared__ f32x4 own[kApart ? NW * kBlocks * kLanes : 1];
    static_assert(kApart || kBlocks * 1024 <= S::kXHalves * 2, "sums fit a slot of x");
    const int tid = threadIdx.x, l = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    if (blockIdx.x == 0 && !a.list)
        w4_status(a);
    const int nt = (a.N + S::kCols * a.tiles - 1) / (S::kCols * a.tiles);
    const int n0 = (int)(blockIdx.x % nt) * S::kCols * a.tiles;
    const W4Tile t = w4_tile<NW>(a, blockIdx.x / nt, ROWS);
    if (t.n <= 0)
        return;
    S st;
    st.init(a, t, n0, l);
    LDS_AS uint16_t *mine = (LDS_AS uint16_t *)x0 + w * S::kXHalves;
    constexpr int kStep = kApart ? kBlocks * kLanes : S::kXHalves / 8;   // between the wavefronts' sums
    LDS_AS f32x4 *red = kApart ? (LDS_AS f32x4 *)own : (LDS_AS f32x4 *)((LDS_AS uint16_t *)x0);
    auto meet = [] {
        __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0)
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
    };
    auto flush = [&](int tile) {
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (!kApart)
            wait_vmcnt<0>();   // (one tile only: the loads past the end)
        else if (tile > 0)
            meet();   // the last tile's sums are read
        if (l < kLanes)
#pragma unroll
            for (int i = 0; i < kBlocks; ++i)
                red[w * kStep + kLanes * i + l] = st.acc[i / NJ][i % NJ];
        meet();
        constexpr int kAcross = GLU ? NJ / 2 : NJ, kUnits = S::MR * kAcross;   // of 64 x 4 results
        for (int u = w; u < kUnits; u += NW) {
            const int i = u / kAcross, q = u % kAcross;
            auto total = [&](int q) {
                f32x4 v = red[kLanes * (i * NJ + q) + (l & (kLanes - 1))];
#pragma unroll
                for (int s = 1; s < NW; ++s)
                    v += red[s * kStep + kLanes * (i * NJ + q) + (l & (kLanes - 1))];
                return v;
            };
            const f32x4 g = total(q), up = GLU ? total(q + NJ / 2) : g;
            const int n = n0 + S::kCols * tile + 16 * q + (l & 15);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int m = 16 * i + 4 * (l >> 4) + r;
                if (m < t.n && n < a.N)
                    w4_store<BF16, GLU>(a, t.row + m, n, g[r], up[r]);
            }
        }
    };
    st.run(w, NW, a.tiles, mine, (LDS_AS uint16_t *)x1 + w * S::kXHalves, (LDS_AS uint16_t *)c0 + w * S::kCHalves,
           (LDS_AS uint16_t *)c1 + w * S::kCHalves, flush);
}

// ---- tiles of many rows, columns over the wavefronts of a block
//
// 128 rows and 256 columns (a gated pair: 128 of each) by 2 x 4 wavefronts of 64 x
// 64, or 64 rows and 128 columns by 1 x 4 of 64 x 32.  x and the codes pass through LDS in stages of 128 k, which all
// wavefronts load and share; a ring of three, one barrier a stage.
//   x      rows of 256 bytes, piece p (8 k) of row r in place p ^ (r % 16)
//   codes  rows of 64 bytes, piece p (32 k) of row r in place p ^ (r / 4 % 4)
// While a stage is multiplied each wavefront prepares the 16 rows of x of the next
// that it has loaded itself: it writes them back in the order of expand8() and
// leaves their groups' sums beside them, once instead of once for each
// wavefront that reads them.  Without zeros all columns subtract the same (16 +
// 8) sum x, which then is what a group's products start from.
// A SIMD issues a product in 8 clocks and another vector instruction in 4.  Four go
// with a product: two make the codes 16-bit numbers, one applies the group's scale,
// and about one is for addresses, the scales and the preparation.  So 24 clocks of
// issue stand against 16 of the matrix unit: 220 us of 16384 rows at 32 experts of 2048 x
// 4096, which take 354 (777 TFLOP/s; tiles that are not full add 12%) with the matrix
// cores busy 40%.  The rest are waits: eight wavefronts in step, one block a CU, at
// a barrier a stage, and a tile's start and end.  One matrix 4096 x 4096, 4096 rows:
// 144 to 148 us (929 to 954 TFLOP/s).
template <bool BF16, int GLOG, bool GLU, bool ZEROS, int NW, int NJ>
struct W4Wide {
    static constexpr int kRows = 16 * NW, kCols = 64 * NJ, kStage = 128, MR = 4;
    static constexpr int kOwn = 16 * NJ;   // code rows of a wavefront
    static constexpr int kXLoads = kRows * kStage * 2 / 1024 / NW, kCLoads = kCols * kStage / 2 / 1024 / NW;
    static constexpr int kXHalves = kRows * kStage, kCHalves = kCols * kStage / 4;   // of a stage
    static constexpr int GS = kStage >> GLOG, kGroupSteps = 4 / GS;
    static constexpr int kSums = GS * kRows;   // of a stage
    static constexpr int kScales = (kOwn * GS + 63) / 64;
    static_assert(kXLoads * 4 * NW == kRows, "a wavefront prepares the rows it loads");
    static_assert(kCLoads * 16 * NW == kCols, "whole loads");

    __amdgpu_buffer_rsrc_t x, c[2];
    uint32_t xoff[kXLoads], coff[kCLoads];
    const uint16_t *sp[kScales];
    const uint8_t *zp[kScales];
    uint32_t zmask;
    int l, w, K, G;
    uint32_t base16;
    uint16_t snext[kScales];
    uint8_t znext[kScales];
    uint32_t now[kScales];   // scale | zero << 16
    f32x4 acc[MR][NJ], tmp[MR][NJ];

    // Column of the matrix that row r of the codes' tile is: of a wavefront's, half
    // are (GLU) the gate's and half the same columns of the other.
    MOE_DEV static int column(int n0, int r) { return n0 + (GLU ? r / kOwn * (kOwn / 2) + r % (kOwn / 2) : r); }
    MOE_DEV static bool second(int r) { return GLU && r % kOwn >= kOwn / 2; }

    MOE_DEV void init(const W4Args &a, const W4Tile &t, int n0, int lane, int wave)
    {
        l = lane;
        w = wave;
        K = a.K;
        G = K >> GLOG;
        base16 = sixteen<BF16>();
        xat = xaddr(16 * MR * (w >> 2));
        pat = xaddr(16 * w);
        cat = (uint32_t)((kOwn * (w & 3) + (l & 15)) * 64 + 16 * ((l >> 2) & 3) + 4 * (l >> 4));
        const int64_t matrix = (int64_t)t.e * a.N;
        x = buf_rsrc(a.x + (int64_t)t.row * a.ldx, (uint32_t)(((t.n - 1) * a.ldx + K) * 2));
#pragma unroll
        for (int i = 0; i < (GLU ? 2 : 1); ++i)
            c[i] = buf_rsrc(a.codes[i] + matrix * (K / 2), (uint32_t)a.N * (uint32_t)(K / 2));
#pragma unroll
        for (int i = 0; i < kXLoads; ++i) {
            const int r = xrow(i);
            xoff[i] = r < t.n ? (uint32_t)((r * a.ldx + xk(i)) * 2) : kOutOfRange;
        }
#pragma unroll
        for (int i = 0; i < kCLoads; ++i)
            coff[i] = (uint32_t)column(n0, crow(i)) * (uint32_t)(K / 2) + (uint32_t)ck(i) / 2;
        zmask = 0;
#pragma unroll
        for (int i = 0; i < kScales; ++i) {
            const int r = kOwn * (w & 3) + min((64 * i + l) / GS, kOwn - 1);
            const bool up = second(r);
            const int64_t row = (matrix + min(column(n0, r), a.N - 1)) * G;
            sp[i] = (up ? a.scales[1] : a.scales[0]) + row;
            const uint8_t *z = up ? a.zeros[1] : a.zeros[0];
            // (one of a pair may have none: some bytes of the scales are read and masked off)
            zp[i] = (z ? z : (const uint8_t *)(up ? a.scales[1] : a.scales[0])) + row;
            zmask |= z ? 1u << i : 0u;
        }
    }
    // Row and first k of the 16 bytes of x, of codes, that lane l's load i holds.
    MOE_DEV int xrow(int i) const { return 4 * (w * kXLoads + i) + (l >> 4); }
    MOE_DEV int xk(int i) const { return 8 * ((l & 15) ^ (xrow(i) & 15)); }
    MOE_DEV int crow(int i) const { return 16 * (w * kCLoads + i) + (l >> 2); }
    MOE_DEV int ck(int i) const { return 32 * ((l & 3) ^ ((crow(i) >> 2) & 3)); }

    // (Past K lies the next row, or nothing, which reads as zeros: no step takes it.)
    MOE_DEV void load(int k0, LDS_AS uint16_t *xs, LDS_AS uint16_t *cs)
    {
#pragma unroll
        for (int i = 0; i < kXLoads; ++i)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(x, (LDS_AS void *)(xs + 512 * (w * kXLoads + i)), 16,
                                                     xoff[i] + 2 * (uint32_t)k0, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < kCLoads; ++i) {
            // (16 rows a load: of one matrix)
            const bool up = second(16 * (w * kCLoads + i));
            __builtin_amdgcn_raw_ptr_buffer_load_lds(up ? c[1] : c[0], (LDS_AS void *)(cs + 512 * (w * kCLoads + i)), 16,
                                                     coff[i] + (uint32_t)(k0 / 2), 0, 0, 0);
        }
    }
    // (Groups past the last one read it again.)
    MOE_DEV void load_scales(int k0)
    {
#pragma unroll
        for (int i = 0; i < kScales; ++i) {
            const int g = min((k0 >> GLOG) + l % GS, G - 1);
            snext[i] = sp[i][g];
            if constexpr (ZEROS)
                znext[i] = zp[i][g];
        }
    }
    // Byte addresses in a stage's slots of the lane's fragments of step 0: of the
    // rows this wavefront multiplies, of those it prepares, of its codes.
    uint32_t xat, pat, cat;
    MOE_DEV uint32_t xaddr(int r0) const { return (uint32_t)((r0 + (l & 15)) * 256 + 16 * ((l >> 4) ^ (l & 15))); }

    // The preparation of this wavefront's rows of x, in three parts.
    u32x4 raw[4];
    MOE_DEV void prepare_read(const LDS_AS uint16_t *xs)
    {
#pragma unroll
        for (int h = 0; h < 4; ++h)
            raw[h] = *(const LDS_AS u32x4 *)((const LDS_AS char *)xs + (pat ^ (64u * h)));
    }
    MOE_DEV void prepare_write(LDS_AS uint16_t *xs)
    {
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            raw[h] = permute8(raw[h]);
            *(LDS_AS u32x4 *)((LDS_AS char *)xs + (pat ^ (64u * h))) = raw[h];
        }
    }
    MOE_DEV void prepare_sums(LDS_AS float *sums)
    {
        // 1, or -24 twice
        const uint32_t one = ZEROS ? (BF16 ? 0x3F803F80u : 0x3C003C00u) : (BF16 ? 0xC1C0C1C0u : 0xCE00CE00u);
        const u32x4 ones = {one, one, one, one};
        f32x4 sum[GS];
#pragma unroll
        for (int h = 0; h < 4; ++h)
            sum[h / kGroupSteps] =
                dense_mfma<BF16>(raw[h], ones, h % kGroupSteps == 0 ? (f32x4){} : sum[h / kGroupSteps]);
        if ((l & 15) == 0)   // (all 16 columns of the product are the same)
#pragma unroll
            for (int g = 0; g < GS; ++g)
                *(LDS_AS f32x4 *)(sums + kRows * g + 16 * w + 4 * (l >> 4)) = sum[g];
    }
    // Fragments of step h of a stage, read while the step before is multiplied.
    u32x4 xn[MR];
    uint32_t cn[NJ];
    f32x4 sn[MR];
    MOE_DEV void read(int h, const LDS_AS uint16_t *xs, const LDS_AS uint16_t *cs, const LDS_AS float *sums)
    {
        if (!ZEROS && h % kGroupSteps == 0)   // (with zeros: where they are needed)
#pragma unroll
            for (int i = 0; i < MR; ++i)
                sn[i] = *(const LDS_AS f32x4 *)(sums + kRows * (h / kGroupSteps) + 64 * (w >> 2) + 16 * i + 4 * (l >> 4));
#pragma unroll
        for (int i = 0; i < MR; ++i)
            xn[i] = *(const LDS_AS u32x4 *)((const LDS_AS char *)xs + (xat ^ (64u * h)) + 4096 * i);
#pragma unroll
        for (int q = 0; q < NJ; ++q)
            cn[q] = *(const LDS_AS uint32_t *)((const LDS_AS char *)cs + (cat ^ (16u * h)) + 1024 * q);
    }
    // Every wavefront has read the stage and prepared its part of the next one.
    MOE_DEV void meet()
    {
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0)
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
    }
    // The stage at k0, from its slots, and meanwhile the preparation of the next;
    // before its last step all its fragments are in registers, and the stage
    // three on is loaded in its place.
    // TAIL: one of the last three, number TAIL of them, which load nothing (the
    // loads past the end would be waited for); it may have fewer than four steps.
    // IDLE: of a wavefront without rows, which loads and prepares its part alone.
    template <int TAIL, bool IDLE>
    MOE_DEV void stage(int k0, LDS_AS uint16_t *xs, LDS_AS uint16_t *cs, const LDS_AS float *sums,
                       LDS_AS uint16_t *xnext, LDS_AS uint16_t *cnext, LDS_AS float *snext_)
    {
        f32x4 sum[MR];
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            const bool first = h % kGroupSteps == 0;
            const int g = h / kGroupSteps;
            if (TAIL && k0 + 32 * h >= K)
                break;
            // (the addresses of a step are computed for it: kept, all of them cost
            // registers that there are not, and a spill waits for all loads in
            // flight)
            asm volatile("" : "+v"(xat), "+v"(pat), "+v"(cat));
            u32x4 xp[MR];
            uint32_t cf[NJ];
            if (h == 3)
                meet();
            __builtin_amdgcn_sched_barrier(0);
            if (!IDLE && !ZEROS && first)
#pragma unroll
                for (int i = 0; i < MR; ++i)
                    sum[i] = sn[i];
            if constexpr (!IDLE) {
#pragma unroll
                for (int i = 0; i < MR; ++i)
                    xp[i] = xn[i];
#pragma unroll
                for (int q = 0; q < NJ; ++q)
                    cf[q] = cn[q];
            }
            if (h == 0) {
                wait_vmcnt<TAIL <= 1 ? kXLoads + kCLoads : 0>();   // the next stage is here, but for its preparation
                if constexpr (!IDLE) {
#pragma unroll
                    for (int i = 0; i < kScales; ++i)
                        now[i] = ZEROS ? snext[i] | ((zmask >> i) & 1u ? (uint32_t)znext[i] << 16 : 8u << 16) : snext[i];
                    load_scales(k0 + kStage);
                }
            }
            if (h == 1)
                prepare_read(xnext);
            if (h == 2)
                prepare_write(xnext);
            if (h == 3 && !TAIL)
                load(k0 + 3 * kStage, xs, cs);
            if constexpr (IDLE) {
                if (h == 2)
                    prepare_sums(snext_);
                continue;
            }
            if (h < 3)
                read(h + 1, xs, cs, sums);
            else
                read(0, xnext, cnext, snext_);
#pragma unroll
            for (int q = 0; q < NJ; ++q) {
                const u32x4 v = expand8<BF16>(cf[q], base16);
#pragma unroll
                for (int i = 0; i < MR; ++i)
                    tmp[i][q] = dense_mfma<BF16>(xp[i], v, !first ? tmp[i][q] : ZEROS ? (f32x4){} : sum[i]);
            }
            if (h == 2)
                prepare_sums(snext_);
            if (h % kGroupSteps != kGroupSteps - 1)
                continue;
            if constexpr (ZEROS)
#pragma unroll
                for (int i = 0; i < MR; ++i)
                    sum[i] = *(const LDS_AS f32x4 *)(sums + kRows * g + 64 * (w >> 2) + 16 * i + 4 * (l >> 4));
#pragma unroll
            for (int q = 0; q < NJ; ++q) {
                const int e = (16 * q + (l & 15)) * GS + g;   // (its register does not depend on the lane)
                const uint32_t v = __builtin_amdgcn_ds_bpermute(4 * (e & 63), now[16 * q * GS / 64]);
                const float s = act_to_f32<BF16>((uint16_t)v), z = 16.0f + (float)(v >> 16);
#pragma unroll
                for (int i = 0; i < MR; ++i)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        acc[i][q][r] = fmaf(s, ZEROS ? fmaf(-z, sum[i][r], tmp[i][q][r]) : tmp[i][q][r], acc[i][q][r]);
            }
#pragma unroll
            for (int q = 0; q < NJ; ++q)
#pragma unroll
                for (int i = 0; i < MR; ++i)
                    asm volatile("" : "+v"(acc[i][q]));
        }
    }
    MOE_DEV void run(bool idle, LDS_AS uint16_t *const (&xs)[3], LDS_AS uint16_t *const (&cs)[3],
                     LDS_AS float *const (&sums)[3])
    {
#pragma unroll
        for (int i = 0; i < MR; ++i)
#pragma unroll
            for (int q = 0; q < NJ; ++q)
                acc[i][q] = (f32x4){};
        load_scales(0);
        __builtin_amdgcn_sched_barrier(0);
        load(0, xs[0], cs[0]);
        load(kStage, xs[1], cs[1]);
        load(2 * kStage, xs[2], cs[2]);
        __builtin_amdgcn_sched_barrier(0);
        wait_vmcnt<2 * (kXLoads + kCLoads)>();
        prepare_read(xs[0]);
        prepare_write(xs[0]);
        prepare_sums(sums[0]);
        meet();
        if (idle) {
            stages<true>(xs, cs, sums);
        } else {
            read(0, xs[0], cs[0], sums[0]);
            stages<false>(xs, cs, sums);
        }
        wait_vmcnt<0>();   // loads past the end still write LDS
    }
    template <bool IDLE>
    MOE_DEV void stages(LDS_AS uint16_t *const (&xs)[3], LDS_AS uint16_t *const (&cs)[3], LDS_AS float *const (&sums)[3])
    {
        int k = 0;
        for (; k + 3 * kStage < K; k += 3 * kStage) {
            stage<0, IDLE>(k, xs[0], cs[0], sums[0], xs[1], cs[1], sums[1]);
            stage<0, IDLE>(k + kStage, xs[1], cs[1], sums[1], xs[2], cs[2], sums[2]);
            stage<0, IDLE>(k + 2 * kStage, xs[2], cs[2], sums[2], xs[0], cs[0], sums[0]);
        }
        stage<1, IDLE>(k, xs[0], cs[0], sums[0], xs[1], cs[1], sums[1]);
        if (k + kStage < K)
            stage<2, IDLE>(k + kStage, xs[1], cs[1], sums[1], xs[2], cs[2], sums[2]);
        if (k + 2 * kStage < K)
            stage<3, IDLE>(k + 2 * kStage, xs[2], cs[2], sums[2], xs[0], cs[0], sums[0]);
    }
};

template <bool BF16, bool GLU, int GLOG, bool ZEROS, int NW, int NJ>
__global__ __launch_bounds__(64 * NW) void w4_wide_kernel(W4Args a)
{
    using S = W4Wide<BF16, GLOG, GLU, ZEROS, NW, NJ>;
    // (slots apart for the compiler, which waits for loads into an array it reads)
    __shared__ __align__(1024) uint16_t x0[S::kXHalves], x1[S::kXHalves], x2[S::kXHalves], c0[S::kCHalves],
        c1[S::kCHalves], c2[S::kCHalves];
    __shared__ __align__(16) float s0[S::kSums], s1[S::kSums], s2[S::kSums];
    const int tid = threadIdx.x, l = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    if (blockIdx.x == 0 && !a.list)
        w4_status(a);
    constexpr int kCols = GLU ? S::kCols / 2 : S::kCols;
    const int nt = (a.N + kCols - 1) / kCols, mt = gridDim.x / nt;
    int c = blockIdx.x / nt, n = blockIdx.x % nt;
    if (mt % 8 == 0)
        xcd_map(blockIdx.x, nt, c, n);
    const W4Tile t = w4_tile<NW>(a, c, S::kRows);
    if (t.n <= 0)
        return;
    const int n0 = n * kCols;
    S st;
    st.init(a, t, n0, l, w);
    LDS_AS uint16_t *const xs[3] = {(LDS_AS uint16_t *)x0, (LDS_AS uint16_t *)x1, (LDS_AS uint16_t *)x2};
    LDS_AS uint16_t *const cs[3] = {(LDS_AS uint16_t *)c0, (LDS_AS uint16_t *)c1, (LDS_AS uint16_t *)c2};
    LDS_AS float *const sums[3] = {(LDS_AS float *)s0, (LDS_AS float *)s1, (LDS_AS float *)s2};
    // an expert's last tile may have no rows for the upper wavefronts: the lower
    // ones then have the SIMDs to themselves (16384 rows at 64 experts, 2048 x 4096:
    // 400 us with all of them multiplying, 388)
    st.run(NW == 8 && t.n <= 16 * S::MR * (w >> 2), xs, cs, sums);
    __syncthreads();
    // results through LDS, for stores of 16 bytes: a wavefront turns 16 rows at
    // a time, the 16-column block q of row r in place q ^ (r / 4 % 4)
    constexpr int kOut = GLU ? S::kOwn / 2 : S::kOwn;   // columns of a wavefront
    LDS_AS float *mine = (LDS_AS float *)(w < 4 ? xs[0] : xs[1]) + (w & 3) * 16 * 64;
    const int row0 = 16 * S::MR * (w >> 2), col0 = n0 + kOut * (w & 3);
#pragma unroll
    for (int i = 0; i < S::MR; ++i) {
        wave_lds_fence();
#pragma unroll
        for (int q = 0; q < kOut / 16; ++q)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                float v = st.acc[i][q][r];
                if constexpr (GLU)
                    v = (a.act == MOE_EXL3_ACT_SILU ? act_value<MOE_EXL3_ACT_SILU>(v)
                                                    : act_value<MOE_EXL3_ACT_GELU_TANH>(v)) *
                        st.acc[i][q + NJ / 2][r];
                const int m = 4 * (l >> 4) + r;
                mine[m * kOut + 16 * (q ^ ((l >> 4) & (kOut / 16 - 1))) + (l & 15)] = v;
            }
        wave_lds_fence();
        constexpr int kLanes = kOut / 8;   // of a row
#pragma unroll
        for (int p = 0; p < (16 * kLanes + 63) / 64; ++p) {
            const int m = (64 / kLanes) * p + l / kLanes, col = 8 * (l % kLanes);
            const LDS_AS float *at = mine + (m & 15) * kOut + 16 * ((col >> 4) ^ ((m >> 2) & (kOut / 16 - 1))) + (col & 15);
            f32x4 v[2] = {*(const LDS_AS f32x4 *)at, *(const LDS_AS f32x4 *)(at + 4)};
            const int row = row0 + 16 * i + m;
            if (m >= 16 || row >= t.n || col0 + col >= a.N)
                continue;
            if (a.base) {
                const u32x4 b = *(const u32x4 *)(a.base + (int64_t)(t.row + row) * a.ldbase + col0 + col);
#pragma unroll
                for (int d = 0; d < 4; ++d) {
                    v[d >> 1][2 * (d & 1)] += act_to_f32<BF16>((uint16_t)b[d]);
                    v[d >> 1][2 * (d & 1) + 1] += act_to_f32<BF16>((uint16_t)(b[d] >> 16));
                }
            }
            *(u32x4 *)(a.y + (int64_t)(t.row + row) * a.ldy + col0 + col) = pack8<BF16>(v[0], v[1]);
        }
    }
}

template <bool BF16, bool GLU, int GLOG, int ROWS, int NJ>
void launch_split(const W4Launch &p, W4Args a, hipStream_t s)
{
    a.tiles = p.tiles;
    if (p.waves == 8)
        w4_split_kernel<BF16, GLU, GLOG, ROWS, NJ, 8><<<p.grid, 512, 0, s>>>(a);
    else
        w4_split_kernel<BF16, GLU, GLOG, ROWS, NJ, 4><<<p.grid, 256, 0, s>>>(a);
}

template <bool BF16, bool GLU, int GLOG, int NW, int NJ>
void launch_wide(const W4Launch &p, const W4Args &a, hipStream_t s)
{
    if (a.zeros[0] || a.zeros[1])
        w4_wide_kernel<BF16, GLU, GLOG, true, NW, NJ><<<p.grid, 64 * NW, 0, s>>>(a);
    else
        w4_wide_kernel<BF16, GLU, GLOG, false, NW, NJ><<<p.grid, 64 * NW, 0, s>>>(a);
}

template <bool BF16, bool GLU, int GLOG>
void launch_variant(const W4Launch &p, const W4Args &a, hipStream_t s)
{
    constexpr int kOne = GLU ? 2 : 1;   // 16-column blocks of the narrow tiles
    switch (p.v) {
    case W4_4x16: return launch_split<BF16, GLU, GLOG, 4, kOne>(p, a, s);
    case W4_4x32: return launch_split<BF16, GLU, GLOG, 4, 2>(p, a, s);
    case W4_16x16: return launch_split<BF16, GLU, GLOG, 16, kOne>(p, a, s);
    case W4_16x32: return launch_split<BF16, GLU, GLOG, 16, 2>(p, a, s);
    case W4_32x32: return launch_split<BF16, GLU, GLOG, 32, 2>(p, a, s);
    case W4_64x128: return launch_wide<BF16, GLU, GLOG, 4, 2>(p, a, s);
    case W4_128x256: return launch_wide<BF16, GLU, GLOG, 8, 4>(p, a, s);
    }
}

template <bool BF16, bool GLU, int GLOG>
void launch_group(const W4Args &args, hipStream_t s)
{
    const W4Plan p = w4_plan({args.R, args.K, args.N, args.E, GLOG, args.zeros[0] || args.zeros[1], GLU});
    W4Args a = args;
    a.list = nullptr;
    if (!p.listed)
        return launch_variant<BF16, GLU, GLOG>(p.launch[0], a, s);
    W4Lists lists{};
    for (int i = 0; i < 2; ++i) {
        lists.count[i] = a.scratch + i;
        lists.most[i] = p.most[i];
        lists.rows[i] = p.rows[i];
        lists.us[i] = p.us[i];
    }
    lists.least_us = p.least_us;
    lists.limit = p.limit;
    lists.list[0] = (int4 *)(a.scratch + 4);
    lists.list[1] = lists.list[0] + lists.most[0] + 1;
    w4_list_kernel<<<1, 1024, 0, s>>>(a, lists);
    for (int i = 1; i >= 0; --i) {
        a.list = lists.list[i];
        a.count = lists.count[i];
        a.most = lists.most[i];
        launch_variant<BF16, GLU, GLOG>(p.launch[i], a, s);
    }
}

template <bool BF16, bool GLU>
void launch_type(const W4Args &a, hipStream_t s)
{
    if (a.group_log2 == 5)
        launch_group<BF16, GLU, 5>(a, s);
    else if (a.group_log2 == 6)
        launch_group<BF16, GLU, 6>(a, s);
    else
        launch_group<BF16, GLU, 7>(a, s);
}

hipError_t launch_w4(bool bf16, bool glu, const W4Args &a, hipStream_t s)
{
    if (bf16)
        glu ? launch_type<true, true>(a, s) : launch_type<true, false>(a, s);
    else
        glu ? launch_type<false, true>(a, s) : launch_type<false, false>(a, s);
    return hipGetLastError();
}

}  // namespace moe
