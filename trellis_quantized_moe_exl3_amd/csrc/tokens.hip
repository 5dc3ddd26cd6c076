// Tokens sorted by expert and back, with weights and gradients, and dropout.
#include "dense_gemm.h"
#include "philox.h"
#include "tokens.h"

#include <algorithm>

namespace moe {

// ---------------------------------------------------------------- sort
// Stable counting sort of the slots by expert.  A block holds a chunk of slots (4096
// where it is the only one, else 2048: the ballots of 16 wavefronts take 3 us for
// 4096), a wavefront a run of them; slots of one expert in 64 consecutive ones are
// ranked from ballots over the index bits, earlier ones from the wavefront's
// counts, earlier wavefronts from theirs, and earlier blocks from the counts
// that a first launch left.  A slot's place never comes from an atomic (only the
// first launch's totals do): the tables are the same on each call.  Bound by latency: 3.8 us for 64
// slots, of which 2.2 are an empty launch's; 12.6 for 57344 in two launches, the
// second with its scattered writes 8.8; 18.2 for 131072.
constexpr int kSortWaves = 16;

MOE_DEV int scan64(int v, int l)   // inclusive, over a wavefront
{
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(v, d, 64);
        v += l >= d ? o : 0;
    }
    return v;
}

// counts[e] of the chunk and, at E, its slots with a bad index
__global__ __launch_bounds__(1024) void sort_count_kernel(SortArgs a)
{
    extern __shared__ int32_t cnt[];
    for (int e = threadIdx.x; e <= a.E; e += 1024)
        cnt[e] = 0;
    __syncthreads();
    const int64_t a0 = (int64_t)blockIdx.x * kSortChunk;
#pragma unroll
    for (int i = 0; i < kSortChunk / 1024; ++i) {   // (blocks of several only)
        const int64_t s = a0 + 1024 * i + threadIdx.x;
        if (s < a.n) {
            const int e = a.idx[s];
            if (e != -1)
                atomicAdd(&cnt[(unsigned)e < (unsigned)a.E ? e : a.E], 1);
        }
    }
    __syncthreads();
    for (int e = threadIdx.x; e <= a.E; e += 1024)
        a.hist[(int64_t)blockIdx.x * (a.E + 1) + e] = cnt[e];
}

// counts of the blocks -> sums of the blocks before, the last row of all
__global__ __launch_bounds__(64) void sort_scan_kernel(SortArgs a)
{
    const int e = blockIdx.x, l = threadIdx.x;
    int run = 0;
    for (int b0 = 0; b0 < a.nblk; b0 += 64) {
        const int b = b0 + l;
        int32_t *p = a.hist + (int64_t)b * (a.E + 1) + e;
        const int v = b < a.nblk ? *p : 0;
        const int s = scan64(v, l);
        if (b < a.nblk)
            *p = run + s - v;
        run += __shfl(s, 63, 64);
    }
    if (l == 0)
        a.hist[(int64_t)a.nblk * (a.E + 1) + e] = run;
}

template <int ITER>
__global__ __launch_bounds__(1024) void sort_kernel(SortArgs a)
{
    constexpr int kSortIter = ITER;
    extern __shared__ int32_t first[];                          // [E]
    uint16_t *cnt = (uint16_t *)(first + a.E);                  // [kSortWaves][E]
    __shared__ int wsum[kSortWaves];
    __shared__ int bad;
    const int tid = threadIdx.x, w = tid >> 6, l = tid & 63;
    const int E = a.E, blk = blockIdx.x;
    for (int i = tid; i < kSortWaves * E; i += 1024)
        cnt[i] = 0;
    if (tid == 0)
        bad = 0;
    int nbits = 0;
    while ((1 << nbits) < E)
        ++nbits;
    const int64_t s0 = ((int64_t)blk * kSortWaves + w) * (64 * kSortIter) + l;
    int ev[kSortIter], rank[kSortIter];
#pragma unroll
    for (int c = 0; c < kSortIter; ++c)
        ev[c] = s0 + 64 * c < a.n ? a.idx[s0 + 64 * c] : -1;
    // the blocks' counts, all of them in flight at once (the others wrote them on
    // other XCDs: 2 us a round trip)
    const int64_t row = E + 1;
    int total = 0, before = 0;
    if (a.nblk > kSortScan) {
        if (tid < E) {
            before = a.hist[blk * row + tid];
            total = a.hist[a.nblk * row + tid];
        }
    } else if (a.nblk > 1 && tid < E) {
        int v[kSortScan];
#pragma unroll
        for (int b = 0; b < kSortScan; ++b)
            v[b] = b < a.nblk ? a.hist[b * row + tid] : 0;
#pragma unroll
        for (int b = 0; b < kSortScan; ++b) {
            total += v[b];
            before += b < blk ? v[b] : 0;
        }
    }
    __syncthreads();
    uint16_t *mine = cnt + w * E;
    bool wrong = false;
#pragma unroll
    for (int c = 0; c < kSortIter; ++c) {
        rank[c] = 0;
        if (s0 - l + 64 * c >= a.n)   // (the whole wavefront)
            break;
        const int e = ev[c];
        const bool valid = (unsigned)e < (unsigned)E;
        wrong |= !valid && e != -1;
        uint64_t m = __ballot(valid);
        for (int b = 0; b < nbits; ++b) {
            const bool bit = (e >> b) & 1;
            const uint64_t bb = __ballot(bit);
            m &= bit ? bb : ~bb;
        }
        rank[c] = valid ? mine[e] + __popcll(m & ((1ull << l) - 1)) : 0;
        wave_lds_fence();
        if (valid && (m >> l) == 1ull)   // the last lane of its expert
            mine[e] += (uint16_t)__popcll(m);
        wave_lds_fence();
    }
    if (wrong)
        bad = 1;
    __syncthreads();
    // per expert: the wavefronts' counts -> their sums before, the chunk's total
    // (of the wavefronts that have slots)
    const int waves =
        (int)min<int64_t>(kSortWaves, (a.n - (s0 - l) + 64 * kSortIter - 1) / (64 * kSortIter) + w);
    int own = 0;
    if (tid < E) {
        int t[kSortWaves];
#pragma unroll
        for (int v = 0; v < kSortWaves; ++v)
            t[v] = v < waves ? cnt[v * E + tid] : 0;
#pragma unroll
        for (int v = 0; v < kSortWaves; ++v) {
            if (v < waves)
                cnt[v * E + tid] = (uint16_t)own;
            own += t[v];
        }
    }
    if (a.nblk == 1)
        total = own;
    const int incl = scan64(total, l);
    if (l == 63)
        wsum[w] = incl;
    __syncthreads();
    int off = incl - total;
#pragma unroll
    for (int v = 0; v < kSortWaves; ++v)
        off += v < w ? wsum[v] : 0;
    if (tid < E)
        first[tid] = off + before;
    if (blk == 0) {
        if (tid < E) {
            a.offsets[tid] = off;
            if (tid == E - 1)
                a.offsets[E] = off + total;
            if (a.counts)
                a.counts[tid] = total;
        }
        if (tid == 0) {
            int faults = a.nblk == 1 ? bad : 0;
            for (int b = a.nblk > kSortScan ? a.nblk : 0; a.nblk > 1 && b < (a.nblk > kSortScan ? a.nblk + 1 : a.nblk); ++b)
                faults |= a.hist[b * row + E];
            *a.status = faults ? MOE_EXL3_STATUS_BAD_INDEX : 0;
        }
    }
    __syncthreads();
#pragma unroll
    for (int c = 0; c < kSortIter; ++c) {
        const int64_t s = s0 + 64 * c;
        if (s >= a.n)
            break;
        const int e = ev[c];
        int p = -1;
        if ((unsigned)e < (unsigned)E) {
            p = first[e] + cnt[w * E + e] + rank[c];
            if (a.sorted)
                a.sorted[p] = (int32_t)s;
        }
        a.pos[s] = p;
    }
}

hipError_t launch_sort(const SortArgs &a, hipStream_t s)
{
    if (a.nblk > 1) {
        sort_count_kernel<<<(unsigned)a.nblk, 1024, (a.E + 1) * sizeof(int32_t), s>>>(a);
        if (a.nblk > kSortScan)
            sort_scan_kernel<<<(unsigned)(a.E + 1), 64, 0, s>>>(a);
    }
    const size_t lds = a.E * sizeof(int32_t) + kSortWaves * a.E * sizeof(uint16_t);
    static_assert(kSortChunk == 2 * 64 * kSortWaves && kSortAlone == 4 * 64 * kSortWaves, "slots of a block");
    if (a.nblk == 1)
        sort_kernel<4><<<1, 1024, lds, s>>>(a);
    else
        sort_kernel<2><<<(unsigned)a.nblk, 1024, lds, s>>>(a);
    return hipGetLastError();
}

// ---------------------------------------------------------------- rows
template <bool BF16>
MOE_DEV void unpack8(u32x4 r, float (&v)[8])
{
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        v[2 * j] = act_to_f32<BF16>((uint16_t)r[j]);
        v[2 * j + 1] = act_to_f32<BF16>((uint16_t)(r[j] >> 16));
    }
}

template <bool BF16>
MOE_DEV u32x4 round8(const float (&v)[8])
{
    return (u32x4){pack16<BF16>(v[0], v[1]), pack16<BF16>(v[2], v[3]), pack16<BF16>(v[4], v[5]),
                   pack16<BF16>(v[6], v[7])};
}

// The products' sums of a block's lanes -> dw, in a fixed order.  Across a wavefront
// the KB sums are halved with the lanes: at each exchange a lane keeps half of its
// sums and gives the others away (KB + 2 exchanges instead of 6 KB).
template <int KB>
MOE_DEV void store_dots(const TokenArgs &a, int64_t t, const float (&dot)[KB])
{
    __shared__ float part[4][KB];
    const int w = threadIdx.x >> 6, l = threadIdx.x & 63, nw = blockDim.x >> 6;
    float v[KB];
#pragma unroll
    for (int j = 0; j < KB; ++j)
        v[j] = dot[j];
    int d = 32;
#pragma unroll
    for (int n = KB / 2; n > 0; n >>= 1, d >>= 1) {
        const bool upper = l & d;
#pragma unroll
        for (int j = 0; j < n; ++j) {
            const float got = __shfl_xor(upper ? v[j] : v[j + n], d, 64);
            v[j] = (upper ? v[j + n] : v[j]) + got;
        }
    }
#pragma unroll
    for (; d > 0; d >>= 1)
        v[0] += __shfl_xor(v[0], d, 64);
    if (l % (64 / KB) == 0)
        part[w][l / (64 / KB)] = v[0];
    __syncthreads();
    if ((int)threadIdx.x < a.k) {
        float s = part[0][threadIdx.x];
        for (int i = 1; i < nw; ++i)
            s += part[i][threadIdx.x];
        a.dw[t * a.k + threadIdx.x] = s;
    }
}

// A block per token reads its row once and writes those of its slots (with DOT it
// reads theirs too); the other way round it reads all its slots' rows, k of
// them in flight, and writes one.  Bound by memory: the sorted rows, read or
// written once, pass the caches by (7168 tokens x 8 of 4096, there and back: 105
// and 118 us with ordinary accesses, 90 and 97 with these: 6.1 TB/s back, where
// all but a ninth is read; a 1 GiB copy reaches 5.1).  w is applied in fp32, and a
// slot without a row costs nothing.
template <bool BF16, int KB, bool DOT>
__global__ __launch_bounds__(256) void spread_kernel(TokenArgs a)
{
    const int64_t t = a.first + blockIdx.x;
    int pos[KB];
    float w[KB], dot[KB];
#pragma unroll
    for (int j = 0; j < KB; ++j) {
        pos[j] = j < a.k ? a.pos[t * a.k + j] : -1;
        if ((uint32_t)pos[j] >= (uint64_t)a.rows)
            pos[j] = -1;
        w[j] = j < a.k && a.w ? a.w[t * a.k + j] : 1.0f;
        dot[j] = 0.0f;
    }
    const uint64_t groups = (uint64_t)(a.H / 8);
    uint64_t seed = 0, offset = 0;
    if (a.drop.rng) {
        seed = a.drop.rng[0];
        offset = a.drop.rng[1] + t * groups;
    }
    for (int c = threadIdx.x; c < a.H / 8; c += blockDim.x) {
        float x[8];
        unpack8<BF16>(*(const u32x4 *)(a.x + t * a.ldx + 8 * c), x);
        u32x4 z[KB];
        if constexpr (DOT)
#pragma unroll
            for (int j = 0; j < KB; ++j)
                if (pos[j] >= 0)
                    z[j] = __builtin_nontemporal_load((const u32x4 *)(a.z + pos[j] * a.ldz + 8 * c));
        if (a.drop.rng)
            drop8(a.drop, seed, offset + c, x);
#pragma unroll
        for (int j = 0; j < KB; ++j) {
            if (pos[j] < 0)
                continue;
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] = w[j] * x[i];
            __builtin_nontemporal_store(round8<BF16>(v), (u32x4 *)(a.out + pos[j] * a.ldo + 8 * c));
            if constexpr (DOT) {
                unpack8<BF16>(z[j], v);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    dot[j] = fmaf(x[i], v[i], dot[j]);
            }
        }
    }
    if constexpr (DOT)
        store_dots<KB>(a, t, dot);
}

template <bool BF16, int KB, bool DOT>
__global__ __launch_bounds__(256) void gather_kernel(TokenArgs a)
{
    const int64_t t = a.first + blockIdx.x;
    int pos[KB];
    float w[KB], dot[KB];
#pragma unroll
    for (int j = 0; j < KB; ++j) {
        pos[j] = j < a.k ? a.pos[t * a.k + j] : -1;
        if ((uint32_t)pos[j] >= (uint64_t)a.rows)
            pos[j] = -1;
        w[j] = j < a.k && a.w ? a.w[t * a.k + j] : 1.0f;
        dot[j] = 0.0f;
    }
    const uint64_t groups = (uint64_t)(a.H / 8);
    uint64_t seed = 0, offset = 0;
    if (a.drop.rng) {
        seed = a.drop.rng[0];
        offset = a.drop.rng[1] + t * groups;
    }
    for (int c = threadIdx.x; c < a.H / 8; c += blockDim.x) {
        u32x4 z[KB];
#pragma unroll
        for (int j = 0; j < KB; ++j)
            if (pos[j] >= 0)
                z[j] = __builtin_nontemporal_load((const u32x4 *)(a.z + pos[j] * a.ldz + 8 * c));
        float x[8], y[8];
        if constexpr (DOT)
            unpack8<BF16>(*(const u32x4 *)(a.x + t * a.ldx + 8 * c), x);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            y[i] = 0.0f;
#pragma unroll
        for (int j = 0; j < KB; ++j) {
            if (pos[j] < 0)
                continue;
            float v[8];
            unpack8<BF16>(z[j], v);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                y[i] = fmaf(w[j], v[i], y[i]);
                if constexpr (DOT)
                    dot[j] = fmaf(x[i], v[i], dot[j]);
            }
        }
        if (a.drop.rng)
            drop8(a.drop, seed, offset + c, y);
        if (a.base) {
            float b[8];
            unpack8<BF16>(*(const u32x4 *)(a.base + t * a.ldbase + 8 * c), b);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                y[i] += b[i];
        }
        __builtin_nontemporal_store(round8<BF16>(y), (u32x4 *)(a.out + t * a.ldo + 8 * c));
    }
    if constexpr (DOT)
        store_dots<KB>(a, t, dot);
}

template <bool BF16, bool SPREAD, int KB>
void launch_rows(const TokenArgs &a, unsigned tokens, hipStream_t s)
{
    const unsigned threads = (unsigned)min(256, (a.H / 8 + 63) / 64 * 64);
    if constexpr (SPREAD) {
        if (a.dw)
            spread_kernel<BF16, KB, true><<<tokens, threads, 0, s>>>(a);
        else
            spread_kernel<BF16, KB, false><<<tokens, threads, 0, s>>>(a);
    } else {
        if (a.dw)
            gather_kernel<BF16, KB, true><<<tokens, threads, 0, s>>>(a);
        else
            gather_kernel<BF16, KB, false><<<tokens, threads, 0, s>>>(a);
    }
}

// A launch takes 2^23 tokens at most: with 256 threads each, half of the 2^32 threads
// that a grid may have.
template <bool BF16, bool SPREAD>
hipError_t launch_rows_k(const TokenArgs &args, hipStream_t s)
{
    constexpr int64_t kTokens = 1 << 23;
    TokenArgs a = args;
    for (a.first = 0; a.first < a.T; a.first += kTokens) {
        const unsigned n = (unsigned)std::min(kTokens, a.T - a.first);
        if (a.k <= 2)
            launch_rows<BF16, SPREAD, 2>(a, n, s);
        else if (a.k <= 4)
            launch_rows<BF16, SPREAD, 4>(a, n, s);
        else if (a.k <= 8)
            launch_rows<BF16, SPREAD, 8>(a, n, s);
        else
            launch_rows<BF16, SPREAD, 16>(a, n, s);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess)
            return e;
    }
    return hipSuccess;
}

hipError_t launch_spread(bool bf16, const TokenArgs &a, hipStream_t s)
{
    return bf16 ? launch_rows_k<true, true>(a, s) : launch_rows_k<false, true>(a, s);
}

hipError_t launch_gather(bool bf16, const TokenArgs &a, hipStream_t s)
{
    return bf16 ? launch_rows_k<true, false>(a, s) : launch_rows_k<false, false>(a, s);
}

// ---------------------------------------------------------------- dropout
template <int DT>
MOE_DEV float load1(const void *p, int64_t i)
{
    if constexpr (DT == MOE_EXL3_DT_F32)
        return ((const float *)p)[i];
    else
        return act_to_f32<DT == MOE_EXL3_DT_BF16>(((const uint16_t *)p)[i]);
}

template <int DT>
MOE_DEV void store1(void *p, int64_t i, float v)
{
    if constexpr (DT == MOE_EXL3_DT_F32)
        ((float *)p)[i] = v;
    else
        ((uint16_t *)p)[i] = DT == MOE_EXL3_DT_BF16 ? f32_to_bf16_bits(v) : f32_to_f16_bits(v);
}

// Eight consecutive elements at any address of theirs (rows of an odd length
// begin anywhere; 16-byte accesses need no alignment here).
typedef u32x4 u32x4_any __attribute__((aligned(2)));
template <int DT>
struct Eight {
    u32x4 v[DT == MOE_EXL3_DT_F32 ? 2 : 1];
    MOE_DEV void load(const void *p, int64_t i)
    {
        if constexpr (DT == MOE_EXL3_DT_F32) {
            v[0] = __builtin_nontemporal_load((const u32x4_any *)((const float *)p + i));
            v[1] = __builtin_nontemporal_load((const u32x4_any *)((const float *)p + i + 4));
        } else {
            v[0] = __builtin_nontemporal_load((const u32x4_any *)((const uint16_t *)p + i));
        }
    }
    MOE_DEV void get(float (&f)[8]) const
    {
        if constexpr (DT == MOE_EXL3_DT_F32) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                f[j] = __uint_as_float(v[j / 4][j % 4]);
        } else {
            unpack8<DT == MOE_EXL3_DT_BF16>(v[0], f);
        }
    }
    MOE_DEV void set(const float (&f)[8])
    {
        if constexpr (DT == MOE_EXL3_DT_F32) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[j / 4][j % 4] = __float_as_uint(f[j]);
        } else {
            v[0] = round8<DT == MOE_EXL3_DT_BF16>(f);
        }
    }
    MOE_DEV void store(void *p, int64_t i) const
    {
        if constexpr (DT == MOE_EXL3_DT_F32) {
            __builtin_nontemporal_store(v[0], (u32x4_any *)((float *)p + i));
            __builtin_nontemporal_store(v[1], (u32x4_any *)((float *)p + i + 4));
        } else {
            __builtin_nontemporal_store(v[0], (u32x4_any *)((uint16_t *)p + i));
        }
    }
};

// A thread takes eight columns of a row (one counter), kDropGroups times, all their
// loads in flight before the first is used.  Bound by memory: 16384 x 4096 in bf16 with a
// residual 60.6 us, its gradient 44.4 (6.6 and 6.0 TB/s, a 64 MiB copy 6.9); with a
// 64-bit division for the row, element-wise tails and ordinary accesses both
// took 323 us instead of 113.
constexpr int kDropGroups = 2;

template <int DT, bool RES>
__global__ __launch_bounds__(256) void dropout_kernel(DropoutArgs a, uint32_t groups, uint32_t total)
{
    const uint32_t i0 = blockIdx.x * (256 * kDropGroups) + threadIdx.x;
    Eight<DT> x[kDropGroups], res[kDropGroups];
    uint32_t row[kDropGroups], col[kDropGroups];
    bool whole[kDropGroups];
#pragma unroll
    for (int u = 0; u < kDropGroups; ++u) {
        const uint32_t i = i0 + 256 * u;
        row[u] = i / groups;
        col[u] = 8 * (i - row[u] * groups);
        whole[u] = i < total && col[u] + 8 <= (uint32_t)a.cols;
        if (whole[u]) {
            x[u].load(a.x, row[u] * a.ldx + col[u]);
            if (RES)
                res[u].load(a.residual, row[u] * a.ldr + col[u]);
        }
    }
    uint64_t seed = 0, offset = 0;
    if (a.drop.rng) {
        seed = a.drop.rng[0];
        offset = a.drop.rng[1] + a.counter;
    }
#pragma unroll
    for (int u = 0; u < kDropGroups; ++u) {
        const uint32_t i = i0 + 256 * u;
        if (i >= total)
            return;
        float v[8], b[8];
        if (whole[u]) {
            x[u].get(v);
            if (a.drop.rng)
                drop8(a.drop, seed, offset + i, v);
            if (RES) {
                res[u].get(b);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    v[j] += b[j];
            }
            x[u].set(v);
            x[u].store(a.y, row[u] * a.ldy + col[u]);
            continue;
        }
        // the last columns of a row that is no multiple of eight
        const int n = a.cols - (int)col[u];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            v[j] = j < n ? load1<DT>(a.x, row[u] * a.ldx + col[u] + j) : 0.0f;
            b[j] = RES && j < n ? load1<DT>(a.residual, row[u] * a.ldr + col[u] + j) : 0.0f;
        }
        if (a.drop.rng)
            drop8(a.drop, seed, offset + i, v);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < n)
                store1<DT>(a.y, row[u] * a.ldy + col[u] + j, RES ? v[j] + b[j] : v[j]);
    }
}

template <int DT>
void launch_dropout_type(const DropoutArgs &a, uint32_t groups, uint32_t total, hipStream_t s)
{
    const unsigned grid = (total + 256 * kDropGroups - 1) / (256 * kDropGroups);
    if (a.residual)
        dropout_kernel<DT, true><<<grid, 256, 0, s>>>(a, groups, total);
    else
        dropout_kernel<DT, false><<<grid, 256, 0, s>>>(a, groups, total);
}

hipError_t launch_dropout(int dtype, const DropoutArgs &args, hipStream_t s)
{
    const int64_t groups = (args.cols + 7) / 8;
    const int64_t step = std::max<int64_t>(1, ((int64_t)1 << 30) / groups);   // rows whose groups 32 bits number
    const int64_t size = dtype == MOE_EXL3_DT_F32 ? 4 : 2;
    DropoutArgs a = args;
    for (int64_t r = 0; r < args.rows; r += step) {
        a.rows = std::min(step, args.rows - r);
        a.x = (const char *)args.x + r * args.ldx * size;
        a.residual = args.residual ? (const char *)args.residual + r * args.ldr * size : nullptr;
        a.y = (char *)args.y + r * args.ldy * size;
        a.counter = (uint64_t)(r * groups);
        const uint32_t total = (uint32_t)(a.rows * groups);
        if (dtype == MOE_EXL3_DT_BF16)
            launch_dropout_type<MOE_EXL3_DT_BF16>(a, (uint32_t)groups, total, s);
        else if (dtype == MOE_EXL3_DT_F16)
            launch_dropout_type<MOE_EXL3_DT_F16>(a, (uint32_t)groups, total, s);
        else
            launch_dropout_type<MOE_EXL3_DT_F32>(a, (uint32_t)groups, total, s);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess)
            return e;
    }
    return hipSuccess;
}

}  // namespace moe
