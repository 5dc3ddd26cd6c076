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

// Rows a block's tile holds.
constexpr int kW4Rows = 16;

// Eight codes -> eight 16-bit numbers 16 + q, in the order of permute8().
template <bool BF16>
MOE_DEV u32x4 expand8(uint32_t c)
{
    if constexpr (BF16)   // 16 = 0x4180, steps of 1 at bit 3
        return (u32x4){((c << 3) & 0x00780078u) | 0x41804180u, ((c >> 1) & 0x00780078u) | 0x41804180u,
                       ((c >> 5) & 0x00780078u) | 0x41804180u, ((c >> 9) & 0x00780078u) | 0x41804180u};
    else                  // 16 = 0x4C00, steps of 1 at bit 6
        return (u32x4){((c << 6) & 0x03C003C0u) | 0x4C004C00u, ((c << 2) & 0x03C003C0u) | 0x4C004C00u,
                       ((c >> 2) & 0x03C003C0u) | 0x4C004C00u, ((c >> 6) & 0x03C003C0u) | 0x4C004C00u};
}

// k 0..7 -> 0 4 1 5 2 6 3 7: what the two halves of a code dword give in turn.
MOE_DEV u32x4 permute8(u32x4 x)
{
    return (u32x4){__builtin_amdgcn_perm(x[2], x[0], 0x05040100u), __builtin_amdgcn_perm(x[2], x[0], 0x07060302u),
                   __builtin_amdgcn_perm(x[3], x[1], 0x05040100u), __builtin_amdgcn_perm(x[3], x[1], 0x07060302u)};
}

// The tile number `c` of a call: its expert and rows (n = 0: past the last one).
// Every thread of the block calls it.
struct W4Tile {
    int e, row, n;
};

MOE_DEV W4Tile w4_tile(const W4Args &a, int c, int tile_rows)
{
    if (!a.offsets) {
        const int row = c * tile_rows;
        return {0, row, row < a.R ? min(tile_rows, a.R - row) : 0};
    }
    __shared__ int found[3], wsum[4];
    const int tid = threadIdx.x, w = tid >> 6, l = tid & 63;
    if (tid == 0)
        found[2] = 0;
    int before = 0;
    for (int e0 = 0; e0 < a.E; e0 += 256) {
        __syncthreads();
        const int e = e0 + tid;
        int lo = 0, hi = 0;
        if (e < a.E) {
            lo = min(max(a.offsets[e], 0), a.R);
            hi = min(max(a.offsets[e + 1], lo), a.R);
        }
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
        for (int i = 0; i < 4; ++i) {
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
{
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

template <bool BF16, bool GLU>
__global__ __launch_bounds__(256) void w4_kernel(W4Args a)
{
    constexpr int NW = GLU ? 2 : 1;
    __shared__ float red[4][NW][16][17];
    const int tid = threadIdx.x, w = tid >> 6, l = tid & 63;
    if (blockIdx.x == 0)
        w4_status(a);
    const int nt = (a.N + 15) / 16, n0 = (int)(blockIdx.x % nt) * 16;
    const W4Tile t = w4_tile(a, blockIdx.x / nt, kW4Rows);
    if (t.n == 0)
        return;
    const int n = n0 + (l & 15), q = l >> 4;
    const bool in = n < a.N;
    const int G = a.K >> a.group_log2;
    const int64_t col = (int64_t)t.e * a.N + (in ? n : 0);
    const uint32_t one = BF16 ? 0x3F803F80u : 0x3C003C00u;
    const u32x4 ones = {one, one, one, one};
    const uint16_t *xr = a.x + (int64_t)(t.row + min(l & 15, t.n - 1)) * a.ldx;
    f32x4 acc[NW] = {}, tmp[NW] = {}, sum = {};
    const int steps = 1 << (a.group_log2 - 5);   // of 32 k, a group
    for (int g = w; g < G; g += 4) {
#pragma unroll
        for (int i = 0; i < NW; ++i)
            tmp[i] = (f32x4){};
        sum = (f32x4){};
        for (int s = 0; s < steps; ++s) {
            const int k = (g << a.group_log2) + 32 * s + 8 * q;
            const u32x4 xf = permute8(*(const u32x4 *)(xr + k));
            sum = dense_mfma<BF16>(xf, ones, sum);
#pragma unroll
            for (int i = 0; i < NW; ++i) {
                const uint32_t c = *(const uint32_t *)(a.codes[i] + col * (a.K / 2) + k / 2);
                tmp[i] = dense_mfma<BF16>(xf, expand8<BF16>(c), tmp[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < NW; ++i) {
            const float sc = act_to_f32<BF16>(a.scales[i][col * G + g]);
            const float z = 16.0f + (a.zeros[i] ? (float)a.zeros[i][col * G + g] : 8.0f);
#pragma unroll
            for (int r = 0; r < 4; ++r)
                acc[i][r] = fmaf(sc, fmaf(-z, sum[r], tmp[i][r]), acc[i][r]);
        }
    }
#pragma unroll
    for (int i = 0; i < NW; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r)
            red[w][i][4 * q + r][l & 15] = acc[i][r];
    __syncthreads();
    const int m = tid >> 4, c = tid & 15, nn = n0 + c;
    if (m >= t.n || nn >= a.N)
        return;
    float v[NW];
#pragma unroll
    for (int i = 0; i < NW; ++i)
        v[i] = (red[0][i][m][c] + red[1][i][m][c]) + (red[2][i][m][c] + red[3][i][m][c]);
    float y = v[0];
    if constexpr (GLU)
        y = (a.act == MOE_EXL3_ACT_SILU ? act_value<MOE_EXL3_ACT_SILU>(v[0]) : act_value<MOE_EXL3_ACT_GELU_TANH>(v[0])) *
            v[1];
    const int64_t row = t.row + m;
    if (a.base)
        y += act_to_f32<BF16>(a.base[row * a.ldbase + nn]);
    a.y[row * a.ldy + nn] = BF16 ? f32_to_bf16_bits(y) : f32_to_f16_bits(y);
}

hipError_t launch_w4(bool bf16, bool glu, const W4Args &a, hipStream_t s)
{
    const unsigned grid = (unsigned)((a.N + 15) / 16) *
                          (unsigned)(a.offsets ? a.R / kW4Rows + min(a.E, a.R) : (a.R + kW4Rows - 1) / kW4Rows);
    if (bf16)
        glu ? w4_kernel<true, true><<<grid, 256, 0, s>>>(a) : w4_kernel<true, false><<<grid, 256, 0, s>>>(a);
    else
        glu ? w4_kernel<false, true><<<grid, 256, 0, s>>>(a) : w4_kernel<false, false><<<grid, 256, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace moe
