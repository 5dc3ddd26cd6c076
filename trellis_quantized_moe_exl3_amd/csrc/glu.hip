// The gated feed-forward block: both projections, the activation and the
// product in one tile kernel, and its backward pass.
#include "dense_stream.h"

namespace moe {

// dg = dh u act'(g), du = dh act(g), eight columns a thread.  The two are
// rounded to the operands' 16 bits once, for the matrix cores that read them
// next: the only rounding of the backward pass besides its outputs' own.
// Memory-bound: 8 bytes of pre-activations and 2 of dh in, 4 out a value.
template <bool BF16>
__global__ __launch_bounds__(256) void glu_grad_kernel(int act, const float *pre, const uint16_t *dh, int64_t lddh,
                                                       int64_t T, int I, uint16_t *dg, uint16_t *du)
{
    const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8;
    if (i >= T * I)
        return;
    const int64_t t = i / I, c = i - t * I;
    const f32x4 *gp = (const f32x4 *)(pre + i), *up = (const f32x4 *)(pre + T * I + i);
    // pre is read once: past the caches, which keep dg and du for the products
    // (16384 x 2048: 92 -> 79 us)
    const f32x4 g[2] = {__builtin_nontemporal_load(gp), __builtin_nontemporal_load(gp + 1)};
    const f32x4 u[2] = {__builtin_nontemporal_load(up), __builtin_nontemporal_load(up + 1)};
    const u32x4 d = *(const u32x4 *)(dh + t * lddh + c);
    u32x4 og, ou;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float vg[2], vu[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float y = act_to_f32<BF16>((uint16_t)(d[j] >> (16 * h)));
            const float x = g[j >> 1][2 * (j & 1) + h];
            float v, s;
            act_value_slope(act, x, v, s);
            vg[h] = y * u[j >> 1][2 * (j & 1) + h] * s;
            vu[h] = y * v;
        }
        og[j] = pack16<BF16>(vg[0], vg[1]);
        ou[j] = pack16<BF16>(vu[0], vu[1]);
    }
    *(u32x4 *)(dg + i) = og;
    *(u32x4 *)(du + i) = ou;
}

hipError_t launch_glu_grad(bool bf16, int act, const float *pre, const uint16_t *dh, int64_t lddh, int64_t T, int I,
                           uint16_t *dg, uint16_t *du, hipStream_t s)
{
    const unsigned grid = (unsigned)((T * I / 8 + 255) / 256);
    if (bf16)
        glu_grad_kernel<true><<<grid, 256, 0, s>>>(act, pre, dh, lddh, T, I, dg, du);
    else
        glu_grad_kernel<false><<<grid, 256, 0, s>>>(act, pre, dh, lddh, T, I, dg, du);
    return hipGetLastError();
}

hipError_t launch_dense_lin(bool bf16, const DenseArgs &a, hipStream_t s);
hipError_t launch_skinny_lin(bool bf16, const DenseArgs &a, hipStream_t s);

hipError_t launch_dense(int mode, bool bf16, const DenseArgs &a, hipStream_t s)
{
    switch (mode) {
    case DENSE_GLU: return launch_any<DENSE_GLU>(bf16, a, s);
    case DENSE_DX: return launch_any<DENSE_DX>(bf16, a, s);
    case DENSE_DW: return launch_any<DENSE_DW>(bf16, a, s);
    default: return launch_dense_lin(bf16, a, s);
    }
}

hipError_t launch_dense_grads(bool bf16, const DenseArgs &dx, const DenseArgs &dw, bool dw_first, hipStream_t s)
{
    const unsigned grid = (unsigned)(dx.mt * dx.nt + dw.mt * dw.nt);
    if (dw.bm == kDenseSmall)
        bf16 ? dense_grads_kernel<true, true><<<grid, 256, 0, s>>>(dx, dw, dw_first)
             : dense_grads_kernel<false, true><<<grid, 256, 0, s>>>(dx, dw, dw_first);
    else
        bf16 ? dense_grads_kernel<true, false><<<grid, 256, 0, s>>>(dx, dw, dw_first)
             : dense_grads_kernel<false, false><<<grid, 256, 0, s>>>(dx, dw, dw_first);
    return hipGetLastError();
}

hipError_t launch_dense_skinny(int mode, bool bf16, const DenseArgs &a, hipStream_t s)
{
    if (mode == DENSE_LIN)
        return launch_skinny_lin(bf16, a, s);
    return bf16 ? launch_skinny<DENSE_GLU, true>(a, s) : launch_skinny<DENSE_GLU, false>(a, s);
}

}  // namespace moe
