// Host side of the products with 4-bit weights: argument checks and launches.
// Declarations and the full contract are in include/moe_exl3.h.
#include "args.h"
#include "w4.h"

using namespace moe;

namespace {

int check_desc(const moe_exl3_w4_desc *d)
{
    if (!d)
        return MOE_EXL3_ERR_INVALID_ARG;
    if (d->group != 32 && d->group != 64 && d->group != 128)
        return MOE_EXL3_ERR_UNSUPPORTED;
    for (const int rc : {check_size(d->n_in), check_size(d->n_out), check_dtype(d->act_dtype)})
        if (rc)
            return rc;
    if (d->n_in % d->group || d->n_experts <= 0)
        return MOE_EXL3_ERR_INVALID_ARG;
    if (d->act != MOE_EXL3_ACT_SILU && d->act != MOE_EXL3_ACT_GELU_TANH)
        return MOE_EXL3_ERR_UNSUPPORTED;
    if (d->n_experts > 1024)
        return MOE_EXL3_ERR_UNSUPPORTED;
    return (int64_t)d->n_in * d->n_out / 2 >= kSpanLimit ? MOE_EXL3_ERR_UNSUPPORTED : MOE_EXL3_OK;
}

// Rows of this length must be addressable.
bool rows_fit(int64_t R, int64_t cols) { return R < kSpanLimit && R * cols * 2 < kSpanLimit; }

// (One expert's zeros in a stack begin at a multiple of 8, N being one; its codes
// and scales at one of 16.)
int check_weights(const moe_exl3_w4 *w)
{
    if (!w || !w->codes || !w->scales)
        return MOE_EXL3_ERR_INVALID_ARG;
    return aligned16(w->codes) && aligned16(w->scales) && (uintptr_t)w->zeros % 8 == 0 ? MOE_EXL3_OK
                                                                                       : MOE_EXL3_ERR_MISALIGNED;
}

bool meets_weights(const Mat &out, const moe_exl3_w4_desc &d, const moe_exl3_w4 &w)
{
    const int64_t groups = (int64_t)d.n_experts * d.n_out * (d.n_in / d.group);
    return spans_meet(out.p, out.span(), w.codes, (int64_t)d.n_experts * d.n_out * d.n_in / 2) ||
           spans_meet(out.p, out.span(), w.scales, 2 * groups) ||
           (w.zeros && spans_meet(out.p, out.span(), w.zeros, groups));
}

int run(const moe_exl3_w4_desc *desc, const void *x, int64_t ldx, const moe_exl3_w4 *const (&w)[2], bool glu,
        const int32_t *offsets, const void *base, int64_t ldbase, int64_t rows, void *y, int64_t ldy, void *workspace,
        size_t ws_bytes, void *stream)
{
    int rc = check_desc(desc);
    if (rc)
        return rc;
    if (rows < 0)
        return MOE_EXL3_ERR_INVALID_ARG;
    if (rows == 0)
        return MOE_EXL3_OK;
    const int n = glu ? 2 : 1;
    for (int i = 0; i < n; ++i)
        if ((rc = check_weights(w[i])))
            return rc;
    if (!offsets && desc->n_experts != 1)
        return MOE_EXL3_ERR_INVALID_ARG;
    if ((uintptr_t)offsets & 3u)
        return MOE_EXL3_ERR_MISALIGNED;
    const int64_t K = desc->n_in, N = desc->n_out;
    const Mat mx{x, rows, K, ldx}, mb{base, base ? rows : 0, N, ldbase}, my{y, rows, N, ldy};
    for (const Mat &m : {mx, mb, my})
        if ((rc = check_mat(m)))
            return rc;
    if (!rows_fit(rows, K) || !rows_fit(rows, N))
        return MOE_EXL3_ERR_UNSUPPORTED;
    if (overlap(my, mx) || (overlap(my, mb) && !(base == y && ldbase == ldy)) ||
        (offsets && spans_meet(y, my.span(), offsets, 4 * ((int64_t)desc->n_experts + 1))))
        return MOE_EXL3_ERR_INVALID_ARG;
    for (int i = 0; i < n; ++i)
        if (meets_weights(my, *desc, *w[i]))
            return MOE_EXL3_ERR_INVALID_ARG;
    if ((rc = check_ws(workspace, ws_bytes, kAlign + align_up(w4_scratch(rows, desc->n_experts)))))
        return rc;
    W4Args a{};
    a.x = (const uint16_t *)x;
    a.ldx = ldx;
    for (int i = 0; i < n; ++i) {
        a.codes[i] = (const uint8_t *)w[i]->codes;
        a.scales[i] = (const uint16_t *)w[i]->scales;
        a.zeros[i] = w[i]->zeros;
    }
    a.offsets = offsets;
    a.base = (const uint16_t *)base;
    a.ldbase = ldbase;
    a.y = (uint16_t *)y;
    a.ldy = ldy;
    a.status = at<int32_t>(workspace, MOE_EXL3_STATUS_OFFSET);
    a.scratch = at<int32_t>(workspace, kAlign);
    a.R = (int)rows;
    a.K = (int)K;
    a.N = (int)N;
    a.E = desc->n_experts;
    a.group_log2 = desc->group == 32 ? 5 : desc->group == 64 ? 6 : 7;
    a.act = desc->act;
    return launch_w4(desc->act_dtype == MOE_EXL3_DT_BF16, glu, a, (hipStream_t)stream) == hipSuccess ? MOE_EXL3_OK
                                                                                                    : MOE_EXL3_ERR_HIP;
}

}  // namespace

extern "C" {

int moe_exl3_w4_workspace_size(const moe_exl3_w4_desc *desc, int64_t max_rows, size_t *bytes)
{
    const int rc = check_desc(desc);
    if (rc)
        return rc;
    if (!bytes || max_rows < 0)
        return MOE_EXL3_ERR_INVALID_ARG;
    if (!rows_fit(max_rows, desc->n_in) || !rows_fit(max_rows, desc->n_out))
        return MOE_EXL3_ERR_UNSUPPORTED;
    *bytes = kAlign + align_up(w4_scratch(max_rows, desc->n_experts));
    return MOE_EXL3_OK;
}

int moe_exl3_w4_linear(const moe_exl3_w4_desc *desc, const void *x, int64_t ldx, const moe_exl3_w4 *w,
                       const int32_t *offsets, const void *base, int64_t ldbase, int64_t rows, void *y, int64_t ldy,
                       void *workspace, size_t ws_bytes, void *stream)
{
    return run(desc, x, ldx, {w, nullptr}, false, offsets, base, ldbase, rows, y, ldy, workspace, ws_bytes, stream);
}

int moe_exl3_w4_glu(const moe_exl3_w4_desc *desc, const void *x, int64_t ldx, const moe_exl3_w4 *w_gate,
                    const moe_exl3_w4 *w_up, const int32_t *offsets, int64_t rows, void *h, int64_t ldh,
                    void *workspace, size_t ws_bytes, void *stream)
{
    return run(desc, x, ldx, {w_gate, w_up}, true, offsets, nullptr, 0, rows, h, ldh, workspace, ws_bytes, stream);
}

}  // extern "C"
