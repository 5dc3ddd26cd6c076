// Host side of the operators around a MoE layer's experts: argument checks,
// workspace plans, launches.  Declarations and the full contract are in
// include/moe_exl3.h.
#include "args.h"
#include "tokens.h"

#include <algorithm>
#include <cmath>

using namespace moe;

namespace {

constexpr int64_t kMaxRows = INT32_MAX;   // of tokens, slots and sorted rows

// A plain array argument.
struct Span {
    const void *p;
    int64_t bytes;
};

int check_desc(const moe_exl3_tokens_desc *d)
{
    if (!d)
        return MOE_EXL3_ERR_INVALID_ARG;
    for (const int rc : {check_size(d->hidden), check_dtype(d->act_dtype)})
        if (rc)
            return rc;
    if (d->n_experts <= 0 || d->top_k <= 0)
        return MOE_EXL3_ERR_INVALID_ARG;
    return d->n_experts > kMaxExperts || d->top_k > kMaxTopK ? MOE_EXL3_ERR_UNSUPPORTED : MOE_EXL3_OK;
}

bool slots_fit(const moe_exl3_tokens_desc &d, int64_t T) { return T <= kMaxRows / d.top_k; }

int64_t sort_blocks(int64_t n) { return n <= kSortAlone ? 1 : cdiv(n, kSortChunk); }

size_t sort_bytes(const moe_exl3_tokens_desc &d, int64_t T)
{
    const int64_t nblk = sort_blocks(T * d.top_k);
    return kAlign + (nblk > 1 ? align_up((size_t)(nblk + 1) * (d.n_experts + 1) * sizeof(int32_t)) : 0);
}

// A table of 4-byte entries, maybe a part of a longer one.
int check_table(const void *p, bool needed)
{
    if (!p)
        return needed ? MOE_EXL3_ERR_INVALID_ARG : MOE_EXL3_OK;
    return (uintptr_t)p & 3u ? MOE_EXL3_ERR_MISALIGNED : MOE_EXL3_OK;
}

int check_drop(const moe_exl3_drop *d, Drop &out)
{
    out = Drop{};
    if (!d)
        return MOE_EXL3_OK;
    if (!(d->p >= 0.0 && d->p <= 1.0))   // (a NaN fails both)
        return MOE_EXL3_ERR_INVALID_ARG;
    const uint32_t least = (uint32_t)std::floor(d->p * 65536.0 + 0.5);
    if (least == 0)
        return MOE_EXL3_OK;
    if (!d->rng)
        return MOE_EXL3_ERR_INVALID_ARG;
    if ((uintptr_t)d->rng & 7u)
        return MOE_EXL3_ERR_MISALIGNED;
    out.rng = d->rng;
    out.least = least;
    out.factor = least < 65536 ? 65536.0f / (float)(65536 - least) : 0.0f;
    return MOE_EXL3_OK;
}

// The written matrix and arrays meet neither what is read nor each other.
// `same`: a matrix read that may be the written one itself.
bool meets(const Mat &out, const Mat *in, int n, const Span *arrays, int m, int same = -1)
{
    for (int i = 0; i < n; ++i)
        if (overlap(out, in[i]) && !(i == same && in[i].p == out.p && in[i].ld == out.ld))
            return true;
    for (int i = 0; i < m; ++i)
        if (out.p && spans_meet(out.p, out.span(), arrays[i].p, arrays[i].p ? arrays[i].bytes : 0))
            return true;
    return false;
}

// The slots' tables, as every row operator takes them, and dw.
int check_slots(const moe_exl3_tokens_desc &d, int64_t T, int64_t rows, const int32_t *pos, const float *w,
                const float *dw)
{
    if (!slots_fit(d, T) || rows > kMaxRows)
        return MOE_EXL3_ERR_UNSUPPORTED;
    for (const int rc : {check_table(pos, true), check_table(w, false), check_table(dw, false)})
        if (rc)
            return rc;
    const int64_t n = 4 * T * d.top_k;
    if (dw && (spans_meet(dw, n, pos, n) || (w && spans_meet(dw, n, w, n))))
        return MOE_EXL3_ERR_INVALID_ARG;
    return MOE_EXL3_OK;
}

int hip_status(hipError_t e) { return e == hipSuccess ? MOE_EXL3_OK : MOE_EXL3_ERR_HIP; }

}  // namespace

extern "C" {

int moe_exl3_sort_workspace_size(const moe_exl3_tokens_desc *desc, int64_t max_tokens, size_t *bytes)
{
    const int rc = check_desc(desc);
    if (rc)
        return rc;
    if (!bytes || max_tokens < 0)
        return MOE_EXL3_ERR_INVALID_ARG;
    if (!slots_fit(*desc, max_tokens))
        return MOE_EXL3_ERR_UNSUPPORTED;
    *bytes = sort_bytes(*desc, max_tokens);
    return MOE_EXL3_OK;
}

int moe_exl3_sort(const moe_exl3_tokens_desc *desc, const int32_t *idx, int64_t T, int32_t *counts, int32_t *offsets,
                  int32_t *sorted_ids, int32_t *pos, void *workspace, size_t ws_bytes, void *stream)
{
    int rc = check_desc(desc);
    if (rc)
        return rc;
    if (T < 0)
        return MOE_EXL3_ERR_INVALID_ARG;
    if (!slots_fit(*desc, T))
        return MOE_EXL3_ERR_UNSUPPORTED;
    const int64_t E = desc->n_experts, n = T * desc->top_k;
    for (const int r : {check_table(idx, T > 0), check_table(counts, false), check_table(offsets, true),
                        check_table(sorted_ids, false), check_table(pos, T > 0)})
        if (r)
            return r;
    const Span out[] = {{counts, 4 * E}, {offsets, 4 * (E + 1)}, {sorted_ids, 4 * n}, {pos, 4 * n}};
    for (int i = 0; i < 4; ++i) {
        if (out[i].p && spans_meet(out[i].p, out[i].bytes, idx, 4 * n))
            return MOE_EXL3_ERR_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if (out[i].p && out[j].p && spans_meet(out[i].p, out[i].bytes, out[j].p, out[j].bytes))
                return MOE_EXL3_ERR_INVALID_ARG;
    }
    if ((rc = check_ws(workspace, ws_bytes, sort_bytes(*desc, T))))
        return rc;
    SortArgs a{};
    a.idx = idx;
    a.n = n;
    a.E = (int)E;
    a.nblk = (int)sort_blocks(n);   // (no slots: one block writes the tables of none)
    a.hist = at<int32_t>(workspace, kAlign);
    a.counts = counts;
    a.offsets = offsets;
    a.sorted = sorted_ids;
    a.pos = pos;
    a.status = at<int32_t>(workspace, MOE_EXL3_STATUS_OFFSET);
    return hip_status(launch_sort(a, (hipStream_t)stream));
}

int moe_exl3_dispatch(const moe_exl3_tokens_desc *desc, const void *x, int64_t ldx, const int32_t *pos, const float *w,
                      int64_t T, int64_t rows, void *out, int64_t ldo, void *stream)
{
    int rc = check_desc(desc);
    if (rc)
        return rc;
    if (T < 0 || rows < 0)
        return MOE_EXL3_ERR_INVALID_ARG;
    if (T == 0 || rows == 0)
        return MOE_EXL3_OK;
    const Mat mx{x, T, desc->hidden, ldx}, mo{out, rows, desc->hidden, ldo};
    for (const int r : {check_mat(mx, kNoLimit), check_mat(mo, kNoLimit), check_slots(*desc, T, rows, pos, w, nullptr)})
        if (r)
            return r;
    const int64_t n = 4 * T * desc->top_k;
    const Span arrays[] = {{pos, n}, {w, n}};
    if (meets(mo, &mx, 1, arrays, 2))
        return MOE_EXL3_ERR_INVALID_ARG;
    TokenArgs a{};
    a.x = (const uint16_t *)x;
    a.ldx = ldx;
    a.out = (uint16_t *)out;
    a.ldo = ldo;
    a.pos = pos;
    a.w = w;
    a.T = T;
    a.rows = rows;
    a.H = desc->hidden;
    a.k = desc->top_k;
    return hip_status(launch_spread(desc->act_dtype == MOE_EXL3_DT_BF16, a, (hipStream_t)stream));
}

int moe_exl3_dispatch_backward(const moe_exl3_tokens_desc *desc, const void *dout, int64_t lddo, const void *x,
                               int64_t ldx, const int32_t *pos, const float *w, int64_t T, int64_t rows, void *dx,
                               int64_t lddx, float *dw, void *stream)
{
    int rc = check_desc(desc);
    if (rc)
        return rc;
    if (T < 0 || rows < 0)
        return MOE_EXL3_ERR_INVALID_ARG;
    if (T == 0)
        return MOE_EXL3_OK;
    const Mat mx{x, dw ? T : 0, desc->hidden, ldx}, mz{dout, rows, desc->hidden, lddo}, mo{dx, T, desc->hidden, lddx};
    for (const int r : {check_mat(mx, kNoLimit), check_mat(mz, kNoLimit), check_mat(mo, kNoLimit),
                        check_slots(*desc, T, rows, pos, w, dw)})
        if (r)
            return r;
    const int64_t n = 4 * T * desc->top_k;
    const Span arrays[] = {{pos, n}, {w, n}, {dw, n}};
    const Mat in[] = {mx, mz};
    if (meets(mo, in, 2, arrays, 3) || (dw && (spans_meet(dw, n, x, mx.span()) || spans_meet(dw, n, dout, mz.span()))))
        return MOE_EXL3_ERR_INVALID_ARG;
    TokenArgs a{};
    a.x = (const uint16_t *)x;
    a.ldx = ldx;
    a.z = (const uint16_t *)dout;
    a.ldz = lddo;
    a.out = (uint16_t *)dx;
    a.ldo = lddx;
    a.pos = pos;
    a.w = w;
    a.dw = dw;
    a.T = T;
    a.rows = rows;
    a.H = desc->hidden;
    a.k = desc->top_k;
    return hip_status(launch_gather(desc->act_dtype == MOE_EXL3_DT_BF16, a, (hipStream_t)stream));
}

int moe_exl3_combine(const moe_exl3_tokens_desc *desc, const void *z, int64_t ldz, const int32_t *pos, const float *w,
                     const void *base, int64_t ldbase, const moe_exl3_drop *drop, int64_t T, int64_t rows, void *y,
                     int64_t ldy, void *stream)
{
    int rc = check_desc(desc);
    if (rc)
        return rc;
    if (T < 0 || rows < 0)
        return MOE_EXL3_ERR_INVALID_ARG;
    TokenArgs a{};
    if ((rc = check_drop(drop, a.drop)))
        return rc;
    if (T == 0)
        return MOE_EXL3_OK;
    const Mat mz{z, rows, desc->hidden, ldz}, mb{base, base ? T : 0, desc->hidden, ldbase}, mo{y, T, desc->hidden, ldy};
    for (const int r : {check_mat(mz, kNoLimit), check_mat(mb, kNoLimit), check_mat(mo, kNoLimit),
                        check_slots(*desc, T, rows, pos, w, nullptr)})
        if (r)
            return r;
    const int64_t n = 4 * T * desc->top_k;
    const Span arrays[] = {{pos, n}, {w, n}, {a.drop.rng, 16}};
    const Mat in[] = {mb, mz};
    if (meets(mo, in, 2, arrays, 3, 0))
        return MOE_EXL3_ERR_INVALID_ARG;
    a.z = (const uint16_t *)z;
    a.ldz = ldz;
    a.out = (uint16_t *)y;
    a.ldo = ldy;
    a.base = (const uint16_t *)base;
    a.ldbase = ldbase;
    a.pos = pos;
    a.w = w;
    a.T = T;
    a.rows = rows;
    a.H = desc->hidden;
    a.k = desc->top_k;
    return hip_status(launch_gather(desc->act_dtype == MOE_EXL3_DT_BF16, a, (hipStream_t)stream));
}

int moe_exl3_combine_backward(const moe_exl3_tokens_desc *desc, const void *dy, int64_t lddy, const void *z, int64_t ldz,
                              const int32_t *pos, const float *w, const moe_exl3_drop *drop, int64_t T, int64_t rows,
                              void *dz, int64_t lddz, float *dw, void *stream)
{
    int rc = check_desc(desc);
    if (rc)
        return rc;
    if (T < 0 || rows < 0)
        return MOE_EXL3_ERR_INVALID_ARG;
    TokenArgs a{};
    if ((rc = check_drop(drop, a.drop)))
        return rc;
    if (T == 0 || (rows == 0 && !dw))
        return MOE_EXL3_OK;
    const Mat my{dy, T, desc->hidden, lddy}, mz{z, dw ? rows : 0, desc->hidden, ldz}, mo{dz, rows, desc->hidden, lddz};
    for (const int r : {check_mat(my, kNoLimit), check_mat(mz, kNoLimit), check_mat(mo, kNoLimit),
                        check_slots(*desc, T, rows, pos, w, dw)})
        if (r)
            return r;
    const int64_t n = 4 * T * desc->top_k;
    const Span arrays[] = {{pos, n}, {w, n}, {dw, n}, {a.drop.rng, 16}};
    const Mat in[] = {mz, my};
    if (meets(mo, in, 2, arrays, 4, 0) ||
        (dw && (spans_meet(dw, n, dy, my.span()) || spans_meet(dw, n, z, mz.span()) ||
                (a.drop.rng && spans_meet(dw, n, a.drop.rng, 16)))))
        return MOE_EXL3_ERR_INVALID_ARG;
    a.x = (const uint16_t *)dy;
    a.ldx = lddy;
    a.z = (const uint16_t *)z;
    a.ldz = ldz;
    a.out = (uint16_t *)dz;
    a.ldo = lddz;
    a.pos = pos;
    a.w = w;
    a.dw = dw;
    a.T = T;
    a.rows = rows;
    a.H = desc->hidden;
    a.k = desc->top_k;
    return hip_status(launch_spread(desc->act_dtype == MOE_EXL3_DT_BF16, a, (hipStream_t)stream));
}

int moe_exl3_dropout(int32_t dtype, const void *x, int64_t ldx, const void *residual, int64_t ldr,
                     const moe_exl3_drop *drop, int64_t rows, int64_t cols, void *y, int64_t ldy, void *stream)
{
    if (dtype != MOE_EXL3_DT_F32 && check_dtype(dtype))
        return MOE_EXL3_ERR_UNSUPPORTED;
    if (rows < 0 || cols < 0 || !drop)
        return MOE_EXL3_ERR_INVALID_ARG;
    DropoutArgs a{};
    int rc = check_drop(drop, a.drop);
    if (rc)
        return rc;
    if (rows == 0 || cols == 0)
        return MOE_EXL3_OK;
    if (cols > kMaxLd)
        return MOE_EXL3_ERR_UNSUPPORTED;
    const int64_t size = dtype == MOE_EXL3_DT_F32 ? 4 : 2;
    const Mat mx{x, rows, cols, ldx, size}, mr{residual, residual ? rows : 0, cols, ldr, size}, mo{y, rows, cols, ldy, size};
    for (const int r : {check_mat(mx, kNoLimit, 1), check_mat(mr, kNoLimit, 1), check_mat(mo, kNoLimit, 1)})
        if (r)
            return r;
    if (cdiv(rows * cdiv(cols, 8), 256) > INT32_MAX)
        return MOE_EXL3_ERR_UNSUPPORTED;
    // y may be x or the residual itself
    const Span rng{a.drop.rng, 16};
    if (meets(mo, &mx, 1, &rng, 1, 0) || meets(mo, &mr, 1, nullptr, 0, 0))
        return MOE_EXL3_ERR_INVALID_ARG;
    a.x = x;
    a.residual = residual;
    a.y = y;
    a.ldx = ldx;
    a.ldr = ldr;
    a.ldy = ldy;
    a.rows = rows;
    a.cols = (int)cols;
    return hip_status(launch_dropout(dtype, a, (hipStream_t)stream));
}

}  // extern "C"
