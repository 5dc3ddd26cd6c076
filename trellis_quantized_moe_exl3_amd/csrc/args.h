// Argument checks and sizes shared by the host entry points of the operators
// beside the layer.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "moe_exl3.h"

namespace moe {

constexpr size_t kAlign = 256;
constexpr int64_t kMaxSize = 65536;
constexpr int64_t kMaxLd = 1 << 20;
constexpr int64_t kSpanLimit = (int64_t)1 << 31;

inline size_t align_up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }
inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

template <class T>
T *at(void *ws, size_t off)
{
    return (T *)((char *)ws + off);
}

// A row-major matrix argument, of 16-bit elements where nothing else is said.
struct Mat {
    const void *p;
    int64_t rows, cols, ld;
    int64_t size = 2;   // bytes of an element
    int64_t span() const { return rows > 0 ? ((rows - 1) * ld + cols) * size : 0; }
};

constexpr int64_t kNoLimit = INT64_MAX;

// The rules of one matrix: address, row stride (a multiple of `step` elements),
// extent.
inline int check_mat(const Mat &m, int64_t limit = kSpanLimit, int64_t step = 8)
{
    if (m.rows == 0)
        return MOE_EXL3_OK;
    if (!m.p || m.ld < m.cols)
        return MOE_EXL3_ERR_INVALID_ARG;
    if (m.ld > kMaxLd)
        return MOE_EXL3_ERR_UNSUPPORTED;
    if (!aligned16(m.p) || m.ld % step)
        return MOE_EXL3_ERR_MISALIGNED;
    if (m.rows > kSpanLimit || m.span() >= limit)
        return MOE_EXL3_ERR_UNSUPPORTED;
    return MOE_EXL3_OK;
}

inline bool spans_meet(const void *a, int64_t an, const void *b, int64_t bn)
{
    return an > 0 && bn > 0 && (uintptr_t)a < (uintptr_t)b + (uint64_t)bn && (uintptr_t)b < (uintptr_t)a + (uint64_t)an;
}

// Whether two matrices share an element: their spans meet, unless they are
// column ranges apart of one buffer (same ld).
inline bool overlap(const Mat &a, const Mat &b)
{
    if (!a.p || !b.p || !spans_meet(a.p, a.span(), b.p, b.span()))
        return false;
    if (a.ld != b.ld)
        return true;
    const int64_t d = ((intptr_t)b.p - (intptr_t)a.p) / a.size;
    const int64_t r = ((d % a.ld) + a.ld) % a.ld;   // b's first column, from a's
    return !(r >= a.cols && r + b.cols <= a.ld);
}

inline int check_dtype(int dt)
{
    return dt == MOE_EXL3_DT_F16 || dt == MOE_EXL3_DT_BF16 ? MOE_EXL3_OK : MOE_EXL3_ERR_UNSUPPORTED;
}

inline int check_size(int64_t v)
{
    if (v <= 0 || v % 8)
        return MOE_EXL3_ERR_INVALID_ARG;
    return v > kMaxSize ? MOE_EXL3_ERR_UNSUPPORTED : MOE_EXL3_OK;
}

inline int check_ws(const void *ws, size_t have, size_t need)
{
    if (!ws)
        return MOE_EXL3_ERR_INVALID_ARG;
    if ((uintptr_t)ws % kAlign)
        return MOE_EXL3_ERR_MISALIGNED;
    return have < need ? MOE_EXL3_ERR_WORKSPACE : MOE_EXL3_OK;
}

}  // namespace moe
