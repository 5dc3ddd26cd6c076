// Host side of the dense operators: argument checks, workspace plans, launch
// sequences.  Declarations and the full contract are in include/moe_exl3.h.
#include "dense.h"

#include <algorithm>
#include <cmath>

using namespace moe;

namespace {

constexpr size_t kAlign = 256;
constexpr int64_t kMaxSize = 65536;
constexpr int64_t kMaxLd = 1 << 20;
constexpr int64_t kSpanLimit = (int64_t)1 << 31;

// k splits of 64 x 64 tiles: at most this many blocks (one a CU), and at most one
// for each this many stages (256 k; the last split takes what is left).
constexpr int64_t kSplitBlocks = 256;
constexpr int64_t kSplitStages = 4;
// Adapters that a call is taken to name at most (plan_tiles).
constexpr int64_t kMostNamed = 64;

size_t align_up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }
int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

template <class T>
T *at(void *ws, size_t off)
{
    return (T *)((char *)ws + off);
}

// A row-major 16-bit matrix argument.
struct Mat {
    const void *p;
    int64_t rows, cols, ld;
    int64_t span() const { return rows > 0 ? ((rows - 1) * ld + cols) * 2 : 0; }
};

// The rules of one matrix: address, row stride, extent.
int check_mat(const Mat &m)
{
    if (m.rows == 0)
        return MOE_EXL3_OK;
    if (!m.p || m.ld < m.cols)
        return MOE_EXL3_ERR_INVALID_ARG;
    if (m.ld > kMaxLd)
        return MOE_EXL3_ERR_UNSUPPORTED;
    if (!aligned16(m.p) || m.ld % 8)
        return MOE_EXL3_ERR_MISALIGNED;
    if (m.rows > kSpanLimit || m.span() >= kSpanLimit)
        return MOE_EXL3_ERR_UNSUPPORTED;
    return MOE_EXL3_OK;
}

bool spans_meet(const void *a, int64_t an, const void *b, int64_t bn)
{
    return an > 0 && bn > 0 && (uintptr_t)a < (uintptr_t)b + (uint64_t)bn && (uintptr_t)b < (uintptr_t)a + (uint64_t)an;
}

// Whether two matrices share an element: their spans meet, unless they are
// column ranges apart of one buffer (same ld).
bool overlap(const Mat &a, const Mat &b)
{
    if (!a.p || !b.p || !spans_meet(a.p, a.span(), b.p, b.span()))
        return false;
    if (a.ld != b.ld)
        return true;
    const int64_t d = ((intptr_t)b.p - (intptr_t)a.p) / 2;
    const int64_t r = ((d % a.ld) + a.ld) % a.ld;   // b's first column, from a's
    return !(r >= a.cols && r + b.cols <= a.ld);
}

int check_dtype(int dt)
{
    return dt == MOE_EXL3_DT_F16 || dt == MOE_EXL3_DT_BF16 ? MOE_EXL3_OK : MOE_EXL3_ERR_UNSUPPORTED;
}

int check_size(int64_t v)
{
    if (v <= 0 || v % 8)
        return MOE_EXL3_ERR_INVALID_ARG;
    return v > kMaxSize ? MOE_EXL3_ERR_UNSUPPORTED : MOE_EXL3_OK;
}

int check_desc(const moe_exl3_glu_desc *d)
{
    if (!d)
        return MOE_EXL3_ERR_INVALID_ARG;
    for (const int rc : {check_size(d->hidden), check_size(d->inter), check_dtype(d->act_dtype)})
        if (rc)
            return rc;
    if (d->act != MOE_EXL3_ACT_SILU && d->act != MOE_EXL3_ACT_GELU_TANH)
        return MOE_EXL3_ERR_UNSUPPORTED;
    return (int64_t)d->hidden * d->inter * 2 >= kSpanLimit ? MOE_EXL3_ERR_UNSUPPORTED : MOE_EXL3_OK;
}

int check_desc(const moe_exl3_lora_desc *d)
{
    if (!d || d->n_adapters <= 0)
        return MOE_EXL3_ERR_INVALID_ARG;
    for (const int rc : {check_size(d->n_in), check_size(d->n_out), check_size(d->rank), check_dtype(d->act_dtype)})
        if (rc)
            return rc;
    if (d->rank > kMaxRank || d->n_adapters > kMaxSize)
        return MOE_EXL3_ERR_UNSUPPORTED;
    return (int64_t)d->n_in * d->n_out * 2 >= kSpanLimit ? MOE_EXL3_ERR_UNSUPPORTED : MOE_EXL3_OK;
}

// T tokens of contiguous rows of this length must be addressable.
bool rows_fit(int64_t T, int64_t cols) { return T < kSpanLimit && T * cols * 2 < kSpanLimit; }

// Columns of a tile of `bm` rows.
int64_t tile_cols(int mode, int64_t bm) { return mode == DENSE_GLU ? bm / 2 : bm; }

int64_t stages_of(int mode, int64_t K) { return (mode == DENSE_DX ? 2 : 1) * cdiv(K, kDenseK); }

int64_t tiles_of(int mode, int64_t M, int64_t N, int64_t bm)
{
    return (mode == DENSE_DW ? 2 : 1) * cdiv(M, bm) * cdiv(N, tile_cols(mode, bm));
}

// Tiles and k splits of a launch.
struct Tiles {
    int64_t bm, mt, nt, splits, per;
    double us;   // estimate
};

// The tile of a launch: the one whose rounds over the 256 CUs are estimated to
// take the least time.  A round costs a fixed part (launch, first loads,
// epilogue) and a part per 64 k, in us as fitted to the block's forward pass, 96
// to 16384 tokens, hidden 512 to 8192, inter 256 to 8192 (calls one after the
// other; the figures behind are the present kernels'):
//   64 x 64     5 + 0.16 for 64 k up to 256 tiles, else 5.4 + 0.34 a round of 512
//               (333 tokens, 1032 x 1384: 10.9; 128 x 128 takes 14.8)
//   128 x 128   4 + 0.48 (1024 tokens, 4096 x 2048: 38; 64 x 64 takes 52,
//               256 x 256 79)
//   256 x 256   10 + 1.40 (4096 tokens, 4096 x 2048: 104; 128 x 128 takes 116)
// Few 64 x 64 tiles with a long k are cut along k, at the price of partial tiles
// and a second launch: 11 + 0.16 for 64 k + 0.1 a split, into as many as make that
// least (calls of 100 tokens, 8192 x 256: 12.5, uncut 24; 4096 x 512: 11.5, uncut
// 14.9; but 200 tokens, 2048 x 1024: 10.3 uncut, 12.1 cut).
// The estimates are there to order the tiles, which they did in each of 17 sizes
// timed in all three; the times themselves can be half as long again, most where
// rows do not begin on a 128-byte line, which has no term (198 tokens, 7528 x
// 6144, 128 x 128: 61 estimated, 94 measured; 64 x 64 takes 103).
//
// An adapter that a tile's tokens name costs 0.6 us for 64 ranks in a 128 x 128
// tile, twice that in a 256 x 256 one; the wavefronts of a 64 x 64 tile share them,
// and so do its splits (116 tokens, 62 adapters of 32, 1984 columns, 840 k: a call
// of 60 us in 128 x 128, 21 in 64 x 64).  Of n adapters a tile of bm tokens is taken
// to name n bm / T and one more, the tokens of a request standing together.  The
// host does not see the ids: n is the stack's length, but no more than kMostNamed,
// as a longer stack says nothing about a call (one request's 7168 tokens, 2048 x
// 4096, rank 32: 113 us with 8 adapters loaded, 199 with 3000 before this limit, 114
// with it).  A fixed number for stacks of any length takes 1 to 2% less over 200
// calls of 1 to 63 named adapters, but up to 1.8 times as long: 16, 219 tokens of
// 51 adapters 31 -> 57 us; 64, 324 tokens of 5 adapters 16 -> 24.
//
// n, rank: of the adapters, 0 without any.
Tiles plan_tiles(int mode, int64_t M, int64_t N, int64_t K, int64_t n = 0, int64_t rank = 0)
{
    const int64_t stages = stages_of(mode, K);
    const double s = (double)stages;
    int64_t bm = 0, cuts = 1;
    double least = 0;
    auto offer = [&](int64_t b, int64_t c, double us) {
        if (bm == 0 || us < least) {
            bm = b;
            cuts = c;
            least = us;
        }
    };
    auto rounds = [&](int64_t tiles, int64_t at_once) { return (double)cdiv(tiles, at_once); };
    auto adapters = [&](int64_t b) {
        return n == 0 ? 0.0 : 0.6 * (double)(std::min({n, b, cdiv(n * b, M) + 1}) * cdiv(rank, 64));
    };
    const double l64 = adapters(kDenseTile), l128 = adapters(kDenseSmall), l256 = 2 * adapters(kDenseLarge);
    const int64_t t64 = tiles_of(mode, M, N, kDenseTile), t128 = tiles_of(mode, M, N, kDenseSmall);
    offer(kDenseLarge, 1, rounds(tiles_of(mode, M, N, kDenseLarge), 256) * (10 + 1.40 * s + l256));
    offer(kDenseSmall, 1, rounds(t128, 256) * (4 + 0.48 * s + l128));
    offer(kDenseTile, 1, t64 <= 256 ? 5 + 0.16 * s + l64 / 4 : rounds(t64, 512) * (5.4 + 0.34 * s + l64 / 2));
    const int64_t most = t64 > 0 ? std::min(kSplitBlocks / t64, stages / kSplitStages) : 0;
    const int64_t c = std::min(most, std::max<int64_t>(2, (int64_t)std::sqrt((0.16 * s + l64) / 0.1)));
    if (c > 1)
        offer(kDenseTile, c, 11 + 0.16 * (double)cdiv(stages, c) + l64 / (double)c + 0.1 * (double)c);
    Tiles t{};
    t.bm = bm;
    t.mt = (mode == DENSE_DW ? 2 : 1) * cdiv(M, bm);
    t.nt = cdiv(N, tile_cols(mode, bm));
    t.per = std::max<int64_t>(1, cdiv(stages, cuts));
    t.splits = std::max<int64_t>(1, cdiv(stages, t.per));
    t.us = least;
    return t;
}

// The same in tiles of one size, whatever they cost, k uncut; us: one block.
Tiles plan_fixed(int mode, int64_t M, int64_t N, int64_t K, int64_t bm)
{
    Tiles t{};
    t.bm = bm;
    t.mt = (mode == DENSE_DW ? 2 : 1) * cdiv(M, bm);
    t.nt = cdiv(N, tile_cols(mode, bm));
    t.per = std::max<int64_t>(1, stages_of(mode, K));
    t.splits = 1;
    t.us = bm == kDenseTile ? 5 + 0.16 * (double)t.per : 4 + 0.48 * (double)t.per;
    return t;
}

// Both kinds' blocks over the 256 CUs.
double merged_sum(const Tiles &a, const Tiles &b)
{
    return ((double)(a.mt * a.nt) * a.us + (double)(b.mt * b.nt) * b.us) / 256;
}

// Whether both kinds of such blocks take less time in one launch, two blocks on
// a CU: three quarters of the sum, at least the longest block, which its
// neighbour slows down.  Whole steps, in one launch and in two, in us: 250 tokens,
// 2048 x 2048: 33.5, 41.5; 1908, 1000 x 1376: 67, 75; 30, 8192 x 2048: 54, 66;
// but with long blocks 128, 1536 x 4096: 44, 40; 60, 1664 x 5816: 64, 51.  Beyond
// a sum of 80 us each gradient fills the CUs by itself, in larger tiles: 3000
// tokens, 2056 x 2056: 256, 218 (9000, 1024 x 1024: 196 both ways).
bool merge_pays(const Tiles &a, const Tiles &b, double apart)
{
    const double sum = merged_sum(a, b);
    return sum <= 80 && std::max(1.3 * std::max(a.us, b.us), 0.75 * sum) < apart;
}

// Bytes of partial tiles that any launch of at most this size can need
// (tiles x splits never exceeds kSplitBlocks or tiles x stages / kSplitStages).
size_t part_bound(int mode, int64_t M, int64_t N, int64_t K)
{
    const int64_t tiles = tiles_of(mode, M, N, kDenseTile), most = stages_of(mode, K) / kSplitStages;
    if (most <= 1 || tiles == 0)
        return 0;
    const int64_t blocks = tiles > kSplitBlocks ? kSplitBlocks : std::min(kSplitBlocks, tiles * most);
    return (size_t)blocks * kDenseTile * kDenseTile * sizeof(float);
}

void set_tiles(DenseArgs &a, const Tiles &t, void *part)
{
    a.bm = (int)t.bm;
    a.mt = (int)t.mt;
    a.nt = (int)t.nt;
    a.splits = (int)t.splits;
    a.per = (int)t.per;
    a.part = (float *)part;
}

// GLU or LIN: few tokens stream the weights through the few-token kernel.
int launch_forward(int mode, int dtype, DenseArgs &a, float *part, void *stream)
{
    const bool bf16 = dtype == MOE_EXL3_DT_BF16;
    hipError_t e;
    if (a.M <= kSkinnyTokens) {
        e = launch_dense_skinny(mode, bf16, a, (hipStream_t)stream);
    } else {
        set_tiles(a, plan_tiles(mode, a.M, a.N, a.K, std::min<int64_t>(a.lora.n, kMostNamed), a.lora.rank), part);
        e = launch_dense(mode, bf16, a, (hipStream_t)stream);
    }
    return e == hipSuccess ? MOE_EXL3_OK : MOE_EXL3_ERR_HIP;
}

struct GluPlan {
    size_t dg, du, part, total;
};

GluPlan plan_glu(const moe_exl3_glu_desc &d, int64_t T)
{
    GluPlan p{};
    p.part = kAlign;
    p.total = p.part + (T <= kSkinnyTokens ? 0 : align_up(part_bound(DENSE_GLU, T, d.inter, d.hidden)));
    return p;
}

GluPlan plan_glu_backward(const moe_exl3_glu_desc &d, int64_t T)
{
    GluPlan p{};
    size_t o = kAlign;
    p.dg = o;
    o += align_up((size_t)T * d.inter * 2);
    p.du = o;
    o += align_up((size_t)T * d.inter * 2);
    p.part = o;
    o += align_up(std::max(part_bound(DENSE_DX, T, d.hidden, d.inter), part_bound(DENSE_DW, d.inter, d.hidden, T)));
    p.total = o;
    return p;
}

struct LoraPlan {
    size_t mid, part, total;
    int rpad;
};

LoraPlan plan_lora(const moe_exl3_lora_desc &d, int64_t T)
{
    LoraPlan p{};
    p.rpad = (int)cdiv(d.rank, 32) * 32;
    size_t o = kAlign;
    p.mid = o;
    // fp32 for the few-token kernel, 16 bits for more tokens: never less than for
    // fewer of them
    o += align_up((size_t)p.rpad * (size_t)std::max(4 * std::min(T, kSkinnyTokens), 2 * T));
    p.part = o;
    o += T <= kSkinnyTokens ? 0 : align_up(part_bound(DENSE_LIN, T, d.n_out, d.n_in));
    p.total = o;
    return p;
}

int check_ws(const void *ws, size_t have, size_t need)
{
    if (!ws)
        return MOE_EXL3_ERR_INVALID_ARG;
    if ((uintptr_t)ws % kAlign)
        return MOE_EXL3_ERR_MISALIGNED;
    return have < need ? MOE_EXL3_ERR_WORKSPACE : MOE_EXL3_OK;
}

}  // namespace

extern "C" {

int moe_exl3_glu_workspace_size(const moe_exl3_glu_desc *desc, int64_t max_tokens, size_t *bytes)
{
    const int rc = check_desc(desc);
    if (rc)
        return rc;
    if (!bytes || max_tokens < 0)
        return MOE_EXL3_ERR_INVALID_ARG;
    if (!rows_fit(max_tokens, desc->hidden) || !rows_fit(max_tokens, desc->inter))
        return MOE_EXL3_ERR_UNSUPPORTED;
    *bytes = plan_glu(*desc, max_tokens).total;
    return MOE_EXL3_OK;
}

int moe_exl3_glu_backward_workspace_size(const moe_exl3_glu_desc *desc, int64_t max_tokens, size_t *bytes)
{
    const int rc = check_desc(desc);
    if (rc)
        return rc;
    if (!bytes || max_tokens < 0)
        return MOE_EXL3_ERR_INVALID_ARG;
    if (!rows_fit(max_tokens, desc->hidden) || !rows_fit(max_tokens, desc->inter))
        return MOE_EXL3_ERR_UNSUPPORTED;
    *bytes = plan_glu_backward(*desc, max_tokens).total;
    return MOE_EXL3_OK;
}

int moe_exl3_lora_workspace_size(const moe_exl3_lora_desc *desc, int64_t max_tokens, size_t *bytes)
{
    const int rc = check_desc(desc);
    if (rc)
        return rc;
    if (!bytes || max_tokens < 0)
        return MOE_EXL3_ERR_INVALID_ARG;
    if (!rows_fit(max_tokens, desc->n_in) || !rows_fit(max_tokens, desc->n_out) || !rows_fit(max_tokens, kMaxRank))
        return MOE_EXL3_ERR_UNSUPPORTED;
    *bytes = plan_lora(*desc, max_tokens).total;
    return MOE_EXL3_OK;
}

int moe_exl3_glu(const moe_exl3_glu_desc *desc, const void *x, int64_t ldx, const void *w_gate, const void *w_up,
                 int64_t T, void *out, int64_t ldo, float *pre, void *workspace, size_t ws_bytes, void *stream)
{
    int rc = check_desc(desc);
    if (rc)
        return rc;
    if (T < 0)
        return MOE_EXL3_ERR_INVALID_ARG;
    if (T == 0)
        return MOE_EXL3_OK;
    const int64_t H = desc->hidden, I = desc->inter;
    const Mat mx{x, T, H, ldx}, mg{w_gate, I, H, H}, mu{w_up, I, H, H}, mo{out, T, I, ldo};
    for (const Mat &m : {mx, mg, mu, mo})
        if ((rc = check_mat(m)))
            return rc;
    if (!rows_fit(T, H) || !rows_fit(T, I))
        return MOE_EXL3_ERR_UNSUPPORTED;
    if (pre && !aligned16(pre))
        return MOE_EXL3_ERR_MISALIGNED;
    for (const Mat &m : {mx, mg, mu})
        if (overlap(mo, m) || (pre && spans_meet(pre, 8 * T * I, m.p, m.span())))
            return MOE_EXL3_ERR_INVALID_ARG;
    if (pre && spans_meet(pre, 8 * T * I, out, mo.span()))
        return MOE_EXL3_ERR_INVALID_ARG;
    const GluPlan p = plan_glu(*desc, T);
    if ((rc = check_ws(workspace, ws_bytes, p.total)))
        return rc;
    DenseArgs a{};
    a.p[0] = (const uint16_t *)x;
    a.q[0] = (const uint16_t *)w_gate;
    a.q[1] = (const uint16_t *)w_up;
    a.ldp = ldx;
    a.ldq = H;
    a.pbytes = (uint32_t)mx.span();
    a.qbytes = (uint32_t)mg.span();
    a.M = (int)T;
    a.N = (int)I;
    a.K = (int)H;
    a.out[0] = (uint16_t *)out;
    a.ldo = ldo;
    a.pre = pre;
    a.act = desc->act;
    return launch_forward(DENSE_GLU, desc->act_dtype, a, at<float>(workspace, p.part), stream);
}

int moe_exl3_glu_backward(const moe_exl3_glu_desc *desc, const void *x, int64_t ldx, const void *w_gate,
                          const void *w_up, const float *pre, const void *dout, int64_t lddo, int64_t T, void *dx,
                          int64_t lddx, void *dw_gate, void *dw_up, void *workspace, size_t ws_bytes, void *stream)
{
    int rc = check_desc(desc);
    if (rc)
        return rc;
    // (no gradient asked for: a mistake, but for no tokens, whose dx has no
    // elements and maybe no address)
    if (T < 0 || !dw_gate != !dw_up || (T > 0 && !dx && !dw_gate))
        return MOE_EXL3_ERR_INVALID_ARG;
    const int64_t H = desc->hidden, I = desc->inter;
    const int64_t wrows = dx ? I : 0;   // the weights are read for dx alone
    const Mat mx{x, T, H, ldx}, mg{w_gate, wrows, H, H}, mu{w_up, wrows, H, H}, mo{dout, T, I, lddo};
    const Mat mdx{dx, dx ? T : 0, H, lddx}, mdg{dw_gate, dw_gate ? I : 0, H, H}, mdu{dw_up, dw_up ? I : 0, H, H};
    for (const Mat &m : {mx, mg, mu, mo, mdx, mdg, mdu})
        if ((rc = check_mat(m)))
            return rc;
    if (!rows_fit(T, H) || !rows_fit(T, I))
        return MOE_EXL3_ERR_UNSUPPORTED;
    if (T > 0) {
        if (!pre)
            return MOE_EXL3_ERR_INVALID_ARG;
        if (!aligned16(pre))
            return MOE_EXL3_ERR_MISALIGNED;
    }
    for (const Mat &o : {mdx, mdg, mdu}) {
        for (const Mat &m : {mx, mg, mu, mo})
            if (overlap(o, m))
                return MOE_EXL3_ERR_INVALID_ARG;
        if (pre && o.p && spans_meet(pre, 8 * T * I, o.p, o.span()))
            return MOE_EXL3_ERR_INVALID_ARG;
    }
    if (overlap(mdx, mdg) || overlap(mdx, mdu) || overlap(mdg, mdu))
        return MOE_EXL3_ERR_INVALID_ARG;
    const GluPlan p = plan_glu_backward(*desc, T);
    if ((rc = check_ws(workspace, ws_bytes, p.total)))
        return rc;
    const bool bf16 = desc->act_dtype == MOE_EXL3_DT_BF16;
    hipStream_t s = (hipStream_t)stream;
    uint16_t *dg = at<uint16_t>(workspace, p.dg), *du = at<uint16_t>(workspace, p.du);
    if (T > 0 && launch_glu_grad(bf16, desc->act, pre, (const uint16_t *)dout, lddo, T, (int)I, dg, du, s) != hipSuccess)
        return MOE_EXL3_ERR_HIP;
    DenseArgs ax{}, aw{};
    ax.p[0] = aw.p[0] = dg;
    ax.p[1] = aw.p[1] = du;
    ax.ldp = aw.ldp = I;
    ax.pbytes = aw.pbytes = (uint32_t)(T * I * 2);
    ax.q[0] = (const uint16_t *)w_gate;
    ax.q[1] = (const uint16_t *)w_up;
    ax.ldq = H;
    ax.qbytes = (uint32_t)mg.span();
    ax.M = (int)T;
    ax.N = (int)H;
    ax.K = (int)I;
    ax.out[0] = (uint16_t *)dx;
    ax.ldo = lddx;
    aw.q[0] = (const uint16_t *)x;
    aw.ldq = ldx;
    aw.qbytes = (uint32_t)mx.span();
    aw.M = (int)I;
    aw.N = (int)H;
    aw.K = (int)T;
    aw.out[0] = (uint16_t *)dw_gate;
    aw.out[1] = (uint16_t *)dw_up;
    aw.ldo = H;
    float *part = at<float>(workspace, p.part);
    const bool want_dx = dx && T > 0, want_dw = dw_gate;
    // Small gradients leave CUs idle on their own: their tiles share one launch,
    // dx in 64 x 64 ones, dw in the better of two.
    // The choice is the same where only one is wanted, and so are its bits.
    const Tiles tx = plan_tiles(DENSE_DX, T, H, I), tw = plan_tiles(DENSE_DW, I, H, T);
    const Tiles sx = plan_fixed(DENSE_DX, T, H, I, kDenseTile);
    Tiles sw = plan_fixed(DENSE_DW, I, H, T, kDenseTile);
    const Tiles lw = plan_fixed(DENSE_DW, I, H, T, kDenseSmall);
    if (std::max(lw.us, merged_sum(sx, lw)) < std::max(sw.us, merged_sum(sx, sw)))
        sw = lw;
    if (T > 0 && merge_pays(sx, sw, tx.us + tw.us)) {
        set_tiles(ax, sx, part);
        set_tiles(aw, sw, part);
        if (!want_dx)
            ax.mt = 0;
        if (!want_dw)
            aw.mt = 0;
        return launch_dense_grads(bf16, ax, aw, sw.us > sx.us, s) == hipSuccess ? MOE_EXL3_OK : MOE_EXL3_ERR_HIP;
    }
    if (want_dx) {
        set_tiles(ax, tx, part);
        if (launch_dense(DENSE_DX, bf16, ax, s) != hipSuccess)
            return MOE_EXL3_ERR_HIP;
    }
    if (want_dw) {
        set_tiles(aw, tw, part);
        if (launch_dense(DENSE_DW, bf16, aw, s) != hipSuccess)
            return MOE_EXL3_ERR_HIP;
    }
    return MOE_EXL3_OK;
}

int moe_exl3_lora_linear(const moe_exl3_lora_desc *desc, const void *x, int64_t ldx, const void *w,
                         const moe_exl3_lora_adapters *adapters, const int32_t *ids, const void *base, int64_t ldbase,
                         int64_t T, void *y, int64_t ldy, void *workspace, size_t ws_bytes, void *stream)
{
    int rc = check_desc(desc);
    if (rc)
        return rc;
    if (T < 0)
        return MOE_EXL3_ERR_INVALID_ARG;
    if (T == 0)
        return MOE_EXL3_OK;
    if (!adapters || !adapters->a || !adapters->b || !ids)
        return MOE_EXL3_ERR_INVALID_ARG;
    const int64_t K = desc->n_in, N = desc->n_out, n = desc->n_adapters, r = desc->rank;
    const Mat mx{x, T, K, ldx}, mw{w, w ? N : 0, K, K}, mb{base, base ? T : 0, N, ldbase}, my{y, T, N, ldy};
    for (const Mat &m : {mx, mw, mb, my})
        if ((rc = check_mat(m)))
            return rc;
    if (!rows_fit(T, K) || !rows_fit(T, N) || !rows_fit(T, kMaxRank))
        return MOE_EXL3_ERR_UNSUPPORTED;
    if (!aligned16(adapters->a) || !aligned16(adapters->b))
        return MOE_EXL3_ERR_MISALIGNED;
    for (const void *q : {(const void *)adapters->scales, (const void *)adapters->ranks, (const void *)ids})
        if ((uintptr_t)q & 3u)
            return MOE_EXL3_ERR_MISALIGNED;
    if (overlap(my, mx) || overlap(my, mw) || (overlap(my, mb) && !(base == y && ldbase == ldy)) ||
        spans_meet(y, my.span(), adapters->a, 2 * n * r * K) || spans_meet(y, my.span(), adapters->b, 2 * n * r * N) ||
        spans_meet(y, my.span(), ids, 4 * T) || spans_meet(y, my.span(), adapters->scales, adapters->scales ? 4 * n : 0) ||
        spans_meet(y, my.span(), adapters->ranks, adapters->ranks ? 4 * n : 0))
        return MOE_EXL3_ERR_INVALID_ARG;
    const LoraPlan p = plan_lora(*desc, T);
    if ((rc = check_ws(workspace, ws_bytes, p.total)))
        return rc;
    const bool bf16 = desc->act_dtype == MOE_EXL3_DT_BF16;
    hipStream_t s = (hipStream_t)stream;
    DenseArgs a{};
    LoraArgs &l = a.lora;
    l.a = (const uint16_t *)adapters->a;
    l.b = (const uint16_t *)adapters->b;
    l.ids = ids;
    l.scales = adapters->scales;
    l.ranks = adapters->ranks;
    l.status = at<int32_t>(workspace, MOE_EXL3_STATUS_OFFSET);
    l.mid = at<void>(workspace, p.mid);
    l.n = (int)n;
    l.rank = (int)r;
    l.rpad = p.rpad;
    l.k = (int)K;
    l.fused = T == 1 && r <= kFusedRank && r * K * 2 <= kFusedBytes && N <= kFusedCols;
    if (!l.fused &&
        launch_lora_shrink(bf16, (const uint16_t *)x, ldx, (uint32_t)mx.span(), T, (int)K, l, s) != hipSuccess)
        return MOE_EXL3_ERR_HIP;
    a.p[0] = (const uint16_t *)x;
    a.q[0] = (const uint16_t *)w;
    a.ldp = ldx;
    a.ldq = K;
    a.pbytes = (uint32_t)mx.span();
    a.qbytes = (uint32_t)mw.span();
    a.M = (int)T;
    a.N = (int)N;
    a.K = w ? (int)K : 0;   // without a projection the tiles start from zero
    a.out[0] = (uint16_t *)y;
    a.ldo = ldy;
    a.base = (const uint16_t *)base;
    a.ldbase = ldbase;
    return launch_forward(DENSE_LIN, desc->act_dtype, a, at<float>(workspace, p.part), stream);
}

}  // extern "C"
