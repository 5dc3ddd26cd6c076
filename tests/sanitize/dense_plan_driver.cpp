// The launches that the dense operators' C entries plan, for a sanitizer build
// of the host code: the kernel launchers are replaced by recorders.  Each line
// of the input is a call (glu T H I | bwd T H I dx dw | lora T K N n r w base),
// its answer one line of launches apart by ';':
//   dense MODE BM ROWTILES COLTILES SPLITS STAGES   (stages of 64 k, uncut)
//   grads BMX TILESX STAGESX BMW TILESW STAGESW DWFIRST
//   skinny MODE T FUSED  |  gluGrad  |  shrink T RANK K
// Workspaces have the advertised size, and every launch's partial tiles have
// to lie inside.
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include <string>

#include "dense.h"

using namespace moe;

namespace {

char *const kBase = (char *)(uintptr_t)0x100000000000u;   // never read
std::string log_;
size_t ws_bytes_;

void *place(int i) { return kBase + ((int64_t)i << 40); }

[[noreturn]] void fail(const char *what)
{
    fprintf(stderr, "check failed: %s after [%s]\n", what, log_.c_str());
    exit(1);
}

template <class... A>
hipError_t note(const char *f, A... a)
{
    char s[256];
    snprintf(s, sizeof s, f, a...);
    log_ += (log_.empty() ? "" : ";") + std::string(s);
    return hipSuccess;
}

int stages(int mode, const DenseArgs &a) { return (mode == DENSE_DX ? 2 : 1) * ((a.K + kDenseK - 1) / kDenseK); }

void check_tiles(int mode, const DenseArgs &a)
{
    const int s = stages(mode, a), cols = mode == DENSE_GLU ? a.bm / 2 : a.bm, tensors = mode == DENSE_DW ? 2 : 1;
    if (a.mt && a.mt != tensors * ((a.M + a.bm - 1) / a.bm))
        fail("row tiles");
    if (a.nt != (a.N + cols - 1) / cols)
        fail("column tiles");
    if (a.splits < 1 || (int64_t)a.splits * a.per < s || (a.splits > 1 && (int64_t)(a.splits - 1) * a.per >= s))
        fail("splits cover k once, none empty");
    if (a.splits == 1)
        return;
    const char *end = (const char *)place(5) + ws_bytes_;
    if (a.bm != kDenseTile || (const char *)a.part < (const char *)place(5) ||
        (const char *)a.part + (int64_t)a.mt * a.nt * a.splits * kDenseTile * kDenseTile * 4 > end)
        fail("partial tiles inside the workspace");
}

}  // namespace

namespace moe {

hipError_t launch_dense(int mode, bool, const DenseArgs &a, hipStream_t)
{
    check_tiles(mode, a);
    return note("dense %d %d %d %d %d %d", mode, a.bm, a.mt, a.nt, a.splits, stages(mode, a));
}

hipError_t launch_dense_grads(bool, const DenseArgs &x, const DenseArgs &w, bool dw_first, hipStream_t)
{
    check_tiles(DENSE_DX, x);
    check_tiles(DENSE_DW, w);
    if (x.splits != 1 || w.splits != 1 || x.bm != kDenseTile)
        fail("tiles of a launch of both gradients");
    return note("grads %d %d %d %d %d %d %d", x.bm, x.mt * x.nt, stages(DENSE_DX, x), w.bm, w.mt * w.nt,
                stages(DENSE_DW, w), (int)dw_first);
}

hipError_t launch_dense_skinny(int mode, bool, const DenseArgs &a, hipStream_t)
{
    if (a.M > kSkinnyTokens)
        fail("tokens of the few-token kernel");
    return note("skinny %d %d %d", mode, a.M, (int)(mode == DENSE_LIN && a.lora.fused));
}

hipError_t launch_glu_grad(bool, int, const float *, const uint16_t *, int64_t, int64_t, int, uint16_t *, uint16_t *,
                           hipStream_t)
{
    return note("%s", "gluGrad");
}

hipError_t launch_lora_shrink(bool, const uint16_t *, int64_t, uint32_t, int64_t T, int K, const LoraArgs &l, hipStream_t)
{
    return note("shrink %d %d %d", (int)T, l.rank, K);
}

}  // namespace moe

int main()
{
    char line[256];
    while (fgets(line, sizeof line, stdin)) {
        char op[16];
        long long v[7] = {};
        sscanf(line, "%15s %lld %lld %lld %lld %lld %lld %lld", op, &v[0], &v[1], &v[2], &v[3], &v[4], &v[5], &v[6]);
        const int64_t T = v[0], A = v[1], B = v[2];
        int rc;
        log_.clear();
        size_t need = 0;
        if (!strcmp(op, "lora")) {
            const moe_exl3_lora_desc d = {(int32_t)A, (int32_t)B, (int32_t)v[3], (int32_t)v[4], MOE_EXL3_DT_BF16};
            const moe_exl3_lora_adapters ad = {place(1), place(2), nullptr, nullptr};
            rc = moe_exl3_lora_workspace_size(&d, T, &need);
            ws_bytes_ = need;
            if (!rc)
                rc = moe_exl3_lora_linear(&d, place(0), A, v[5] ? place(3) : nullptr, &ad, (int32_t *)place(6),
                                          v[6] ? place(7) : nullptr, B, T, place(4), B, place(5), need, nullptr);
        } else {
            const moe_exl3_glu_desc d = {(int32_t)A, (int32_t)B, MOE_EXL3_DT_BF16, MOE_EXL3_ACT_SILU};
            const bool back = !strcmp(op, "bwd");
            rc = back ? moe_exl3_glu_backward_workspace_size(&d, T, &need) : moe_exl3_glu_workspace_size(&d, T, &need);
            ws_bytes_ = need;
            if (!rc && !back)
                rc = moe_exl3_glu(&d, place(0), A, place(1), place(2), T, place(3), B, nullptr, place(5), need, nullptr);
            else if (!rc)
                rc = moe_exl3_glu_backward(&d, place(0), A, place(1), place(2), (float *)place(4), place(3), B, T,
                                           v[3] ? place(6) : nullptr, A, v[4] ? place(7) : nullptr,
                                           v[4] ? place(8) : nullptr, place(5), need, nullptr);
        }
        if (rc)
            printf("error %d\n", rc);
        else
            printf("%s\n", log_.c_str());
    }
    return 0;
}
