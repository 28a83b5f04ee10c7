// C-ABI entry points of the token operators: validation, variant selection,
// launch. Validation finishes before the first launch; nothing here allocates
// device memory or synchronises.
#include <algorithm>
#include <cmath>
#include <cstdio>

#include "igconv.h"
#include "token_ops.h"

namespace {

using namespace igc;

constexpr int64_t kRowsMax = 2147483647;

// Test hook (linear_debug_force): per thread, like the conv hooks.
thread_local int g_force_linear_tile = -1;
thread_local int g_force_linear_splits = 0;

bool aligned(const void *p, int bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }
bool is_code(int t) { return t == IGC_INT8 || t == IGC_FP8_E4M3FN; }
bool is_value(int t) { return t == IGC_BF16 || t == IGC_F32; }

// One operand of a row operator: `ld` elements from row to row.
struct Operand {
    const char *name;
    const void *p;
    int64_t ld, need;
};

int check_rows(const char *fn, int64_t rows, int64_t cols, int64_t max_cols)
{
    if (rows < 0 || rows > kRowsMax)
        return report_error(IGC_ERR_INVALID, "%s: rows = %lld must be in [0, 2^31)", fn, (long long)rows);
    if (cols < 1)
        return report_error(IGC_ERR_INVALID, "%s: cols = %lld must be >= 1", fn, (long long)cols);
    if (cols > max_cols)
        return report_error(IGC_ERR_UNSUPPORTED, "%s: cols = %lld, rows of at most %lld elements are taken",
                            fn, (long long)cols, (long long)max_cols);
    return IGC_OK;
}

int check_operand(const char *fn, const Operand &o)
{
    if (!o.p)
        return report_error(IGC_ERR_INVALID, "%s: null %s", fn, o.name);
    if (o.ld < o.need)
        return report_error(IGC_ERR_INVALID, "%s: row stride of %s is %lld elements, needs at least %lld", fn, o.name,
                            (long long)o.ld, (long long)o.need);
    if (o.ld > (int64_t(1) << 40))
        return report_error(IGC_ERR_INVALID, "%s: row stride of %s is %lld elements, at most 2^40 are taken", fn,
                            o.name, (long long)o.ld);
    if (!aligned(o.p, 16))
        return report_error(IGC_ERR_ALIGN, "%s: %s not 16-byte aligned", fn, o.name);
    return IGC_OK;
}

// Rows of codes: whole 128-code steps, 16-byte aligned.
int check_codes(const char *fn, const Operand &o)
{
    if (int rc = check_operand(fn, o))
        return rc;
    if (o.ld % 16 != 0)
        return report_error(IGC_ERR_INVALID, "%s: row stride of %s is %lld codes, not a multiple of 16", fn, o.name,
                            (long long)o.ld);
    return IGC_OK;
}

int check_scales(const char *fn, const char *name, const float *p)
{
    if (!p)
        return report_error(IGC_ERR_INVALID, "%s: null %s", fn, name);
    if (!aligned(p, 4))
        return report_error(IGC_ERR_ALIGN, "%s: %s not 4-byte aligned", fn, name);
    return IGC_OK;
}

int done(const char *fn, hipError_t e)
{
    if (e != hipSuccess)
        return report_error(IGC_ERR_HIP, "%s: launch failed: %s", fn, hipGetErrorString(e));
    return report_ok();
}

// ------------------------------------------------------------------ linear plan

// Tiles of the linear kernel and what they cost, in us on an MI355X: T = launch +
// rounds * (steps * step + round), rounds = tiles over CUs rounded up, times
// `shared` where two workgroups are resident on a CU and there are two or more.
// Fitted to 600 random shapes (1..8192 tokens, 64..10240 features, 64..8192 codes
// to sum, both types) on every tile: choosing by it is 1.6 % slower than the best
// tile of each shape on average. fp8 codes widened to bf16 (fp32 outputs) cost
// `widened` times as much a step, fitted to 220 more (0.7 % slower than their best).
// Two sets of operands in turn were timed: weights of those shapes, 84 MB at most, come
// from the 256 MB cache. From HBM a few tokens take longer on every tile (1 x 8192 x
// 8192 fp8 14.9 us, 12.8 from the cache; 48 x 8192 x 8192 19.0 and 13.8) and the choice
// is within 3 % of the best tile on those tried but 4 x 8192 x 8192 (16.2 us, 15.4 on
// 16 x 16).
struct TileCost {
    int bn, bm;  // features x tokens
    double step, round, shared, widened;
};
constexpr TileCost kTileCost[kNumLinearTiles] = {
    {256, 256, 1.37, 7.0, 1.0, 1.6},   // LT_256
    {128, 128, 0.52, 1.8, 1.0, 1.9},   // LT_128
    {64, 64, 0.20, 1.1, 0.91, 2.1},    // LT_64
    {32, 64, 0.176, 0.86, 0.80, 1.7},  // LT_32x64
    {32, 32, 0.128, 0.82, 0.74, 1.5},  // LT_32
    {16, 16, 0.29, 0.4, 0.65, 1.25},   // LT_SKINNY: see linear_cost
    {256, 128, 0.74, 4.5, 1.0, 1.5},   // LT_256x128
    {64, 128, 0.29, 1.4, 1.0, 2.1},    // LT_64x128
};
constexpr double kLaunch = 1.7;

// A split reduction's second launch, and the bytes a us its sums are written and read at.
constexpr double kSplitLaunch = 3.5, kSplitRate = 3e6;
constexpr int kMaxSplits = 16;
constexpr int64_t kMaxTiles = (int64_t(1) << 23) - 1;  // of 512 threads: a launch has fewer than 2^32
constexpr size_t kLinearSplitRoom = size_t(64) << 20;  // no split is worth more workspace than this

struct LinearPlan {
    int tile = LT_256;
    int bn = 0, bm = 0;  // features x tokens of a tile
    int tiles_m = 0, tiles_n = 0;
    int nk = 0;
    int group = 8;  // 256 x 256 tiles, 9500 x 10240 x 1280 fp8: 128.3 us, 131.0 with 4, 136.9 with 16
    int splits = 1, ksplit = 0;
    int64_t ws_need = 0;
};

int check_linear(const char *fn, int64_t m, int64_t n, int64_t k, int dtype, int y_dtype)
{
    if (m < 0 || m > kRowsMax - 256)
        return report_error(IGC_ERR_INVALID, "%s: m = %lld must be in [0, 2^31 - 256)", fn, (long long)m);
    if (n < 1 || n > kRowsMax - 256)
        return report_error(IGC_ERR_INVALID, "%s: n = %lld must be in [1, 2^31 - 256)", fn, (long long)n);
    if (k < 1)
        return report_error(IGC_ERR_INVALID, "%s: k = %lld must be >= 1", fn, (long long)k);
    if (!is_code(dtype))
        return report_error(IGC_ERR_INVALID, "%s: dtype %d is neither IGC_INT8 nor IGC_FP8_E4M3FN", fn, dtype);
    if (!is_value(y_dtype))
        return report_error(IGC_ERR_INVALID, "%s: y_dtype %d is neither IGC_BF16 nor IGC_F32", fn, y_dtype);
    if (k > kMaxLinearK)
        return report_error(IGC_ERR_UNSUPPORTED, "%s: k = %lld, at most %lld products keep an int32 sum exact", fn,
                            (long long)k, (long long)kMaxLinearK);
    return IGC_OK;
}

// Cost of `tiles` workgroups of tile t (all splits), each of `steps` steps.
double linear_cost(int t, int64_t m, int64_t tiles, int64_t steps, bool widened, int64_t cus)
{
    const TileCost &c = kTileCost[t];
    const double rounds = (double)((tiles + cus - 1) / cus);
    if (t == LT_SKINNY) {
        // the steps go round the waves; what a workgroup loads for one grows with its tokens
        const double turns = (double)((steps + kSkinnyWaves - 1) / kSkinnyWaves);
        const double rows = (double)(kSkinnyFeatures + std::min<int64_t>(m, kSkinnyTokens)) / 32.0;
        return kLaunch + c.round + turns * (c.step + c.shared * (widened ? c.widened : 1.0) * rounds * rows);
    }
    return kLaunch + (rounds > 1.0 ? rounds * c.shared : 1.0) * ((double)steps * c.step * (widened ? c.widened : 1.0) + c.round);
}

// A few tokens over a large weight: the time is its way from HBM into the CUs, and the
// 16 x 16 workgroups, whose waves wait for no barrier, take it fastest (1 x 12288 x 8192
// fp8 20.1 us, 23.8 us on the best of the other tiles; 1 x 16384 x 8192 25.6 and 32.8; 1 x
// 60000 x 4096 44.7 and 49.0; 4 x 32768 x 8192 49.0 and 55.4), where their waves' rounds of
// loads are nearly full (1 x 30000 x 5120, 40 steps in rounds of 32: 35.4 us, 31.0 us by
// cost) and the tokens' rows are few beside the weight's (16 x 32768 x 8192 68.3 and 55.3
// us). Below 96 MB the costs above choose; 96 MB is where three weights in turn no longer
// fit the 256 MB cache, as they were when this was fitted.
bool streams_weight(int64_t m, int64_t n, int64_t nk)
{
    constexpr int64_t round = kSkinnyWaves * kSkinnyLoads;
    return m <= 4 && n * nk * kCodePad >= int64_t(96) << 20 && 10 * nk >= 9 * ((nk + round - 1) / round * round);
}

// The tile and split of the least cost. A reduction is split only where its tiles
// leave room in one round of the GPU.
int plan_linear(const char *fn, int64_t m, int64_t n, int64_t k, int dtype, int y_dtype, size_t ws_bytes,
                LinearPlan &pl)
{
    const int64_t cus = compute_units(), nk = code_cols(k) / kCodePad;
    const bool widened = dtype == IGC_FP8_E4M3FN && y_dtype == IGC_F32;
    pl.nk = (int)nk;
    double best = 0.0;
    const bool stream = streams_weight(m, n, nk);
    for (int t = 0; t < kNumLinearTiles; ++t) {
        if (g_force_linear_tile >= 0 ? t != g_force_linear_tile : stream && t != LT_SKINNY)
            continue;
        const TileCost &c = kTileCost[t];
        const int64_t tm = (m + c.bm - 1) / c.bm, tn = (n + c.bn - 1) / c.bn;
        if (tm > kMaxTiles / tn)
            continue;
        // beyond two of these workgroups per CU their start and end outweigh the steps (1 x 10240 x 1280, 640 of them:
        // 7.4 us, 6.4 us on 64 x 64 tiles; 6.2 and 5.2 us with the weight in the cache)
        if (t == LT_SKINNY && g_force_linear_tile < 0 && !stream && tm * tn > 2 * cus)
            continue;
        for (int64_t s = 1; s <= (t == LT_SKINNY ? 1 : kMaxSplits); ++s) {
            if (s > 1 && (g_force_linear_splits > 0 ? s > g_force_linear_splits : tm * tn * s > cus))
                break;
            const int64_t ks = (nk + s - 1) / s, splits = (nk + ks - 1) / ks;
            const int64_t need = splits > 1 ? splits * m * n * 4 : 0;
            if (splits != s || need > (int64_t)std::min<size_t>(ws_bytes, kLinearSplitRoom))
                continue;
            double cost = linear_cost(t, m, tm * tn * s, ks, widened, cus);
            if (s > 1)
                cost += kSplitLaunch + (double)need * 2 / kSplitRate;
            if (g_force_linear_splits > 0)  // the most splits that fit, on the tile that is best without any
                cost = linear_cost(t, m, tm * tn, nk, widened, cus) / (double)(1 + s * 1e-3);
            if (best != 0.0 && cost >= best)
                continue;
            best = cost;
            pl.tile = t;
            pl.bn = c.bn;
            pl.bm = c.bm;
            pl.tiles_m = (int)tm;
            pl.tiles_n = (int)tn;
            pl.splits = (int)splits;
            pl.ksplit = (int)ks;
            pl.ws_need = need;
        }
    }
    if (best == 0.0)
        return report_error(IGC_ERR_UNSUPPORTED, "%s: %lld x %lld outputs are too many tiles", fn, (long long)m,
                            (long long)n);
    return IGC_OK;
}

}  // namespace

extern "C" {

int64_t linear_packed_cols(int64_t k)
{
    if (k < 1 || k > kMaxLinearK)
        return report_error(IGC_ERR_INVALID, "linear_packed_cols: k = %lld must be in [1, %lld]", (long long)k,
                            (long long)kMaxLinearK);
    report_ok();
    return code_cols(k);
}

int norm_fwd(const void *x, int64_t ldx, const void *residual, int64_t ldr, const void *weight, void *h, int64_t ldh,
             void *y, int64_t ldy, float *y_scales_dev, int64_t rows, int64_t cols, float eps, int dtype, int y_dtype,
             void *stream)
{
    const char *fn = "norm_fwd";
    if (int rc = check_rows(fn, rows, cols, kMaxNormCols))
        return rc;
    if (!is_value(dtype))
        return report_error(IGC_ERR_INVALID, "%s: dtype %d is neither IGC_BF16 nor IGC_F32", fn, dtype);
    if (y_dtype != dtype && !is_code(y_dtype))
        return report_error(IGC_ERR_INVALID, "%s: y_dtype %d is neither dtype nor IGC_INT8 nor IGC_FP8_E4M3FN", fn,
                            y_dtype);
    if (!(eps >= 0.0f) || std::isinf(eps))
        return report_error(IGC_ERR_INVALID, "%s: eps = %g must be finite and >= 0", fn, eps);
    if (h && !residual)
        return report_error(IGC_ERR_INVALID, "%s: h is x + residual and needs a residual", fn);
    if (rows == 0)
        return report_ok();
    if (int rc = check_operand(fn, {"x", x, ldx, cols}))
        return rc;
    if (int rc = check_operand(fn, {"weight", weight, cols, cols}))
        return rc;
    if (residual)
        if (int rc = check_operand(fn, {"residual", residual, ldr, cols}))
            return rc;
    if (h)
        if (int rc = check_operand(fn, {"h", h, ldh, cols}))
            return rc;
    if (is_code(y_dtype)) {
        if (int rc = check_codes(fn, {"y", y, ldy, code_cols(cols)}))
            return rc;
        if (int rc = check_scales(fn, "y_scales_dev", y_scales_dev))
            return rc;
    } else if (int rc = check_operand(fn, {"y", y, ldy, cols})) {
        return rc;
    }
    const NormParams p{x, residual, weight, h, y, y_scales_dev, ldx, ldr, ldh, ldy, rows, (int)cols, eps};
    return done(fn, launch_norm_fwd(p, (Elem)dtype, (Elem)y_dtype, static_cast<hipStream_t>(stream)));
}

int64_t norm_bwd_workspace_bytes(int64_t rows, int64_t cols)
{
    if (int rc = check_rows("norm_bwd_workspace_bytes", rows, cols, kMaxNormBwdCols))
        return rc;
    report_ok();
    const int64_t cus = compute_units();  // room for either type
    return std::max(norm_bwd_groups(rows, cols, 2, cus), norm_bwd_groups(rows, cols, 4, cus)) * cols * 4;
}

int norm_bwd(const void *dy, int64_t lddy, const void *h, int64_t ldh, const void *weight, const void *dres,
             int64_t lddres, void *dx, int64_t lddx, float *dw, int64_t rows, int64_t cols, float eps, int dtype,
             void *workspace_dev, size_t workspace_bytes, void *stream)
{
    const char *fn = "norm_bwd";
    if (int rc = check_rows(fn, rows, cols, kMaxNormBwdCols))
        return rc;
    if (!is_value(dtype))
        return report_error(IGC_ERR_INVALID, "%s: dtype %d is neither IGC_BF16 nor IGC_F32", fn, dtype);
    if (!(eps >= 0.0f) || std::isinf(eps))
        return report_error(IGC_ERR_INVALID, "%s: eps = %g must be finite and >= 0", fn, eps);
    if (int rc = check_operand(fn, {"weight", weight, cols, cols}))
        return rc;
    if (int rc = check_operand(fn, {"dw", dw, cols, cols}))
        return rc;
    if (rows > 0) {
        if (int rc = check_operand(fn, {"dy", dy, lddy, cols}))
            return rc;
        if (int rc = check_operand(fn, {"h", h, ldh, cols}))
            return rc;
        if (dres)
            if (int rc = check_operand(fn, {"dres", dres, lddres, cols}))
                return rc;
        if (int rc = check_operand(fn, {"dx", dx, lddx, cols}))
            return rc;
    }
    const int64_t cus = compute_units();
    const int groups2 = norm_bwd_groups(rows, cols, 2, cus), groups4 = norm_bwd_groups(rows, cols, 4, cus);
    const int groups = dtype == IGC_BF16 ? groups2 : groups4;
    const size_t need = (size_t)std::max(groups2, groups4) * cols * 4;
    if (!workspace_dev || workspace_bytes < need)
        return report_error(IGC_ERR_INVALID, "%s: needs a workspace of %zu bytes, got %zu", fn, need,
                            workspace_dev ? workspace_bytes : (size_t)0);
    if (!aligned(workspace_dev, 16))
        return report_error(IGC_ERR_ALIGN, "%s: workspace not 16-byte aligned", fn);
    const NormBwdParams p{dy, h, weight, dres, dx, dw, static_cast<float *>(workspace_dev), lddy, ldh, lddres, lddx,
                          rows, (int)cols, eps, groups};
    return done(fn, launch_norm_bwd(p, (Elem)dtype, static_cast<hipStream_t>(stream)));
}

int linear_quant(const void *x, int64_t ldx, void *q, int64_t ldq, float *scales_dev, int64_t rows, int64_t cols,
                 int dtype, int q_dtype, int act, void *stream)
{
    const char *fn = "linear_quant";
    if (int rc = check_rows(fn, rows, cols, kMaxQuantCols))
        return rc;
    if (!is_value(dtype))
        return report_error(IGC_ERR_INVALID, "%s: dtype %d is neither IGC_BF16 nor IGC_F32", fn, dtype);
    if (!is_code(q_dtype))
        return report_error(IGC_ERR_INVALID, "%s: q_dtype %d is neither IGC_INT8 nor IGC_FP8_E4M3FN", fn, q_dtype);
    if (act != IGC_ACT_NONE && act != IGC_ACT_SILU_GLU)
        return report_error(IGC_ERR_INVALID, "%s: act %d is neither IGC_ACT_NONE nor IGC_ACT_SILU_GLU", fn, act);
    if (rows == 0)
        return report_ok();
    if (int rc = check_operand(fn, {"x", x, ldx, act == IGC_ACT_SILU_GLU ? 2 * cols : cols}))
        return rc;
    if (int rc = check_codes(fn, {"q", q, ldq, code_cols(cols)}))
        return rc;
    if (int rc = check_scales(fn, "scales_dev", scales_dev))
        return rc;
    const QuantParams p{x, q, scales_dev, ldx, ldq, rows, (int)cols};
    return done(fn, launch_linear_quant(p, (Elem)dtype, (Elem)q_dtype, act == IGC_ACT_SILU_GLU,
                                        static_cast<hipStream_t>(stream)));
}

int64_t linear_fwd_workspace_bytes(int64_t m, int64_t n, int64_t k, int dtype, int y_dtype)
{
    const char *fn = "linear_fwd_workspace_bytes";
    LinearPlan pl;
    if (int rc = check_linear(fn, m, n, k, dtype, y_dtype))
        return rc;
    if (int rc = plan_linear(fn, m, n, k, dtype, y_dtype, SIZE_MAX, pl))
        return rc;
    report_ok();
    return pl.ws_need;
}

int linear_plan(int64_t m, int64_t n, int64_t k, int dtype, int y_dtype, size_t workspace_bytes, char *buf, size_t len)
{
    const char *fn = "linear_plan";
    LinearPlan pl;
    if (int rc = check_linear(fn, m, n, k, dtype, y_dtype))
        return rc;
    if (!buf || len == 0)
        return report_error(IGC_ERR_INVALID, "%s: null buffer", fn);
    if (int rc = plan_linear(fn, m, n, k, dtype, y_dtype, workspace_bytes, pl))
        return rc;
    snprintf(buf, len, "tile=%dx%d grid=%lld steps=%d splits=%d ksplit=%d workspace=%lld", pl.bn, pl.bm,
             (long long)pl.tiles_m * pl.tiles_n * pl.splits, pl.nk, pl.splits, pl.ksplit, (long long)pl.ws_need);
    return report_ok();
}

int linear_debug_force(int tile, int splits)
{
    if (tile < -1 || tile >= kNumLinearTiles)
        return report_error(IGC_ERR_INVALID, "linear_debug_force: tile %d unknown", tile);
    if (splits < 0 || splits > kMaxSplits)
        return report_error(IGC_ERR_INVALID, "linear_debug_force: splits = %d must be in [0, %d]", splits, kMaxSplits);
    g_force_linear_tile = tile;
    g_force_linear_splits = splits;
    return report_ok();
}

int linear_fwd(const void *a, int64_t lda, const float *a_scales_dev, const void *w, int64_t ldw,
               const float *w_scales_dev, const float *bias_dev, void *y, int64_t ldy, int64_t m, int64_t n, int64_t k,
               int dtype, int y_dtype, void *workspace_dev, size_t workspace_bytes, void *stream)
{
    const char *fn = "linear_fwd";
    if (int rc = check_linear(fn, m, n, k, dtype, y_dtype))
        return rc;
    if (!workspace_dev && workspace_bytes != 0)
        return report_error(IGC_ERR_INVALID, "%s: null workspace of %zu bytes", fn, workspace_bytes);
    if (!aligned(workspace_dev, 16))
        return report_error(IGC_ERR_ALIGN, "%s: workspace not 16-byte aligned", fn);
    if (m == 0)
        return report_ok();
    const int64_t kp = code_cols(k);
    if (int rc = check_codes(fn, {"a", a, lda, kp}))
        return rc;
    if (int rc = check_codes(fn, {"w", w, ldw, kp}))
        return rc;
    if (lda > kMaxCodeStride || ldw > kMaxCodeStride)
        return report_error(IGC_ERR_UNSUPPORTED, "%s: row strides above %lld codes are not taken", fn,
                            (long long)kMaxCodeStride);
    if (int rc = check_operand(fn, {"y", y, ldy, n}))
        return rc;
    if (int rc = check_scales(fn, "a_scales_dev", a_scales_dev))
        return rc;
    if (int rc = check_scales(fn, "w_scales_dev", w_scales_dev))
        return rc;
    if (!aligned(bias_dev, 4))
        return report_error(IGC_ERR_ALIGN, "%s: bias_dev not 4-byte aligned", fn);
    LinearPlan pl;
    if (int rc = plan_linear(fn, m, n, k, dtype, y_dtype, workspace_bytes, pl))
        return rc;
    LinearParams p{};
    p.a = a;
    p.w = w;
    p.sa = a_scales_dev;
    p.sw = w_scales_dev;
    p.bias = bias_dev;
    p.y = y;
    p.lda = lda;
    p.ldw = ldw;
    p.ldy = ldy;
    p.m = (int)m;
    p.n = (int)n;
    p.nk = pl.nk;
    p.tiles_m = pl.tiles_m;
    p.tiles_n = pl.tiles_n;
    p.splits = pl.splits;
    p.ksplit = pl.ksplit;
    p.group = pl.group;
    p.part = workspace_dev;
    hipStream_t s = static_cast<hipStream_t>(stream);
    hipError_t e = pl.tile == LT_SKINNY
                       ? launch_linear_skinny(p, (Elem)dtype, (Elem)y_dtype, s)
                       : launch_linear(p, pl.tile, (Elem)dtype, (Elem)y_dtype, s);
    if (e == hipSuccess && pl.splits > 1)
        e = launch_linear_reduce(p, (Elem)dtype, (Elem)y_dtype, s);
    return done(fn, e);
}

}  // extern "C"
