// Internal declarations of the token operators: the RMS norm (with the
// residual's addition, an 8-bit output and a backward pass), the row quantiser
// and the linear layer on 8-bit operands (not part of the C ABI).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace igc {

// Element types, as the C ABI numbers them.
enum Elem { E_BF16 = 0, E_FP8 = 1, E_F32 = 2, E_INT8 = 3 };

// Rows of codes are padded with zeros to a multiple of this many elements (one
// 128-byte reduction step of the linear kernels).
constexpr int kCodePad = 128;
constexpr int64_t code_cols(int64_t k) { return (k + kCodePad - 1) / kCodePad * kCodePad; }

// Longest rows the norm's kernels hold in registers: 1024 threads x 4 runs of 8
// forward, which holds the residual and the weight next to the row; 512 threads x
// 4 runs backward, which keeps h, w * dy, w and dw.
constexpr int64_t kMaxNormCols = 32768;
constexpr int64_t kMaxNormBwdCols = 16384;
// Longest reduction of the linear layer: 131071 products of int8 codes, each at
// most 2^14, stay below 2^31.
constexpr int64_t kMaxLinearK = 131071;
constexpr int64_t kMaxQuantCols = kMaxLinearK;  // longer rows have no use here
// Largest row stride (bytes) of a code matrix: 256 rows of a tile stay within
// the 2^31 bytes a buffer resource addresses.
constexpr int64_t kMaxCodeStride = int64_t(1) << 22;

struct NormParams {
    const void *x, *r, *w;
    void *h, *y;
    float *scales;
    int64_t ldx, ldr, ldh, ldy;
    int64_t rows;
    int cols;
    float eps;
};

struct NormBwdParams {
    const void *dy, *h, *w, *dres;
    void *dx;
    float *dw, *part;
    int64_t lddy, ldh, lddres, lddx;
    int64_t rows;
    int cols;
    float eps;
    int groups;  // workgroups over the rows, one row of `part` each
};

struct QuantParams {
    const void *x;
    void *q;
    float *scales;
    int64_t ldx, ldq;
    int64_t rows;
    int cols;
};

struct LinearParams {
    const void *a, *w;       // codes: tokens [m][lda], features [n][ldw], k contiguous
    const float *sa, *sw;    // scale of each token / of each feature
    const float *bias;       // one per feature, or null
    void *y;                 // [m][ldy]
    int64_t lda, ldw, ldy;
    int m, n;
    int nk;                  // reduction steps of 128 codes
    int tiles_m, tiles_n;
    int group;               // token tiles a raster group walks together
    int splits, ksplit;      // split j runs steps [j * ksplit, min(nk, (j + 1) * ksplit))
    void *part;              // splits > 1: sums [split][m][n], int32 (int8 codes) or fp32 (fp8)
};

// Rows of one launch of a row kernel: with 1024 threads a row, 2^31 threads.
constexpr int64_t kRowsPerLaunch = int64_t(1) << 21;

hipError_t launch_norm_fwd(const NormParams &p, Elem t, Elem out, hipStream_t stream);
// Workgroups norm_bwd runs (rows of its partial sums of dw) on elements of `es` bytes.
int norm_bwd_groups(int64_t rows, int64_t cols, int64_t es, int64_t cus);
hipError_t launch_norm_bwd(const NormBwdParams &p, Elem t, hipStream_t stream);
hipError_t launch_linear_quant(const QuantParams &p, Elem t, Elem out, bool glu, hipStream_t stream);

// Kernel variants of the linear layer.
enum LinearTile { LT_256 = 0, LT_128, LT_64, LT_32x64, LT_32, LT_SKINNY, LT_256x128, LT_64x128, kNumLinearTiles };
// Workgroups of 16 features x 16 tokens, the reduction over their waves, each of
// which loads this many of its steps together.
constexpr int kSkinnyFeatures = 16, kSkinnyTokens = 16, kSkinnyWaves = 8, kSkinnyLoads = 4;
hipError_t launch_linear_skinny(const LinearParams &p, Elem t, Elem out, hipStream_t stream);
hipError_t launch_linear(const LinearParams &p, int tile, Elem t, Elem out, hipStream_t stream);
hipError_t launch_linear_reduce(const LinearParams &p, Elem t, Elem out, hipStream_t stream);

// From the C ABI's translation unit: record an error text / success for
// conv_last_error, and the current device's compute units.
int report_error(int code, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
int report_ok();
int64_t compute_units();

}  // namespace igc
