// RMS norm of token rows, forward and backward.
//
//   h = T(x + r)            the residual stream, rounded to its type T
//   n = h * rstd,  rstd = 1 / sqrt(mean_k h^2 + eps)
//   v = n * w               (fp32)  ->  y as T, or as 8-bit codes and a scale
//
// The norm is of the stored, rounded h, so that the backward pass, which reads
// it, differentiates the function that ran. Backward, with g = w * dy:
//
//   dx[k] = rstd * (g[k] - n[k] * mean_j(g[j] n[j])) + dres[k]
//   dw[k] = sum over rows of dy[k] * n[k]
//
// dx is the gradient of x and of r alike; dres is the gradient that arrives at h
// along the residual stream. All sums are fp32.
//
// Every operand is read once and every result written once, a few operations a
// byte: HBM bandwidth bounds both directions, and one row on its own is a launch and
// its dependent trips to memory. A copy of 4 GiB reaches 4.8 TB/s on the same card;
// that is no upper bound: these kernels read more than they write, and go to 5.8.
#include <algorithm>
#include <type_traits>

#include "token_rows.h"

namespace igc {

// The row stays in registers between its sum and its output, x, r and w are loaded
// together, and the sum (and the maximum for codes) are lane exchanges, through LDS
// only where several waves share a row. Measured: 8192 x 8192 bf16 with a residual
// and h 92 us, 5.8 TB/s; 9500 x 1280 bf16 to int8 the same way 19 us, 4.4 TB/s; 8192 x
// 8191, no row aligned, 112 us; 1 x 1280 to fp8 2.4 us.
template <typename T, Elem OUT, int TPR, int CH>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void norm_fwd_kernel(NormParams p)
{
    constexpr int NT = TPR < 256 ? 256 : TPR, RPB = NT / TPR;
    __shared__ float red[2][NT / 64];
    const int t = threadIdx.x % TPR;
    const int64_t row = (int64_t)blockIdx.x * RPB + (TPR < 256 ? threadIdx.x / TPR : 0);
    if (row >= p.rows)  // all threads of the row; rows over several waves have a workgroup each
        return;
    const T *x = static_cast<const T *>(p.x) + row * p.ldx;
    const T *w = static_cast<const T *>(p.w);

    float v[CH][8];
    float ss = 0.0f;
    RowRuns<T, TPR, CH> rx;
    rx.load(x, p.cols, t);
    if (p.r) {
        RowRuns<T, TPR, CH> rr;
        rr.load(static_cast<const T *>(p.r) + row * p.ldr, p.cols, t);
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            float a[8];
            rx.unpack(c, p.cols, t, v[c]);
            rr.unpack(c, p.cols, t, a);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[c][i] = Run<T>::rounded(v[c][i] + a[i]);
        }
        if (p.h) {
            T *h = static_cast<T *>(p.h) + row * p.ldh;
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                const int k = 8 * (c * TPR + t);
                Run<T>::store(h + k, p.cols - k, v[c]);
            }
        }
    } else {
#pragma unroll
        for (int c = 0; c < CH; ++c)
            rx.unpack(c, p.cols, t, v[c]);
    }
    RowRuns<T, TPR, CH> rw;
    rw.load(w, p.cols, t);
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            ss = fmaf(v[c][i], v[c][i], ss);
    ss = row_sum<TPR>(ss, red[0]);
    const float rstd = __fdiv_rn(1.0f, __fsqrt_rn(__fdiv_rn(ss, (float)p.cols) + p.eps));

    unsigned m = 0;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        float g[8];
        rw.unpack(c, p.cols, t, g);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            v[c][i] = v[c][i] * rstd * g[i];
            if constexpr (OUT == E_INT8 || OUT == E_FP8)
                m = max(m, abs_bits(v[c][i]));
        }
    }
    if constexpr (OUT == E_INT8 || OUT == E_FP8) {
        m = row_max<TPR>(m, reinterpret_cast<unsigned *>(red[1]));
        const RowCodes<OUT> rc(m);
        if (t == 0)
            p.scales[row] = rc.scale;
        uint8_t *q = static_cast<uint8_t *>(p.y) + row * p.ldy;
        const int end = (int)code_cols(p.cols);  // zero codes from cols to here
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int k = 8 * (c * TPR + t);
            if (k < end)
                *reinterpret_cast<u32x2 *>(q + k) = rc.codes(v[c]);
        }
    } else {
        T *y = static_cast<T *>(p.y) + row * p.ldy;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int k = 8 * (c * TPR + t);
            Run<T>::store(y + k, p.cols - k, v[c]);
        }
    }
}

template <typename T, Elem OUT>
static hipError_t norm_fwd_typed(const NormParams &all, hipStream_t stream)
{
    const bool coded = OUT == E_INT8 || OUT == E_FP8;
    return with_row_shape<kMaxNormCols>((coded ? code_cols(all.cols) : all.cols + 7) / 8, all.rows, [&](auto tpr, auto ch) {
        constexpr int TPR = decltype(tpr)::value, CH = decltype(ch)::value;
        constexpr int NT = TPR < 256 ? 256 : TPR, RPB = NT / TPR;
        for (int64_t r0 = 0; r0 < all.rows; r0 += kRowsPerLaunch) {
            NormParams p = all;
            p.rows = std::min(all.rows - r0, kRowsPerLaunch);
            p.x = static_cast<const T *>(all.x) + r0 * all.ldx;
            p.r = all.r ? static_cast<const T *>(all.r) + r0 * all.ldr : nullptr;
            p.h = all.h ? static_cast<T *>(all.h) + r0 * all.ldh : nullptr;
            p.y = static_cast<char *>(all.y) + r0 * all.ldy * (int64_t)(coded ? 1 : sizeof(T));
            p.scales = coded ? all.scales + r0 : nullptr;
            hipLaunchKernelGGL((norm_fwd_kernel<T, OUT, TPR, CH>), dim3((unsigned)((p.rows + RPB - 1) / RPB)), dim3(NT),
                               0, stream, p);
            if (const hipError_t e = hipGetLastError(); e != hipSuccess)
                return e;
        }
        return hipSuccess;
    });
}

hipError_t launch_norm_fwd(const NormParams &p, Elem t, Elem out, hipStream_t stream)
{
    if (t == E_BF16) {
        if (out == E_INT8)
            return norm_fwd_typed<uint16_t, E_INT8>(p, stream);
        if (out == E_FP8)
            return norm_fwd_typed<uint16_t, E_FP8>(p, stream);
        return norm_fwd_typed<uint16_t, E_BF16>(p, stream);
    }
    if (out == E_INT8)
        return norm_fwd_typed<float, E_INT8>(p, stream);
    if (out == E_FP8)
        return norm_fwd_typed<float, E_FP8>(p, stream);
    return norm_fwd_typed<float, E_F32>(p, stream);
}

// ------------------------------------------------------------------ backward
// A workgroup walks rows g, g + groups, ... and keeps its part of dw in
// registers; the parts go to the workspace as rows of fp32 and a second kernel
// adds them in a fixed order, so dw does not depend on the order in which
// workgroups finish. rstd is computed again: the row of h has to be read anyway.
// HBM bandwidth bounds it: 9500 x 1280 bf16 with dres 20 us, 4.8 TB/s; 16384 x 4096
// fp32 192 us with the sum of the parts, 5.6 TB/s. Rows that are not aligned and do not
// fill their threads or turns stay behind: 2049 x 4097 fp32 without dres 29 us with the
// sum, 3.5 TB/s.

constexpr int bwd_threads(int tpr) { return tpr < 256 ? 256 : tpr; }

template <typename T, int TPR, int CH>
__global__ __launch_bounds__(bwd_threads(TPR)) void norm_bwd_kernel(NormBwdParams p)
{
    constexpr int NT = bwd_threads(TPR), RPB = NT / TPR;
    __shared__ float red[2][2][NT / 64];
    const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;

    float w[CH][8], dw[CH][8];
    // A row's operands are loaded while the DEPTH rows before it are worked on: one, as
    // far as the registers hold them; two for fp32 rows over 6 waves, whose single
    // workgroup per CU has too few loads in flight otherwise (2049 x 4097 28.9 us, 30.8
    // with one; 5000 x 5120 63.0 and 67.5; 8192 x 6144 115 and 112). bf16 and the other
    // shapes lose by the second (9500 x 1280 bf16 27.8 us, 22.9 with one; 8192 x 8192 bf16
    // 106 and 101; 2048 x 4095 fp32 28.8 and 26.7).
    constexpr int DEPTH = TPR == 384 && sizeof(T) == 4 ? 2 : CH * TPR <= 1536 ? 1 : 0;
    struct Operands {
        RowRuns<T, TPR, CH> h, g, r;
    };
    auto fetch = [&](Operands &o, int64_t row) __attribute__((always_inline)) {
        row = min(row, p.rows - 1);  // a row past the last is dropped on unpacking
        o.h.load(static_cast<const T *>(p.h) + row * p.ldh, p.cols, t);
        o.g.load(static_cast<const T *>(p.dy) + row * p.lddy, p.cols, t);
        if (DEPTH > 0 && p.dres)
            o.r.load(static_cast<const T *>(p.dres) + row * p.lddres, p.cols, t);
    };
    // every wave of the workgroup makes the same number of turns: its rows' sums meet at barriers
    const int64_t step = (int64_t)p.groups * RPB;
    int64_t base = (int64_t)blockIdx.x * RPB;
    Operands ops[DEPTH == 2 ? 2 : 1];
#pragma unroll
    for (int i = 0; i < DEPTH; ++i)
        if (base + i * step < p.rows)
            fetch(ops[i], base + i * step + sub);
    RowRuns<T, TPR, CH> rw;
    rw.load(static_cast<const T *>(p.w), p.cols, t);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        rw.unpack(c, p.cols, t, w[c]);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            dw[c][i] = 0.0f;
    }
    // `flip`: the LDS words of one row's sums are not those of the next
    auto turn = [&](Operands &op, int flip) __attribute__((always_inline)) {
        const int64_t row = base + sub;
        const int cols = row < p.rows ? p.cols : 0;
        if (DEPTH == 0)
            fetch(op, row);
        float h[CH][8], g[CH][8], o[CH][8];
        float ss = 0.0f;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            op.h.unpack(c, p.cols, t, h[c]);
            op.g.unpack(c, p.cols, t, g[c]);
            if (DEPTH > 0 && p.dres) {
                op.r.unpack(c, p.cols, t, o[c]);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    o[c][i] = 0.0f;
            }
        }
        if (RPB > 1 && row >= p.rows) {
#pragma unroll
            for (int c = 0; c < CH; ++c)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    h[c][i] = g[c][i] = 0.0f;
        }
        if (DEPTH > 0 && base + DEPTH * step < p.rows)
            fetch(op, row + DEPTH * step);
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                ss = fmaf(h[c][i], h[c][i], ss);
        ss = row_sum<TPR>(ss, red[flip][0]);
        // a row past the last adds nothing to dw: its rstd would be infinite with eps = 0, and 0 * inf is NaN
        const float rstd = RPB > 1 && row >= p.rows ? 0.0f
                                                    : __fdiv_rn(1.0f, __fsqrt_rn(__fdiv_rn(ss, (float)p.cols) + p.eps));
        float gn = 0.0f;
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                h[c][i] *= rstd;
                dw[c][i] = fmaf(g[c][i], h[c][i], dw[c][i]);
                g[c][i] *= w[c][i];
                gn = fmaf(g[c][i], h[c][i], gn);
            }
        const float mean = __fdiv_rn(row_sum<TPR>(gn, red[flip][1]), (float)p.cols);
        T *dx = static_cast<T *>(p.dx) + row * p.lddx;
        const T *rp = static_cast<const T *>(p.dres) + row * p.lddres;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int k = 8 * (c * TPR + t);
            if (DEPTH == 0)
                Run<T>::load(rp + k, p.dres ? cols - k : 0, o[c]);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                o[c][i] = fmaf(rstd, fmaf(-h[c][i], mean, g[c][i]), o[c][i]);
            Run<T>::store(dx + k, cols - k, o[c]);
        }
    };
    for (int flip = 0; base < p.rows; base += step) {
        turn(ops[0], flip);
        if constexpr (DEPTH == 2) {
            base += step;
            if (base >= p.rows)
                break;
            turn(ops[1], 1);
        } else {
            flip ^= 1;
        }
    }
    float *part = p.part + (int64_t)blockIdx.x * p.cols;
    if constexpr (RPB > 1) {  // the rows' parts meet in LDS, element i of run c of thread t at (8 c + i) * TPR + t
        __shared__ float sum[RPB][CH * 8 * TPR];
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                sum[sub][(8 * c + i) * TPR + t] = dw[c][i];
        __syncthreads();
        for (int k = threadIdx.x; k < p.cols; k += NT) {
            const int run = k >> 3, at = (8 * (run / TPR) + (k & 7)) * TPR + run % TPR;
            float s = sum[0][at];
#pragma unroll
            for (int r = 1; r < RPB; ++r)
                s += sum[r][at];
            part[k] = s;
        }
    } else {
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int k = 8 * (c * TPR + t);
            Run<float>::store(part + k, p.cols - k, dw[c]);
        }
    }
}

// dw[k] = sum over groups of part[g][k]: 16 columns a workgroup, its 16-lane groups
// over interleaved rows with up to 8 loads in flight each, the sums added across
// the wave and then in wave order. 4 waves take up to 128 rows in one round of
// loads, 16 waves 512. Latency bounds it, a launch, a trip for the parts that other
// XCDs wrote and the sums: 475 x 1280 4 to 5 us, 228 x 4097 4.9 us.
template <int NW>
__global__ __launch_bounds__(NW * 64) void norm_dw_kernel(NormBwdParams p)
{
    constexpr int U = 8, STEP = 4 * NW;
    __shared__ float sum[NW][16];
    const int col = threadIdx.x & 15, first = threadIdx.x >> 4;
    const int k = blockIdx.x * 16 + col;
    float s = 0.0f;
    if (k < p.cols) {
        const float *src = p.part + k;
        for (int g = first; g < p.groups; g += U * STEP) {
            float v[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                v[u] = g + u * STEP < p.groups ? src[(int64_t)(g + u * STEP) * p.cols] : 0.0f;
#pragma unroll
            for (int u = 0; u < U; ++u)
                s += v[u];
        }
    }
    s += __shfl_xor(s, 16);
    s += __shfl_xor(s, 32);
    if ((threadIdx.x & 48) == 0)
        sum[threadIdx.x >> 6][col] = s;
    __syncthreads();
    if (threadIdx.x < 16 && k < p.cols) {
        s = sum[0][col];
#pragma unroll
        for (int w = 1; w < NW; ++w)
            s += sum[w][col];
        p.dw[k] = s;
    }
}

// Workgroups of 4 waves for rows of `es` bytes an element: two per CU, three where one
// holds less than 4 KB of each operand (152000 x 80 bf16 24.8 us, 27.7 with two), and one
// where that does as well, since every workgroup's part of dw is written and read once
// more:
//  - its rows take more than 4 waves (2049 x 4097 bf16 25.1 us, 29.6 with two), or it
//    holds 16 KB of each operand in aligned loads (16384 x 4096 fp32 192 us, 202 with
//    two; 2048 x 4095 fp32 keeps two, 26.7 us, 29.6 with one);
//  - the parts of two would add more than about a fifth to the operands' bytes, a
//    third for unaligned rows, whose loads take longer (2048 x 4096 bf16 17.4 us, 18.2
//    with two; 2500 x 3001 keeps two, 19.8 us, 22.7 with one);
//  - two would leave CUs idle for a quarter of their turns (3000 x 2047 fp32, 750
//    workgroups' rows: 20.6 us, 25.3 with two turns of 375).
// And no more than the longest of them needs: a few over that would leave the rest
// waiting for their CUs.
int norm_bwd_groups(int64_t rows, int64_t cols, int64_t es, int64_t cus)
{
    if (rows == 0)
        return 1;
    int64_t rpb = 1;  // rows a workgroup works on at once
    bool large = false;
    (void)with_row_shape<kMaxNormBwdCols, true>((cols + 7) / 8, rows, [&](auto tpr, auto) {
        rpb = bwd_threads(decltype(tpr)::value) / decltype(tpr)::value;
        large = decltype(tpr)::value > 256;
        return hipSuccess;
    });
    const int64_t held = es * cols * rpb;
    auto turns = [&](int64_t per_cu) { return (rows + per_cu * cus * rpb - 1) / (per_cu * cus * rpb); };
    const bool whole = cols % 8 == 0;
    const bool one = large || (whole && held >= 16000) || rows * es <= (whole ? 24 : 16) * cus || 4 * turns(1) <= 3 * 2 * turns(2);
    const int64_t n = turns(one ? 1 : held < 4096 ? 3 : 2);
    return (int)((rows + n * rpb - 1) / (n * rpb));
}

template <typename T>
static hipError_t norm_bwd_typed(NormBwdParams p, hipStream_t stream)
{
    if (p.groups == 1)  // the only part is dw
        p.part = p.dw;
    return with_row_shape<kMaxNormBwdCols, true>((p.cols + 7) / 8, p.rows, [&](auto tpr, auto ch) {
        constexpr int TPR = decltype(tpr)::value, CH = decltype(ch)::value;
        hipLaunchKernelGGL((norm_bwd_kernel<T, TPR, CH>), dim3((unsigned)p.groups), dim3(bwd_threads(TPR)), 0, stream, p);
        const dim3 grid((unsigned)((p.cols + 15) / 16));
        if (p.groups > 128)
            hipLaunchKernelGGL(norm_dw_kernel<16>, grid, dim3(1024), 0, stream, p);
        else if (p.groups > 1)
            hipLaunchKernelGGL(norm_dw_kernel<4>, grid, dim3(256), 0, stream, p);
        return hipGetLastError();
    });
}

hipError_t launch_norm_bwd(const NormBwdParams &p, Elem t, hipStream_t stream)
{
    return t == E_BF16 ? norm_bwd_typed<uint16_t>(p, stream) : norm_bwd_typed<float>(p, stream);
}

}  // namespace igc
