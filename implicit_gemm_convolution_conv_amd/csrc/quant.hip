// Row quantisation: 8-bit codes and one scale for each row of x, or of the gated
// activation silu(gate) * up of rows that hold both halves side by side.
//
//   v = x                                  (fp32)
//   v = g / (1 + exp(-g)) * u              g = x[:cols], u = x[cols:2 cols]
//
// The rows of a weight matrix are its output channels, those of an activation
// its tokens. One read of x and one write of the codes: HBM bandwidth bounds it.
#include <algorithm>
#include <type_traits>

#include "token_rows.h"

namespace igc {

// exp(x) to about the accuracy of the hardware's 2^f: x * log2(e) is taken as a
// rounded product p and its remainder e (from the fma, plus the part of log2(e)
// below its fp32 value), and 2^(p + e) = 2^p * (1 + e ln 2) to first order, e
// being below 2^-17 for |x| < 128. A plain 2^(x * log2 e)
// would carry a relative error of |x| * 2^-24, which moves codes.
__device__ __attribute__((always_inline)) inline float exp_f32(float x)
{
    constexpr float L = 0x1.715476p+0f, l = 0x1.4ae0cp-26f;  // log2(e) = L + l
    const float p = x * L;
    const float e = fmaf(x, l, fmaf(x, L, -p));
    const float b = __builtin_amdgcn_exp2f(p);
    return fmaf(b * e, 0x1.62e43p-1f, b);
}

// g / (1 + exp(-g)) for g >= kGateTail. The exponent is kept above -90, where the
// sum is 1, and no infinity enters the remainder term above. The reciprocal's
// quotient is corrected once by its remainder: each of these roundings moves a code
// now and then.
constexpr float kGateTail = -80.0f;

__device__ __attribute__((always_inline)) inline float silu(float g)
{
    const float d = 1.0f + exp_f32(fmaxf(-g, -90.0f));
    const float r = __builtin_amdgcn_rcpf(d);
    const float q = g * r;
    return fmaf(fmaf(-d, q, g), r, q);
}

// silu(g) * u for g below kGateTail, where 1 + exp(-g) is exp(-g) in fp32: g exp(g)
// u as (g e)(e u), e = exp(g / 2). The reciprocal above would leave fp32's range
// from -88 on; e does so below -174, where the result is under 2^-100 whatever u
// is. Gates down to the type's lowest value give zero.
__device__ __attribute__((always_inline)) inline float gated_tail(float g, float u)
{
    const float e = exp_f32(fmaxf(0.5f * g, -100.0f));
    return (g * e) * (e * u);
}

// v = silu(v) * u for a run. Few rows hold gates below kGateTail: a wave without
// them skips that part.
__device__ __attribute__((always_inline)) inline void gate(float (&v)[8], const float (&u)[8])
{
    float low = v[0], g[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        low = fminf(low, v[i]);
        g[i] = v[i];
        v[i] = silu(g[i]) * u[i];
    }
    if (__any(low < kGateTail)) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = g[i] < kGateTail ? gated_tail(g[i], u[i]) : v[i];
    }
}

// The row's values stay in registers between its maximum and its codes (gate and up
// as they lie in memory, all loads together). Measured: 9500 rows of 2 x 5120 bf16,
// gated, to fp8 47 us, 5.2 TB/s; 8192 x 8192 bf16 to fp8 36 us, 5.5 TB/s; 77 x 2047
// fp32 to int8 2.7 us, a launch and two trips to memory.
//
// CH = 0: rows longer than the registers hold are read twice, the second time
// from the L2 cache for all but the widest grids.
template <typename T, Elem OUT, bool GLU, int TPR, int CH>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void linear_quant_kernel(QuantParams p)
{
    constexpr int NT = TPR < 256 ? 256 : TPR, RPB = NT / TPR;
    __shared__ unsigned red[NT / 64];
    const int t = threadIdx.x % TPR;
    const int64_t row = (int64_t)blockIdx.x * RPB + (TPR < 256 ? threadIdx.x / TPR : 0);
    if (row >= p.rows)
        return;
    const T *x = static_cast<const T *>(p.x) + row * p.ldx;
    const int end = (int)code_cols(p.cols);  // zero codes from cols to here
    auto run = [&](int k, float (&v)[8]) __attribute__((always_inline)) {
        Run<T>::load(x + k, p.cols - k, v);
        if constexpr (GLU) {
            float u[8];
            Run<T>::load(x + p.cols + k, p.cols - k, u);
            gate(v, u);
        }
    };
    unsigned m = 0;
    auto top = [&](const float (&v)[8]) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            m = max(m, abs_bits(v[i]));
    };

    float v[CH > 0 ? CH : 1][8];
    if constexpr (CH > 0) {
        RowRuns<T, TPR, CH> rx, ru;
        rx.load(x, p.cols, t);
        if constexpr (GLU)
            ru.load(x + p.cols, p.cols, t);
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            rx.unpack(c, p.cols, t, v[c]);
            if constexpr (GLU) {
                float u[8];
                ru.unpack(c, p.cols, t, u);
                gate(v[c], u);
            }
            top(v[c]);
        }
    } else {
        for (int k = 8 * t; k < p.cols; k += 8 * TPR) {
            run(k, v[0]);
            top(v[0]);
        }
    }
    m = row_max<TPR>(m, red);
    const RowCodes<OUT> rc(m);
    if (t == 0)
        p.scales[row] = rc.scale;
    uint8_t *q = static_cast<uint8_t *>(p.q) + row * p.ldq;
    if constexpr (CH > 0) {
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int k = 8 * (c * TPR + t);
            if (k < end)
                *reinterpret_cast<u32x2 *>(q + k) = rc.codes(v[c]);
        }
    } else {
        for (int k = 8 * t; k < end; k += 8 * TPR) {
            run(k, v[0]);
            *reinterpret_cast<u32x2 *>(q + k) = rc.codes(v[0]);
        }
    }
}

template <typename T, Elem OUT, bool GLU>
static hipError_t quant_typed(const QuantParams &all, hipStream_t stream)
{
    return with_row_shape<kMaxQuantCols>(code_cols(all.cols) / 8, all.rows, [&](auto tpr, auto ch) {
        constexpr int TPR = decltype(tpr)::value, CH = decltype(ch)::value;
        constexpr int NT = TPR < 256 ? 256 : TPR, RPB = NT / TPR;
        for (int64_t r0 = 0; r0 < all.rows; r0 += kRowsPerLaunch) {
            QuantParams p = all;
            p.rows = std::min(all.rows - r0, kRowsPerLaunch);
            p.x = static_cast<const T *>(all.x) + r0 * all.ldx;
            p.q = static_cast<uint8_t *>(all.q) + r0 * all.ldq;
            p.scales = all.scales + r0;
            hipLaunchKernelGGL((linear_quant_kernel<T, OUT, GLU, TPR, CH>), dim3((unsigned)((p.rows + RPB - 1) / RPB)),
                               dim3(NT), 0, stream, p);
            if (const hipError_t e = hipGetLastError(); e != hipSuccess)
                return e;
        }
        return hipSuccess;
    });
}

template <typename T>
static hipError_t quant_out(const QuantParams &p, Elem out, bool glu, hipStream_t stream)
{
    if (out == E_INT8)
        return glu ? quant_typed<T, E_INT8, true>(p, stream) : quant_typed<T, E_INT8, false>(p, stream);
    return glu ? quant_typed<T, E_FP8, true>(p, stream) : quant_typed<T, E_FP8, false>(p, stream);
}

hipError_t launch_linear_quant(const QuantParams &p, Elem t, Elem out, bool glu, hipStream_t stream)
{
    return t == E_BF16 ? quant_out<uint16_t>(p, out, glu, stream) : quant_out<float>(p, out, glu, stream);
}

}  // namespace igc
