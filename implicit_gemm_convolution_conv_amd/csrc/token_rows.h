// Pieces shared by the kernels that take one row (a token, or an output channel
// of a weight matrix) at a time: the row in registers, sums and maxima over it,
// and its quantisation to 8 bits.
//
// A row of `cols` elements is held by TPR threads (part of a wave, a wave, 4 or 16
// waves, in the norm's backward pass also 6 or 8), CH runs of 8 consecutive elements
// each, run c of thread t at element 8 * (c * TPR + t): every load of a wave covers runs side by side. The row
// is read from memory once; all that follows works on the registers.
#pragma once

#include "conv_igemm.h"
#include "token_ops.h"

namespace igc {

// 16-byte accesses whose address is only aligned to the element: a row of an odd
// length starts anywhere.
typedef int i32x4_a2 __attribute__((ext_vector_type(4), aligned(2)));
typedef float f32x4_a4 __attribute__((ext_vector_type(4), aligned(4)));
typedef float f32x8 __attribute__((ext_vector_type(8)));

template <typename T>
struct Run;

template <>
struct Run<uint16_t> {  // bf16
    using Raw = i32x4;  // as it lies in memory, for loads ahead of their use
    static __device__ __attribute__((always_inline)) Raw whole(const uint16_t *p)
    {
        return *reinterpret_cast<const i32x4_a2 *>(p);
    }
    // the `left` elements at p (8 of them at most), zeros following
    static __device__ __attribute__((always_inline)) Raw raw(const uint16_t *p, int left)
    {
        if (left >= 8)
            return whole(p);
        Raw u = {0, 0, 0, 0};
        if (left > 0) {  // the row's last run: all loads go out together, those past the end to its first element
            unsigned e[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                e[i] = p[i < left ? i : 0];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                u[i >> 1] |= i < left ? (int)(e[i] << (16 * (i & 1))) : 0;
        }
        return u;
    }
    // element i of the result is element i + s of u, zero past the last
    static __device__ __attribute__((always_inline)) Raw shifted(Raw u, int s)
    {
        const Raw zero = {0, 0, 0, 0};
        u = s & 4 ? __builtin_shufflevector(u, zero, 2, 3, 4, 5) : u;
        u = s & 2 ? __builtin_shufflevector(u, zero, 1, 2, 3, 4) : u;
        const Raw next = __builtin_shufflevector(u, zero, 1, 2, 3, 4);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            u[i] = s & 1 ? (int)__builtin_amdgcn_alignbit((unsigned)next[i], (unsigned)u[i], 16) : u[i];
        return s < 8 ? u : zero;
    }
    static __device__ __attribute__((always_inline)) void unpack(const Raw &u, float (&v)[8])
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float((unsigned)u[i] << 16);
            v[2 * i + 1] = __uint_as_float((unsigned)u[i] & 0xffff0000u);
        }
    }
    static __device__ __attribute__((always_inline)) void load(const uint16_t *p, int left, float (&v)[8])
    {
        unpack(raw(p, left), v);
    }
    static __device__ __attribute__((always_inline)) void store(uint16_t *p, int left, const float (&v)[8])
    {
        if (left >= 8) {
            i32x4 u;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                u[i] = (int)bf16_pack2(v[2 * i], v[2 * i + 1]);
            *reinterpret_cast<i32x4_a2 *>(p) = u;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < left)
                    p[i] = (uint16_t)f32_to_bf16_rne(v[i]);
        }
    }
    // what a store and a load leave of v
    static __device__ __attribute__((always_inline)) float rounded(float v)
    {
        return __uint_as_float(f32_to_bf16_rne(v) << 16);
    }
};

template <>
struct Run<float> {
    using Raw = f32x8;
    static __device__ __attribute__((always_inline)) Raw whole(const float *p)
    {
        const f32x4 a = *reinterpret_cast<const f32x4_a4 *>(p), b = *reinterpret_cast<const f32x4_a4 *>(p + 4);
        return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
    }
    static __device__ __attribute__((always_inline)) Raw raw(const float *p, int left)
    {
        if (left >= 8)
            return whole(p);
        Raw u = {0, 0, 0, 0, 0, 0, 0, 0};
        if (left > 0) {
            float e[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                e[i] = p[i < left ? i : 0];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                u[i] = i < left ? e[i] : 0.0f;
        }
        return u;
    }
    static __device__ __attribute__((always_inline)) Raw shifted(Raw u, int s)
    {
        const Raw zero = {0, 0, 0, 0, 0, 0, 0, 0};
        u = s & 4 ? __builtin_shufflevector(u, zero, 4, 5, 6, 7, 8, 9, 10, 11) : u;
        u = s & 2 ? __builtin_shufflevector(u, zero, 2, 3, 4, 5, 6, 7, 8, 9) : u;
        u = s & 1 ? __builtin_shufflevector(u, zero, 1, 2, 3, 4, 5, 6, 7, 8) : u;
        return s < 8 ? u : zero;
    }
    static __device__ __attribute__((always_inline)) void unpack(const Raw &u, float (&v)[8])
    {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = u[i];
    }
    static __device__ __attribute__((always_inline)) void load(const float *p, int left, float (&v)[8])
    {
        unpack(raw(p, left), v);
    }
    static __device__ __attribute__((always_inline)) void store(float *p, int left, const float (&v)[8])
    {
        if (left >= 8) {
            *reinterpret_cast<f32x4_a4 *>(p) = f32x4{v[0], v[1], v[2], v[3]};
            *reinterpret_cast<f32x4_a4 *>(p + 4) = f32x4{v[4], v[5], v[6], v[7]};
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < left)
                    p[i] = v[i];
        }
    }
    static __device__ __attribute__((always_inline)) float rounded(float v) { return v; }
};

// One thread's CH runs of a row, as they lie in memory, loaded without a branch, all
// loads in flight together: a run that is not whole is loaded as the row's last 8
// elements, and on unpacking shifted to its place or dropped. Only the one c whose
// runs cross the row's end is shifted (8192 x 8192 bf16 norm 93 us; 100 us with a
// branch a run, which waits for its load inside).
template <typename T, int TPR, int CH>
struct RowRuns {
    static constexpr bool kShort = TPR == 16;  // rows below 8 elements come here
    typename Run<T>::Raw u[CH];

    __device__ __attribute__((always_inline)) void load(const T *p, int cols, int t)
    {
        if (kShort && cols < 8) {
#pragma unroll
            for (int c = 0; c < CH; ++c)
                u[c] = Run<T>::raw(p + 8 * (c * TPR + t), cols - 8 * (c * TPR + t));
        } else if constexpr (CH == 1) {
            u[0] = typename Run<T>::Raw{};
            if (8 * t < cols)
                u[0] = Run<T>::whole(p + min(8 * t, cols - 8));
        } else {
#pragma unroll
            for (int c = 0; c < CH; ++c)
                u[c] = Run<T>::whole(p + min(8 * (c * TPR + t), cols - 8));
        }
    }
    __device__ __attribute__((always_inline)) void unpack(int c, int cols, int t, float (&v)[8]) const
    {
        const int end = 8 * TPR * (c + 1);  // of this c's runs
        typename Run<T>::Raw w = u[c];
        if (end > cols && !(kShort && cols < 8)) {
            const int s = max(end - 8 * TPR + 8 * t + 8 - cols, 0);
            if (cols & 7) {
                w = Run<T>::shifted(w, s);
            } else {
#pragma unroll
                for (unsigned i = 0; i < sizeof(w) / 4; ++i)
                    w[i] = s < 8 ? w[i] : 0;
            }
        }
        Run<T>::unpack(w, v);
    }
};

// v combined by `op` over lanes 0..N-1, N..2N-1, ... of the wave, N = 16, 32 or 64,
// in every lane of each. Lane exchanges in the vector unit: neighbours, pairs,
// mirrored halves and rows of 16 lanes, then swapped rows and half waves, a few
// cycles each where a shuffle through LDS takes a trip there and back.
template <int N, typename Op>
__device__ __attribute__((always_inline)) inline unsigned lanes_combine(unsigned v, Op &&op)
{
    v = op(v, (unsigned)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xf, 0xf, true));   // lane ^ 1
    v = op(v, (unsigned)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xf, 0xf, true));   // lane ^ 2
    v = op(v, (unsigned)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xf, 0xf, true));  // mirrored in 8: the other 4
    v = op(v, (unsigned)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xf, 0xf, true));  // mirrored in 16: the other 8
    if constexpr (N >= 32) {
        const auto s = __builtin_amdgcn_permlane16_swap(v, v, false, false);
        v = op(s[0], s[1]);
    }
    if constexpr (N >= 64) {
        const auto s = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        v = op(s[0], s[1]);
    }
    return v;
}

// Sum / maximum over the TPR threads of a row, in every one of them. `red` is
// LDS of one word for each wave of the workgroup, the kernel's own for each call;
// all threads of a workgroup call it together where TPR > 64. The order of the sum
// is fixed by TPR, so results do not change from call to call.
template <int TPR>
__device__ __attribute__((always_inline)) inline float row_sum(float v, float *red)
{
    v = __uint_as_float(lanes_combine<(TPR < 64 ? TPR : 64)>(__float_as_uint(v), [](unsigned a, unsigned b) {
        return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
    }));
    if constexpr (TPR > 64) {
        if ((threadIdx.x & 63) == 0)
            red[threadIdx.x >> 6] = v;
        __syncthreads();
        red += threadIdx.x / TPR * (TPR / 64);
        v = red[0];
#pragma unroll
        for (int i = 1; i < TPR / 64; ++i)
            v += red[i];
    }
    return v;
}

template <int TPR>
__device__ __attribute__((always_inline)) inline unsigned row_max(unsigned v, unsigned *red)
{
    v = lanes_combine<(TPR < 64 ? TPR : 64)>(v, [](unsigned a, unsigned b) { return max(a, b); });
    if constexpr (TPR > 64) {
        if ((threadIdx.x & 63) == 0)
            red[threadIdx.x >> 6] = v;
        __syncthreads();
        v = red[0];
#pragma unroll
        for (int i = 1; i < TPR / 64; ++i)
            v = max(v, red[i]);
    }
    return v;
}

// 8-bit codes of a row. The row maximum a = max |v| is taken over bit patterns
// (non-negative floats order like them, and a NaN comes out on top), floored at
// 2^-100 so that neither quotient overflows; scale = a / top, code =
// round-to-nearest-even(fp32(v * (top / a))), top = 127 (int8) or 448 (E4M3FN). A row
// with an infinity or a NaN gets the scale NaN and zero codes: all of it
// dequantises to NaN.
template <Elem OUT>
struct RowCodes {
    float scale, inv;

    __device__ __attribute__((always_inline)) explicit RowCodes(unsigned amax_bits)
    {
        constexpr float top = OUT == E_INT8 ? 127.0f : 448.0f;
        const float a = fmaxf(__uint_as_float(amax_bits), 0x1p-100f);
        const bool finite = amax_bits < 0x7f800000u;
        scale = finite ? __fdiv_rn(a, top) : __uint_as_float(0x7fc00000u);
        inv = finite ? __fdiv_rn(top, a) : 0.0f;
    }
    // Codes of 8 elements, of the product v * inv rounded to fp32. int8: adding
    // 1.5 * 2^23 rounds the product (at most 127 * (1 + 2^-23)) to an integer in
    // the low mantissa bits, whose low byte is the code in two's complement. One
    // fma would decide ties by the error of inv: v = a / 2, on the tie 63.5, is
    // common in bf16 rows. fp8: the hardware conversion; 448 * (1 + 2^-23) still
    // rounds to 448. A zero `inv` (a row that is not finite) gives zero codes
    // without looking at v.
    __device__ __attribute__((always_inline)) u32x2 codes(const float (&v)[8]) const
    {
#pragma clang fp contract(off)
        u32x2 c = {0, 0};
        if (inv == 0.0f)
            return c;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if constexpr (OUT == E_INT8) {
                unsigned b[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    b[e] = __float_as_uint(v[4 * i + e] * inv + 12582912.0f);
                const unsigned lo = __builtin_amdgcn_perm(b[1], b[0], 0x0c0c0400u);
                const unsigned hi = __builtin_amdgcn_perm(b[3], b[2], 0x04000c0cu);
                c[i] = lo | hi;
            } else {
                int d = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i] * inv, v[4 * i + 1] * inv, 0, false);
                c[i] = (unsigned)__builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i + 2] * inv, v[4 * i + 3] * inv, d, true);
            }
        }
        return c;
    }
};

__device__ __attribute__((always_inline)) inline unsigned abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// Launch shape of a row of `runs` runs of 8 elements: f(TPR, CH) as integral
// constants, the smallest register tile that holds the row (CH = 0: none does). A
// wave takes a whole row where enough rows fill the GPU with waves (9500 x 1280 bf16
// to fp8 16.9 us, 18.6 us with 4 waves a row), and several short ones; fewer rows
// spread over 4 waves. SHORT_RUNS, where a kernel works long on each run (the norm's
// backward pass), spreads long rows over 6 or 8 waves: 2048 x 4104 bf16 20.8 us, 22.7 us
// with 4 waves of 3 runs; 4000 x 12288 80.8 and 117.5; 8192 x 8192 fp32 151.1 and 149.2.
template <int64_t MAX_COLS, bool SHORT_RUNS = false, typename F>
hipError_t with_row_shape(int64_t runs, int64_t rows, F &&f)
{
    using std::integral_constant;
#define IGC_ROW(TPR_, CH_) return f(integral_constant<int, TPR_>{}, integral_constant<int, CH_>{})
    if (runs <= 16) IGC_ROW(16, 1);
    if (runs <= 32) IGC_ROW(32, 1);
    if (rows >= 1024) {
        if (runs <= 64) IGC_ROW(64, 1);
        if (runs <= 128) IGC_ROW(64, 2);
        if (runs <= 192) IGC_ROW(64, 3);
        if (runs <= 256) IGC_ROW(64, 4);
    } else if (runs <= 64) {
        IGC_ROW(64, 1);
    }
    if (runs <= 256) IGC_ROW(256, 1);
    if (runs <= 512) IGC_ROW(256, 2);
    if constexpr (SHORT_RUNS) {
        if (runs <= 768) IGC_ROW(384, 2);
        if (runs <= 1024) IGC_ROW(512, 2);
        if (runs <= 1536) IGC_ROW(512, 3);
        if (runs <= 2048) IGC_ROW(512, 4);
    } else {
        if (runs <= 768) IGC_ROW(256, 3);
        if (runs <= 1024) IGC_ROW(256, 4);
        if (runs <= 1536) IGC_ROW(256, 6);
        if (runs <= 2048) IGC_ROW(256, 8);
        if (runs <= 4096) IGC_ROW(1024, 4);
        if constexpr (MAX_COLS > 4096 * 8)
            IGC_ROW(1024, 0);
    }
    return hipErrorInvalidValue;
#undef IGC_ROW
}

}  // namespace igc
