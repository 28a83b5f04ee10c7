// Linear layer on 8-bit operands: y[m][n] = (sum_k a[m][k] w[n][k]) * sa[m] *
// sw[n] + bias[n], int8 codes with int32 sums or fp8 E4M3FN codes with fp32 sums.
//
// The matrix instruction's rows are features and its columns tokens, so that a
// lane's four accumulators are four neighbouring outputs of one token. Both
// operands are k-contiguous rows of 128-byte steps and go straight from memory
// into LDS.
#pragma once

#include <type_traits>

#include "conv_igemm_buf.h"
#include "token_ops.h"

namespace igc {

typedef int i32x4_a2 __attribute__((ext_vector_type(4), aligned(2)));
typedef float f32x4_a4 __attribute__((ext_vector_type(4), aligned(4)));

// Matrix instructions of one operand type on 16 x 16 blocks. A 128-code step
// of a row is 8 chunks of 16 bytes, chunk q at slot q ^ lsw. Which codes a
// lane group holds is free as long as both operands agree.
//
// PRECISE matters for fp8: within one fp8 instruction (any width) products are
// aligned to the largest of them and lose what falls about 13 bits below it
// (measured: up to 2^-11.4 of the largest product, 4e-5 of the result's 2-norm on
// codes of mixed exponents); the running sum itself is fp32. Where large products
// do not cancel, that is far below a bf16 output's rounding of 2^-8 and the codes'
// own 2^-4, so bf16 outputs take it; where they do, as with outlier channels of
// opposite signs, it may be more than the small result itself. An fp32 output gets
// the exact codes widened to bf16 and the bf16 instruction, at half the rate: that
// is the way to fp32 sums, and the header says so.
template <Elem T, bool PRECISE>
struct Mma;

// int8: a slice is one chunk per group of 16 lanes.
template <bool PRECISE>
struct Mma<E_INT8, PRECISE> {
    using Frag = i32x4;
    using Acc = i32x4;
    static constexpr int kSlices = 2;
    static __device__ __attribute__((always_inline)) Frag frag(const char *rowp, int h, int lgrp, int lsw)
    {
        return *reinterpret_cast<const i32x4 *>(rowp + (((h * 4 + lgrp) ^ lsw) * 16));
    }
    static __device__ __attribute__((always_inline)) void mma(const Frag &a, const Frag &b, Acc &c)
    {
        c = __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
    }
};

// fp8: the whole step in one slice, two chunks per lane group, 4 chunks apart (the
// int8 slices' chunks, whose LDS reads touch every bank once).
template <>
struct Mma<E_FP8, false> {
    using Frag = i32x8;
    using Acc = f32x4;
    static constexpr int kSlices = 1;
    static __device__ __attribute__((always_inline)) Frag frag(const char *rowp, int, int lgrp, int lsw)
    {
        const i32x4 lo = *reinterpret_cast<const i32x4 *>(rowp + ((lgrp ^ lsw) * 16));
        const i32x4 hi = *reinterpret_cast<const i32x4 *>(rowp + (((lgrp + 4) ^ lsw) * 16));
        return i32x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    }
    static __device__ __attribute__((always_inline)) void mma(const Frag &a, const Frag &b, Acc &c)
    {
        c = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, 0, 0, 0, 0);
    }
};

// fp8 widened to bf16 (exact: 4 of 8 significant bits), two bf16 instructions for
// each chunk.
template <>
struct Mma<E_FP8, true> {
    struct Frag {
        bf16x8 half[2];
    };
    using Acc = f32x4;
    static constexpr int kSlices = 2;
    static __device__ __attribute__((always_inline)) Frag widen(const i32x4 &u)
    {
        Frag f;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const bf16x2_t lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((unsigned)u[q], 1.0f, false);
            const bf16x2_t hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((unsigned)u[q], 1.0f, true);
            f.half[q >> 1][4 * (q & 1) + 0] = lo[0];
            f.half[q >> 1][4 * (q & 1) + 1] = lo[1];
            f.half[q >> 1][4 * (q & 1) + 2] = hi[0];
            f.half[q >> 1][4 * (q & 1) + 3] = hi[1];
        }
        return f;
    }
    static __device__ __attribute__((always_inline)) i32x4 narrow(const char *rowp, int h, int lgrp, int lsw)
    {
        return *reinterpret_cast<const i32x4 *>(rowp + (((h * 4 + lgrp) ^ lsw) * 16));
    }
    static __device__ __attribute__((always_inline)) Frag frag(const char *rowp, int h, int lgrp, int lsw)
    {
        return widen(narrow(rowp, h, lgrp, lsw));
    }
    static __device__ __attribute__((always_inline)) void mma(const Frag &a, const Frag &b, Acc &c)
    {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.half[i], b.half[i], c, 0, 0, 0);
    }
};

// acc * sa * sw + bias in fp32 for four neighbouring features (an int32 sum above
// 2^24 is rounded to fp32 first, half a unit of the result).
template <typename Acc>
__device__ __attribute__((always_inline)) inline f32x4 scaled(const Acc &acc, float sa, const f32x4 &sw, const f32x4 &bias)
{
    f32x4 v;
#pragma unroll
    for (int e = 0; e < 4; ++e)
        v[e] = fmaf((float)acc[e] * sa, sw[e], bias[e]);
    return v;
}

// Outputs n .. n + 3 (those below p.n) of token m.
template <Elem OUT>
__device__ __attribute__((always_inline)) inline void store_outputs(const LinearParams &p, int m, int n, const f32x4 &v)
{
    const int64_t off = (int64_t)m * p.ldy + n;
    if constexpr (OUT == E_F32) {
        float *y = static_cast<float *>(p.y) + off;
        if (n + 3 < p.n) {
            *reinterpret_cast<f32x4_a4 *>(y) = f32x4{v[0], v[1], v[2], v[3]};
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (n + e < p.n)
                    y[e] = v[e];
        }
    } else {
        typedef uint32_t u32x2_a2 __attribute__((ext_vector_type(2), aligned(2)));
        uint16_t *y = static_cast<uint16_t *>(p.y) + off;
        if (n + 3 < p.n) {
            *reinterpret_cast<u32x2_a2 *>(y) = u32x2{bf16_pack2(v[0], v[1]), bf16_pack2(v[2], v[3])};
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (n + e < p.n)
                    y[e] = (uint16_t)f32_to_bf16_rne(v[e]);
        }
    }
}

// Scales and bias of features n .. n + 3; those past the last are not used.
__device__ __attribute__((always_inline)) inline void feature_terms(const LinearParams &p, int n, f32x4 &sw, f32x4 &bias)
{
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int i = min(n + e, p.n - 1);
        sw[e] = p.sw[i];
        bias[e] = p.bias ? p.bias[i] : 0.0f;
    }
}

}  // namespace igc
