// Linear layer of few outputs: 16 features x 16 tokens a workgroup, for grids that
// the LDS tiles would leave mostly empty, and for a few tokens over a weight that
// comes from HBM. The time is one pass over the codes.
//
// A workgroup's 8 waves take the 128-byte reduction steps in turn, wave w steps w,
// w + 8, ... Every byte of its operands is used by one wave only, so it goes
// straight from memory (or the caches) into the registers of the matrix
// instruction, without LDS. The waves' sums meet in LDS at the end and are added in
// wave order. No workspace and no second launch. Against the best other tile, weights
// from HBM (enough of them in turn that no cache holds one): 1 x 1280 x 5120 int8 6.6
// us, 8.4 on 32 x 32 tiles; 1 x 8192 x 8192 fp8 14.9 and 16.1 us; 1 x 32768 x 8192
// 47.4, 5.7 TB/s, and 55.4. Weights that the 256 MB cache holds: 5.1 and 6.4, 12.8
// and 12.3 us; the last is too large for that. Loading a second register set ahead
// lost 1 us.
#include "linear.h"

namespace igc {

__device__ __attribute__((always_inline)) inline i32x4 buffer_load16(__amdgpu_buffer_rsrc_t r, unsigned off)
{
    return __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
}

// The 128 codes of a step from a lane's chunks g and g + 4 of both operands.
template <Elem T, bool PRECISE, typename Acc>
__device__ __attribute__((always_inline)) inline void mma_step(const i32x4 (&w)[2], const i32x4 (&a)[2], Acc &c)
{
    if constexpr (T == E_INT8) {
        c = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[0], a[0], c, 0, 0, 0);
        c = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[1], a[1], c, 0, 0, 0);
    } else if constexpr (PRECISE) {
        using M = Mma<E_FP8, true>;
        M::mma(M::widen(w[0]), M::widen(a[0]), c);
        M::mma(M::widen(w[1]), M::widen(a[1]), c);
    } else {
        const i32x8 x = {w[0][0], w[0][1], w[0][2], w[0][3], w[1][0], w[1][1], w[1][2], w[1][3]};
        const i32x8 y = {a[0][0], a[0][1], a[0][2], a[0][3], a[1][0], a[1][1], a[1][2], a[1][3]};
        c = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, c, 0, 0, 0, 0, 0, 0);
    }
}

template <Elem T, Elem OUT>
__global__ __launch_bounds__(kSkinnyWaves * 64) void linear_skinny_kernel(LinearParams p)
{
    constexpr int NW = kSkinnyWaves, U = kSkinnyLoads;
    using Acc = typename Mma<T, OUT == E_F32>::Acc;
    __shared__ Acc part[NW][64];
    const int lane = threadIdx.x & 63, lrow = lane & 15, lgrp = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int tm = blockIdx.x / p.tiles_n, n0 = (blockIdx.x - tm * p.tiles_n) * kSkinnyFeatures, m0 = tm * kSkinnyTokens;
    // rows past the last lie past the end of these buffers and read as zeros, without memory traffic
    const __amdgpu_buffer_rsrc_t wr = buffer_rsrc(static_cast<const char *>(p.w) + (int64_t)n0 * p.ldw,
                                                  (int)(min(kSkinnyFeatures, p.n - n0) * p.ldw));
    const __amdgpu_buffer_rsrc_t ar = buffer_rsrc(static_cast<const char *>(p.a) + (int64_t)m0 * p.lda,
                                                  (int)(min(kSkinnyTokens, p.m - m0) * p.lda));
    const unsigned wbase = (unsigned)lrow * (unsigned)p.ldw + lgrp * 16;
    const unsigned abase = (unsigned)lrow * (unsigned)p.lda + lgrp * 16;

    Acc acc{};
    for (int s = wave; s < p.nk; s += NW * U) {
        i32x4 w[U][2], a[U][2];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int step = s + u * NW;
            const bool in = step < p.nk;  // so does a step past the last
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                w[u][c] = buffer_load16(wr, in ? wbase + step * 128 + c * 64 : kPastEnd);
                a[u][c] = buffer_load16(ar, in ? abase + step * 128 + c * 64 : kPastEnd);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            mma_step<T, OUT == E_F32>(w[u], a[u], acc);
    }
    part[wave][lane] = acc;
    __syncthreads();
    if (wave != 0)
        return;
#pragma unroll
    for (int w = 1; w < NW; ++w)
        acc += part[w][lane];
    const int n = n0 + 4 * lgrp, m = m0 + lrow;
    if (m < p.m && n < p.n) {
        f32x4 fs, fb;
        feature_terms(p, n, fs, fb);
        store_outputs<OUT>(p, m, n, scaled(acc, p.sa[m], fs, fb));
    }
}

hipError_t launch_linear_skinny(const LinearParams &p, Elem t, Elem out, hipStream_t stream)
{
    const dim3 grid((unsigned)p.tiles_m * p.tiles_n), block(kSkinnyWaves * 64);
    if (t == E_INT8) {
        if (out == E_F32)
            hipLaunchKernelGGL((linear_skinny_kernel<E_INT8, E_F32>), grid, block, 0, stream, p);
        else
            hipLaunchKernelGGL((linear_skinny_kernel<E_INT8, E_BF16>), grid, block, 0, stream, p);
    } else {
        if (out == E_F32)
            hipLaunchKernelGGL((linear_skinny_kernel<E_FP8, E_F32>), grid, block, 0, stream, p);
        else
            hipLaunchKernelGGL((linear_skinny_kernel<E_FP8, E_BF16>), grid, block, 0, stream, p);
    }
    return hipGetLastError();
}

}  // namespace igc
