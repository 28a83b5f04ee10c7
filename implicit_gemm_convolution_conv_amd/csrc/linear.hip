// Linear layer, tiles staged through LDS (linear.h has the operator).
#include "linear.h"

namespace igc {

// Workgroup -> tile: workgroups go to the 8 XCDs round-robin; renumbered so that
// neighbouring tiles share an XCD's L2, then walked in groups of p.group token
// tiles, all feature tiles of a group before the next.
__device__ __attribute__((always_inline)) inline void linear_tile_of(const LinearParams &p, int bid, int &tm, int &tn)
{
    const int nblk = p.tiles_m * p.tiles_n;
    const int xcd = bid & 7, idx = bid >> 3, q = nblk >> 3, r = nblk & 7;
    const int lin = xcd * q + min(xcd, r) + idx;
    const int gsz = p.group * p.tiles_n;
    const int g = lin / gsz, in = lin - g * gsz;
    const int rows = min(p.tiles_m - g * p.group, p.group);
    tn = in / rows;
    tm = g * p.group + in - tn * rows;
}

// Four neighbouring words (those of `left` features) of a split's partial sums.
__device__ __attribute__((always_inline)) inline void store_part(int *dst, int left, const i32x4 &v)
{
    if (left >= 4) {
        *reinterpret_cast<i32x4_a4 *>(dst) = v;
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (e < left)
                dst[e] = v[e];
    }
}

// 16 bytes of token m's outputs from feature n on (those of features below p.n), 8 bf16 or 4 fp32.
template <Elem OUT>
__device__ __attribute__((always_inline)) inline void store_piece(const LinearParams &p, int m, int n, const i32x4 &v)
{
    using U = typename std::conditional<OUT == E_BF16, uint16_t, uint32_t>::type;
    using V = typename std::conditional<OUT == E_BF16, i32x4_a2, i32x4_a4>::type;
    constexpr int PER = 16 / sizeof(U);
    U *dst = static_cast<U *>(p.y) + (int64_t)m * p.ldy + n;
    if (n + PER <= p.n) {
        *reinterpret_cast<V *>(dst) = v;
    } else {
#pragma unroll
        for (int e = 0; e < PER; ++e)
            if (n + e < p.n)
                dst[e] = OUT == E_BF16 ? (U)((unsigned)v[e >> 1] >> (16 * (e & 1))) : (U)v[e];
    }
}

// A workgroup computes BN features x BM tokens, WN x WM waves of 16 x 16 blocks.
// Rings of SW (features) and SA (tokens) stages of 128-byte steps in LDS, filled
// by buffer loads; rows past the last read as zeros, the buffer of each tile ends
// with its last row. Step ks: wait until this thread's loads of step ks have
// landed, barrier (the step is visible and the slots of step ks - 1 are no longer
// read), then compute while issuing A(ks + SA - 1) and W(ks + SW - 1) into those
// slots, spread over the step's first SPREAD rows of blocks.
//
// What bounds it: large products the power the matrix units draw (8192^3 fp8 403 us,
// 2730 TFLOP/s, int8 419 us, 2620 TOP/s, the units 67 % busy at 2.0 and 1.8 GHz; on
// codes that are all zero 355 and 342 us; fp8 widened for fp32 outputs 750 us, 1470
// TFLOP/s); short reductions their outputs as well
// (9500 x 10240 x 1280 int8 to bf16 135 us, of which writing 195 MB takes 44; the
// fewer the steps, the more: 8000 x 8000 x 512 int8 to fp32 84 us, 264 MB, one
// workgroup a CU whose outputs go with no loads beside them); few tokens the weight's
// way into the CUs (48 x 8192 x 8192 fp8 19 us from HBM, 3.5 TB/s; 13 to 14 us where
// the 256 MB cache holds the weight); small ones a launch and the latency of each step
// (777 x 1283 x 1291 int8 to fp32, 64 x 128 tiles, 7.1 us, 11 steps of 0.3 us after
// 1.7).
template <Elem T, Elem OUT, int BN, int BM, int WN, int WM, int SW, int SA, int SPREAD>
__global__ __launch_bounds__(WN *WM * 64) void linear_tile_kernel(LinearParams p)
{
    constexpr int NW = WN * WM, NT = NW * 64, KB = 128;
    constexpr int WIT = BN / (8 * NW), AIT = BM / (8 * NW);  // 8 rows a load instruction
    constexpr int LPS = WIT + AIT;
    constexpr int FN = BN / WN / 16, FM = BM / WM / 16;
    constexpr int WSTAGE = BN * KB, ASTAGE = BM * KB;
    using M = Mma<T, OUT == E_F32>;
    using Acc = typename M::Acc;
    constexpr int ROWS = M::kSlices * FN;
    constexpr bool WIDENED = T == E_FP8 && OUT == E_F32;
    static_assert(SW == SA || SW == SA + 1, "the features' ring is the deeper one");
    static_assert(SPREAD >= 1 && SPREAD <= ROWS, "loads spread within a step");
    constexpr int RING = SW * WSTAGE + SA * ASTAGE;
    // outputs leave through LDS, [token][feature] rows of OS bytes, in as many passes over the tokens as fit
    constexpr int ES = OUT == E_BF16 ? 2 : 4, OS = ES * BN + 16;
    constexpr int PASSES = BM * OS <= RING ? 1 : 2, BMP = BM / PASSES;
    static_assert(BMP * OS <= RING && WM % PASSES == 0, "a pass takes whole waves");
    __shared__ __attribute__((aligned(1024))) char smem[RING];
    char *const ws = smem, *const as = smem + SW * WSTAGE;

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wn = wave % WN, wm = wave / WN;
    const int ntiles = p.tiles_m * p.tiles_n;
    const int split = blockIdx.x / ntiles;
    int tm, tn;
    linear_tile_of(p, blockIdx.x - split * ntiles, tm, tn);
    const int n0 = tn * BN, m0 = tm * BM;
    const int kbeg = split * p.ksplit, nk = min(p.nk, kbeg + p.ksplit) - kbeg;

    const int lr = lane >> 3, jc = (lane & 7) ^ lr;  // row r keeps chunk q at slot q ^ (r & 7)
    const __amdgpu_buffer_rsrc_t wr =
        buffer_rsrc(static_cast<const char *>(p.w) + (int64_t)n0 * p.ldw, (int)(min(BN, p.n - n0) * p.ldw));
    const __amdgpu_buffer_rsrc_t ar =
        buffer_rsrc(static_cast<const char *>(p.a) + (int64_t)m0 * p.lda, (int)(min(BM, p.m - m0) * p.lda));
    unsigned woff[WIT], aoff[AIT];
#pragma unroll
    for (int i = 0; i < WIT; ++i)
        woff[i] = (unsigned)(8 * (wave + i * NW) + lr) * (unsigned)p.ldw + jc * 16 + kbeg * KB;
#pragma unroll
    for (int i = 0; i < AIT; ++i)
        aoff[i] = (unsigned)(8 * (wave + i * NW) + lr) * (unsigned)p.lda + jc * 16 + kbeg * KB;
    // load instruction j of a step, A rows first: A step `sa` into slot sta, W step `sw` into slot stw
    auto issue = [&](int j, int sta, int stw, int sa, int sw) __attribute__((always_inline)) {
        if (j < AIT)
            buffer_to_lds16(ar, as + sta * ASTAGE + 8 * (wave + j * NW) * KB, aoff[j] + sa * KB);
        else
            buffer_to_lds16(wr, ws + stw * WSTAGE + 8 * (wave + (j - AIT) * NW) * KB, woff[j - AIT] + sw * KB);
    };
    auto issue_a = [&](int st, int step) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < AIT; ++j)
            issue(j, st, 0, step, 0);
    };
    auto issue_w = [&](int st, int step) __attribute__((always_inline)) {
#pragma unroll
        for (int j = AIT; j < LPS; ++j)
            issue(j, 0, st, 0, step);
    };

    Acc acc[FN][FM];
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
        for (int j = 0; j < FM; ++j)
            acc[i][j] = Acc{};
    const int lrow = lane & 15, lgrp = lane >> 4, lsw = lrow & 7;
    auto compute = [&](int sta, int stw, auto &&hook) __attribute__((always_inline)) {
        const char *wp = ws + stw * WSTAGE + (wn * (BN / WN) + lrow) * KB;
        const char *ap = as + sta * ASTAGE + (wm * (BM / WM) + lrow) * KB;
        if constexpr (FN * FM <= (WIDENED ? 8 : 2)) {
            // all of the step's fragments first, its loads go out while these arrive: widened ones, a wait and 8
            // conversions each, gain 10 to 35 %, int8 on 32 x 64 tiles up to 7 %; 64 x 128 int8 lost 5 %
            typename M::Frag af[M::kSlices][FM], wf[M::kSlices][FN];
#pragma unroll
            for (int h = 0; h < M::kSlices; ++h) {
#pragma unroll
                for (int j = 0; j < FM; ++j)
                    af[h][j] = M::frag(ap + j * 16 * KB, h, lgrp, lsw);
#pragma unroll
                for (int i = 0; i < FN; ++i)
                    wf[h][i] = M::frag(wp + i * 16 * KB, h, lgrp, lsw);
            }
#pragma unroll
            for (int row = 0; row < ROWS; ++row)
                hook(row);
#pragma unroll
            for (int h = 0; h < M::kSlices; ++h)
#pragma unroll
                for (int i = 0; i < FN; ++i)
#pragma unroll
                    for (int j = 0; j < FM; ++j)
                        M::mma(wf[h][i], af[h][j], acc[i][j]);
        } else if constexpr (WIDENED) {
#pragma unroll
            for (int h = 0; h < M::kSlices; ++h) {
                // one feature fragment read ahead, so that its conversions do not wait for LDS: 8192^3 750 us, 995 us
                // without; two ahead are no faster, four do not fit the registers
                i32x4 an[FM], next = M::narrow(wp, h, lgrp, lsw);
                typename M::Frag af[FM];
#pragma unroll
                for (int j = 0; j < FM; ++j)
                    an[j] = M::narrow(ap + j * 16 * KB, h, lgrp, lsw);
#pragma unroll
                for (int j = 0; j < FM; ++j)
                    af[j] = M::widen(an[j]);
#pragma unroll
                for (int i = 0; i < FN; ++i) {
                    const typename M::Frag wf = M::widen(next);
                    if (i + 1 < FN)
                        next = M::narrow(wp + (i + 1) * 16 * KB, h, lgrp, lsw);
#pragma unroll
                    for (int j = 0; j < FM; ++j)
                        M::mma(wf, af[j], acc[i][j]);
                    hook(h * FN + i);
                }
            }
        } else {
#pragma unroll
            for (int h = 0; h < M::kSlices; ++h) {
                typename M::Frag af[FM];
#pragma unroll
                for (int j = 0; j < FM; ++j)
                    af[j] = M::frag(ap + j * 16 * KB, h, lgrp, lsw);
#pragma unroll
                for (int i = 0; i < FN; ++i) {
                    const typename M::Frag wf = M::frag(wp + i * 16 * KB, h, lgrp, lsw);
#pragma unroll
                    for (int j = 0; j < FM; ++j)
                        M::mma(wf, af[j], acc[i][j]);
                    hook(h * FN + i);
                }
            }
        }
    };

    // steps before the first, in the order of the steady state
#pragma unroll
    for (int j = -(SW - 1); j < 0; ++j) {
        if (j + SA - 1 >= 0 && j + SA - 1 < nk)
            issue_a(j + SA - 1, j + SA - 1);
        if (j + SW - 1 < nk)
            issue_w(j + SW - 1, j + SW - 1);
    }
    constexpr int AHEAD = (SW == SA ? 0 : WIT) + (SA - 2) * LPS;  // loads issued after a step's last one
    int ks = 0, sa = 0, sw = 0, ia = SA - 1, iw = SW - 1;
    auto next = [&]() __attribute__((always_inline)) {
        sa = sa + 1 == SA ? 0 : sa + 1;
        ia = ia + 1 == SA ? 0 : ia + 1;
        sw = sw + 1 == SW ? 0 : sw + 1;
        iw = iw + 1 == SW ? 0 : iw + 1;
    };
    for (; ks < nk - SW + 1; ++ks) {
        wait_vmcnt<AHEAD>();
        // this wave's LDS reads of step ks - 1 are done too, wherever its last MFMAs were scheduled
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        compute(sa, sw, [&](int row) __attribute__((always_inline)) {
#pragma unroll
            for (int j = 0; j < LPS; ++j)
                if (j * SPREAD / LPS == row)
                    issue(j, ia, iw, ks + SA - 1, ks + SW - 1);
        });
        next();
    }
    for (; ks < nk; ++ks) {
        wait_vmcnt<0>();
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        if (ks + SA - 1 < nk)
            issue_a(ia, ks + SA - 1);
        if (ks + SW - 1 < nk)
            issue_w(iw, ks + SW - 1);
        compute(sa, sw, [](int) {});
        next();
    }

    if (p.splits > 1) {
        int *part = static_cast<int *>(p.part) + (int64_t)split * p.m * p.n;
#pragma unroll
        for (int i = 0; i < FN; ++i) {
            const int n = n0 + wn * (BN / WN) + i * 16 + 4 * lgrp;
#pragma unroll
            for (int j = 0; j < FM; ++j) {
                const int m = m0 + wm * (BM / WM) + j * 16 + lrow;
                if (m < p.m && n < p.n)
                    store_part(part + (int64_t)m * p.n + n, p.n - n, __builtin_bit_cast(i32x4, acc[i][j]));
            }
        }
        return;
    }
    float scale[FM];
#pragma unroll
    for (int j = 0; j < FM; ++j)
        scale[j] = p.sa[min(m0 + wm * (BM / WM) + j * 16 + lrow, p.m - 1)];
    constexpr int PER = 16 / ES, PIECES = BN / PER;  // outputs of a 16-byte piece, pieces of a token's row
#pragma unroll
    for (int pass = 0; pass < PASSES; ++pass) {
        __syncthreads();  // every wave has finished reading the rings, or the pass before
        if (PASSES == 1 || wm / (WM / PASSES) == pass) {
#pragma unroll
            for (int i = 0; i < FN; ++i) {
                const int col = wn * (BN / WN) + i * 16 + 4 * lgrp;
                f32x4 fs, fb;
                feature_terms(p, n0 + col, fs, fb);
#pragma unroll
                for (int j = 0; j < FM; ++j) {
                    const int row = wm * (BM / WM) + j * 16 + lrow - pass * BMP;
                    const f32x4 o = scaled(acc[i][j], scale[j], fs, fb);
                    if constexpr (OUT == E_BF16)
                        *reinterpret_cast<u32x2 *>(smem + row * OS + col * 2) = u32x2{bf16_pack2(o[0], o[1]), bf16_pack2(o[2], o[3])};
                    else
                        *reinterpret_cast<f32x4 *>(smem + row * OS + col * 4) = o;
                }
            }
        }
        __syncthreads();
#pragma unroll
        for (int it = 0; it < (BMP * PIECES + NT - 1) / NT; ++it) {
            const int idx = it * NT + (int)threadIdx.x, row = idx / PIECES, n = n0 + (idx % PIECES) * PER;
            const int m = m0 + pass * BMP + row;
            if (row >= BMP || m >= p.m || n >= p.n)
                continue;
            store_piece<OUT>(p, m, n, *reinterpret_cast<const i32x4 *>(smem + row * OS + (idx % PIECES) * 16));
        }
    }
}

// Adds the splits' sums in split order and writes the outputs, four neighbouring
// features a thread. A launch and one pass over the sums, which the caches hold:
// 333 x 640 x 10240 int8 in 4 splits takes 13.0 us with it, 19.0 us unsplit on the same
// tile; 64 x 64 x 65536 in 16 splits 13.8 us, 60 us unsplit.
template <Elem T, Elem OUT>
__global__ __launch_bounds__(256) void linear_reduce_kernel(LinearParams p)
{
    using Acc = typename Mma<T, false>::Acc;
    const int quads = (p.n + 3) >> 2;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int m = (int)(i / quads), n = 4 * (int)(i - (int64_t)m * quads);
    if (m >= p.m)
        return;
    Acc acc{};
    for (int s = 0; s < p.splits; ++s) {
        const int *src = static_cast<const int *>(p.part) + ((int64_t)s * p.m + m) * p.n + n;
        i32x4 v = {0, 0, 0, 0};
        if (n + 3 < p.n) {
            v = *reinterpret_cast<const i32x4_a4 *>(src);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (n + e < p.n)
                    v[e] = src[e];
        }
        acc += __builtin_bit_cast(Acc, v);
    }
    f32x4 sw, bias;
    feature_terms(p, n, sw, bias);
    store_outputs<OUT>(p, m, n, scaled(acc, p.sa[m], sw, bias));
}

// Waves of a 256 x 256 tile: 64 features x 128 tokens each (2 % ahead of 128 x 64
// on int8, even on fp8), 128 x 64 where fp8 is widened, whose fragments would not
// fit the registers otherwise. Rings: 3 + 2 stages of 32 KB are the whole LDS; the
// smaller tiles keep 3 to 8 stages in flight, since a few resident waves have to
// cover the memory latency by themselves (64 x 64 with 8 waves and 4 stages 16.9 us,
// with 4 waves 17.9 us on 100 x 8192 x 8192 int8; 128 x 128 with 8 waves and 4 stages
// 11.0 us, 4 waves and 3 + 2 stages 15.1 us on 1500 x 2048 x 2048).
template <Elem T, Elem OUT>
static hipError_t launch_typed(const LinearParams &p, int tile, hipStream_t stream)
{
    const dim3 grid((unsigned)p.tiles_m * p.tiles_n * p.splits);
    constexpr bool WIDENED = T == E_FP8 && OUT == E_F32;
#define IGC_LINEAR(TILE, BN_, BM_, WN_, WM_, SW_, SA_, SP_)                                                          \
    case TILE:                                                                                                      \
        hipLaunchKernelGGL((linear_tile_kernel<T, OUT, BN_, BM_, WN_, WM_, SW_, SA_, SP_>), grid,               \
                           dim3(WN_ * WM_ * 64), 0, stream, p);                                                     \
        return hipGetLastError()
    switch (tile) {
        IGC_LINEAR(LT_256, 256, 256, (WIDENED ? 2 : 4), (WIDENED ? 4 : 2), 3, 2, 4);
        IGC_LINEAR(LT_256x128, 256, 128, 4, 2, 3, 3, 4);
        IGC_LINEAR(LT_128, 128, 128, 4, 2, 4, 4, 2);
        IGC_LINEAR(LT_64x128, 64, 128, 4, 2, 4, 4, 1);
        IGC_LINEAR(LT_64, 64, 64, 4, 2, 4, 4, 1);
        IGC_LINEAR(LT_32x64, 32, 64, 2, 2, 6, 6, 1);
        IGC_LINEAR(LT_32, 32, 32, 2, 2, 8, 8, 1);
    default: return hipErrorInvalidValue;
    }
#undef IGC_LINEAR
}

hipError_t launch_linear(const LinearParams &p, int tile, Elem t, Elem out, hipStream_t stream)
{
    if (t == E_INT8)
        return out == E_F32 ? launch_typed<E_INT8, E_F32>(p, tile, stream) : launch_typed<E_INT8, E_BF16>(p, tile, stream);
    return out == E_F32 ? launch_typed<E_FP8, E_F32>(p, tile, stream) : launch_typed<E_FP8, E_BF16>(p, tile, stream);
}

hipError_t launch_linear_reduce(const LinearParams &p, Elem t, Elem out, hipStream_t stream)
{
    const int64_t work = (int64_t)p.m * ((p.n + 3) / 4);
    const dim3 grid((unsigned)((work + 255) / 256));
    if (t == E_INT8) {
        if (out == E_F32)
            hipLaunchKernelGGL((linear_reduce_kernel<E_INT8, E_F32>), grid, dim3(256), 0, stream, p);
        else
            hipLaunchKernelGGL((linear_reduce_kernel<E_INT8, E_BF16>), grid, dim3(256), 0, stream, p);
    } else {
        if (out == E_F32)
            hipLaunchKernelGGL((linear_reduce_kernel<E_FP8, E_F32>), grid, dim3(256), 0, stream, p);
        else
            hipLaunchKernelGGL((linear_reduce_kernel<E_FP8, E_BF16>), grid, dim3(256), 0, stream, p);
    }
    return hipGetLastError();
}

}  // namespace igc
