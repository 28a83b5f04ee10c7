"""Codes of the norm and of the quantiser held to the 64-bit form by a check that a NaN cannot pass: token_ref.check_codes
compares with `>`, which is false for a NaN code, so a conversion that overflowed to NaN at a row's maximum would go
unseen there. Without a GPU: the check accepts the nearest codes and nothing else. With one: every row shape.

Every GPU case prints its name before touching the GPU.
"""

import numpy as np
import pytest
import torch

from implicit_gemm_convolution_conv_amd import binding as B

import token_ref as R

INT8, FP8 = B.IGC_INT8, B.IGC_FP8_E4M3FN
KINDS = [INT8, FP8]


def check(codes, scales, v, kind, ulps, name):
    """Scales within their roundings of max|v| / top, every code within half a step (and the error of v) of v / scale."""
    ref = np.maximum(np.abs(v).max(axis=1), R.TINY) / R.TOP[kind]
    s = scales.cpu().double().numpy()
    assert np.all(np.abs(s - ref) <= (ulps + 16) * R.U * ref), f"{name}: scales"
    c, want = R.f64(codes), v / ref[:, None]
    step = 1.0
    if kind == FP8:
        step = 2.0 ** (np.floor(np.log2(np.clip(np.maximum(np.abs(want), np.abs(c)), 2.0 ** -6, 448.0))) - 3)
    near = np.abs(c - want) <= 0.5 * step + 2 * (ulps + 16) * R.U * np.abs(want) + 1e-30
    assert near.all(), f"{name}: {int((~near).sum())} codes are not nearest, first {c[~near][:3]} for {want[~near][:3]}"
    assert np.abs(c).max() <= R.TOP[kind], name


def _nearest(v, kind):
    scale = np.maximum(np.abs(v).max(axis=1, keepdims=True), R.TINY) / R.TOP[kind]
    q = torch.from_numpy(v / scale)
    codes = q.round().to(torch.int8) if kind == INT8 else q.float().to(torch.float8_e4m3fn)
    return codes, torch.from_numpy(scale[:, 0]).float()


@pytest.mark.parametrize("kind", KINDS)
def test_check_accepts_nearest_codes_only(kind):
    v = np.random.default_rng(3).standard_normal((5, 130))
    codes, scales = _nearest(v, kind)
    check(codes, scales, v, kind, 8, "nearest")
    top = codes.view(torch.uint8).clone()
    for row, col in ((0, 0), (4, 129), (2, int(np.abs(v[2]).argmax()))):
        for step in (1, -1):  # a neighbouring code: one step in int8, the next number in fp8
            wrong = top.clone()
            wrong[row, col] = (int(wrong[row, col]) + step) % 256
            with pytest.raises(AssertionError):
                check(wrong.view(codes.dtype), scales, v, kind, 8, "a step off")
    for bad in (float("nan"), float("inf"), float(scales[1]) * 1.001):
        off = scales.clone()
        off[1] = bad
        with pytest.raises(AssertionError):
            check(codes, off, v, kind, 8, "scale")
    if kind == FP8:
        for wrong in (torch.full_like(top, 0x7F), torch.where(top == top[0, 0], 0xFF, top).to(torch.uint8)):
            with pytest.raises(AssertionError):
                check(wrong.view(codes.dtype), scales, v, kind, 8, "NaN codes")


SHAPES = [(1, 1), (3, 7), (5, 128), (70, 200), (9, 512), (1030, 520), (1025, 1291), (1500, 2048), (3, 2047), (33, 4097),
          (7, 6144), (2, 8192), (5, 12288), (3, 16384), (1, 32768)]


def _maximum_everywhere(rows, cols, dtype, seed):
    """Rows whose largest magnitude sits at another place each, over several exponents."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, cols), generator=g) * torch.exp2(torch.randint(-20, 20, (rows, 1), generator=g).float())
    at = (torch.arange(rows) * 7919) % cols
    x[torch.arange(rows), at] = 1.37 * x.abs().amax(1)
    return x.to(R.TORCH[dtype]).cuda()


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", [B.IGC_BF16, B.IGC_F32])
@pytest.mark.parametrize("shape", SHAPES)
def test_every_code_is_a_nearest_one(shape, dtype, kind):
    rows, cols = shape
    print(f"[case] codes {rows}x{cols} dtype={dtype} kind={kind}", flush=True)
    x, up = (_maximum_everywhere(rows, cols, dtype, rows + cols + i) for i in range(2))
    w = (1 + 0.2 * torch.randn((cols,), generator=torch.Generator().manual_seed(cols))).to(R.TORCH[dtype]).cuda()
    wide = B.linear_packed_cols(cols)

    def out():
        return torch.full((rows, wide), 0x7F, dtype=torch.uint8, device="cuda").view(R.TORCH[kind]), \
            torch.full((rows,), float("nan"), device="cuda")

    (nq, ns), (qq, qs), (gq, gs) = out(), out(), out()
    both = torch.cat([x, up], 1)
    B.norm_fwd(x, cols, None, 0, w, None, 0, nq, wide, ns, rows, cols, 1e-6, dtype, kind)
    B.linear_quant(x, cols, qq, wide, qs, rows, cols, dtype, kind)
    B.linear_quant(both, 2 * cols, gq, wide, gs, rows, cols, dtype, kind, B.IGC_ACT_SILU_GLU)
    torch.cuda.synchronize()
    eps = float(np.float32(1e-6))
    check(nq[:, :cols], ns, R.norm(R.f64(x), None, R.f64(w), eps, dtype)[1], kind, 64, "norm")
    check(qq[:, :cols], qs, R.f64(x), kind, 8, "quantiser")
    with np.errstate(all="ignore"):
        check(gq[:, :cols], gs, R.silu_glu(R.f64(both), cols), kind, 16, "gated quantiser")
    for q in (nq, qq, gq):
        assert bool((q[:, cols:].view(torch.uint8) == 0).all()), "padding"
