"""The 8-bit codes of the row quantiser, bit for bit, against the formula in 32 bits on the CPU: scale = a / top,
code = the nearest to fp32(v * fp32(top / a)), ties to even. Rows of bf16 values hold exact ties (v = a / 2 lies on 63.5).

Every case prints its name before touching the GPU.
"""

import numpy as np
import pytest
import torch

from implicit_gemm_convolution_conv_amd import binding as B

import token_ref as R

pytestmark = pytest.mark.gpu

DEV = R.DEV


def _quantise(x, kind):
    rows, cols = x.shape
    q = torch.empty((rows, B.linear_packed_cols(cols)), dtype=R.TORCH[kind], device=DEV)
    s = torch.empty((rows,), device=DEV)
    x = x.to(DEV)
    B.linear_quant(x, cols, q, q.stride(0), s, rows, cols, B.IGC_BF16 if x.dtype == torch.bfloat16 else B.IGC_F32, kind)
    torch.cuda.synchronize()
    return q[:, :cols].cpu(), s.cpu()


def _want(x, kind):
    v = x.float().numpy()
    top = np.float32(R.TOP[kind])
    a = np.maximum(np.abs(v).max(axis=1, keepdims=True), np.float32(R.TINY))
    p = v * (top / a)
    assert p.dtype == np.float32
    codes = torch.from_numpy(np.rint(p)).to(torch.int8) if kind == B.IGC_INT8 else torch.from_numpy(p).to(torch.float8_e4m3fn)
    return codes, torch.from_numpy((a / top)[:, 0])


def _same(x, kind, name):
    codes, scales = _quantise(x, kind)
    want, want_scales = _want(x, kind)
    assert torch.equal(scales, want_scales), f"{name}: scales"
    off = codes.view(torch.uint8) != want.view(torch.uint8)
    at = off.nonzero()[:3].tolist()
    assert not off.any(), f"{name}: {int(off.sum())} of {off.numel()} codes, first {[(float(x[i, j]), float(codes[i, j])) for i, j in at]}"


@pytest.mark.parametrize("kind", [B.IGC_INT8, B.IGC_FP8_E4M3FN])
def test_codes_on_ties(kind):
    """Rows whose maximum a runs over every bf16 significand and several exponents, holding a and its halves, and the
    multiples of a / 256 around the other ties."""
    print(f"[case] codes on ties kind={kind}", flush=True)
    a = (1 + torch.arange(128) / 128.0)[:, None] * torch.tensor([2.0 ** -90, 2.0 ** -7, 1.0, 2.0 ** 100])[None, :]
    a = a.reshape(-1, 1)
    x = torch.cat([a, -a / 2, a / 2, a / 4, -a / 4, a / 8, a / 16, a / 512], 1).to(torch.bfloat16)
    _same(x, kind, "bf16 halves")
    odd = torch.arange(1, 254, 2) / 254.0
    _same(torch.cat([a, a * odd, -a * odd], 1), kind, "fp32 ties")


@pytest.mark.parametrize("kind", [B.IGC_INT8, B.IGC_FP8_E4M3FN])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", [(1, 1), (3, 7), (300, 129), (1100, 1280), (5, 5121), (2, 33000)])
def test_codes_of_random_rows(shape, dtype, kind):
    print(f"[case] codes of random rows {shape} {dtype} kind={kind}", flush=True)
    g = torch.Generator().manual_seed(shape[0] + shape[1])
    _same((torch.randn(shape, generator=g) * 3).to(dtype), kind, str(shape))
