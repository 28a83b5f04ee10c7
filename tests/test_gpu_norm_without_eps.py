"""Gradients of the RMS norm with eps = 0, over row counts that do not fill a workgroup's last turn, against the 64-bit
form; and a zero row there, whose gradients are NaN as the formula's are, while other rows keep theirs.

Every case prints its name before touching the GPU.
"""

import numpy as np
import pytest
import torch

from implicit_gemm_convolution_conv_amd import binding as B

import token_ref as R

pytestmark = pytest.mark.gpu

DEV = R.DEV


def _grads(dy, h, w, eps, dtype):
    rows, cols = h.shape
    dx, dw = torch.full_like(h, float("nan")), torch.full((cols,), float("nan"), device=DEV)
    ws = torch.full((B.norm_bwd_workspace_bytes(rows, cols),), 0xFF, dtype=torch.uint8, device=DEV)
    B.norm_bwd(dy, cols, h, cols, w, None, 0, dx, cols, dw, rows, cols, eps, dtype, ws)
    torch.cuda.synchronize()
    return dx, dw


def _inputs(rows, cols, dtype):
    g = torch.Generator(device=DEV)
    g.manual_seed(rows + cols)
    h, dy = (torch.randn((rows, cols), generator=g, device=DEV).to(R.TORCH[dtype]) for _ in range(2))
    return dy, h, (1 + 0.2 * torch.randn((cols,), generator=g, device=DEV)).to(R.TORCH[dtype])


@pytest.mark.parametrize("dtype", [B.IGC_BF16, B.IGC_F32])
@pytest.mark.parametrize("shape", [(1, 1), (1, 64), (17, 128), (5, 200), (9, 256), (3, 512), (1030, 520), (1025, 1291),
                                   (4099, 2048), (1, 1280), (5, 4097), (3, 16384)])
def test_norm_backward_without_eps(shape, dtype):
    rows, cols = shape
    print(f"[case] norm_bwd eps=0 {rows}x{cols} dtype={dtype}", flush=True)
    dy, h, w = _inputs(rows, cols, dtype)
    h[h == 0] = 1  # no row of zeros
    dx, dw = _grads(dy, h, w, 0.0, dtype)
    rdx, rdw, mdx, mdw = R.norm_bwd(R.f64(dy), R.f64(h), R.f64(w), None, 0.0)
    # the row's two means (100 u each) enter every term; then 6 roundings and the result's own
    assert np.all(np.abs(R.f64(dx) - rdx) <= R.round_bound(rdx, dtype, 1) + 256 * R.U * mdx)
    assert np.all(np.abs(R.f64(dw) - rdw) <= (rows + 128) * R.U * mdw + 1e-38)


@pytest.mark.parametrize("dtype", [B.IGC_BF16, B.IGC_F32])
def test_zero_row_without_eps(dtype):
    print(f"[case] norm_bwd eps=0, a zero row, dtype={dtype}", flush=True)
    dy, h, w = _inputs(21, 96, dtype)
    h[7] = 0
    dx, dw = _grads(dy, h, w, 0.0, dtype)
    keep = [i for i in range(21) if i != 7]
    assert torch.isnan(dx[7]).all() and torch.isnan(dw).all()
    rdx, _, mdx, _ = R.norm_bwd(R.f64(dy[keep]), R.f64(h[keep]), R.f64(w), None, 0.0)
    assert np.all(np.abs(R.f64(dx[keep]) - rdx) <= R.round_bound(rdx, dtype, 1) + 256 * R.U * mdx)
    # with an eps the zero row's gradients are finite: dx = w * dy / sqrt(eps), nothing for dw
    dx, dw = _grads(dy, h, w, 1e-4, dtype)
    rdx, rdw, mdx, mdw = R.norm_bwd(R.f64(dy), R.f64(h), R.f64(w), None, float(np.float32(1e-4)))
    assert np.all(np.abs(R.f64(dx) - rdx) <= R.round_bound(rdx, dtype, 1) + 256 * R.U * mdx)
    assert np.all(np.abs(R.f64(dw) - rdw) <= (21 + 128) * R.U * mdw + 1e-38)
