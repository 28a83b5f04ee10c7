"""Products of fp8 codes whose largest terms cancel: with an fp32 output the small rest is right to fp32's roundings, with
a bf16 output to what the header states, 2^-11 of the largest product for every 128 codes; int8 is exact.

Every case prints its name before touching the GPU.
"""

import numpy as np
import pytest
import torch

from implicit_gemm_convolution_conv_amd import binding as B

import token_ref as R

pytestmark = pytest.mark.gpu

DEV = R.DEV


@pytest.mark.parametrize("tile", [-1, 0, 1, 2, 3, 4, 5, 6, 7])
@pytest.mark.parametrize("kind", [B.IGC_INT8, B.IGC_FP8_E4M3FN])
def test_outlier_channels_of_opposite_signs(kind, tile):
    m, n, k = 40, 72, 1280
    print(f"[case] cancelling outliers kind={kind} tile={tile}", flush=True)
    g = torch.Generator().manual_seed(3)
    top = R.TOP[kind]
    a, w = torch.randint(-3, 4, (m, k), generator=g).float(), torch.randint(-3, 4, (n, k), generator=g).float()
    if kind == B.IGC_FP8_E4M3FN:
        a, w = a / 4, w / 4
    for at, sign in ((5, 1.0), (77, -1.0), (600, 1.0), (1210, -1.0)):  # within one step of 128, and far apart
        a[:, at], w[:, at] = top, sign * top
    aq, wq = a.to(R.TORCH[kind]).to(DEV), w.to(R.TORCH[kind]).to(DEV)
    sa, sw = torch.full((m,), 0.5, device=DEV), torch.full((n,), 0.25, device=DEV)
    exact = (a.double() @ w.double().t()).numpy() / 8
    B.linear_debug_force(tile, 0)
    try:
        for y_dtype in (B.IGC_F32, B.IGC_BF16):
            y = torch.full((m, n), float("nan"), dtype=R.TORCH[y_dtype], device=DEV)
            B.linear_fwd(aq, k, sa, wq, k, sw, None, y, n, m, n, k, kind, y_dtype)
            torch.cuda.synchronize()
            err = np.abs(R.f64(y) - exact)
            if kind == B.IGC_INT8:
                bound = R.round_bound(exact, y_dtype, 0)
            elif y_dtype == B.IGC_F32:
                # one fp32 rounding of sums below 2^19 for each instruction of 32 products
                bound = (k // 32) * 2.0 ** (18 - 24) / 8
            else:
                bound = (k // 128) * 2.0 ** -11 * top * top / 8 + R.round_bound(exact, y_dtype, 1)
            print(f"y_dtype={y_dtype}: off by {err.max():.4g} beside results of {np.abs(exact).max():.4g}", flush=True)
            assert np.all(err <= bound), (y_dtype, err.max())
    finally:
        B.linear_debug_force()
