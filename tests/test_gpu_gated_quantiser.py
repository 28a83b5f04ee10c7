"""The gated quantiser at gates far below zero, where silu decays to nothing: down to the type's lowest value (a masked
gate), alone in a row, beside ordinary ones and under large factors, against the 64-bit form.

Bound: below -80 the value is (g e)(e u) with e = exp(g / 2), twice an exponential's 3 roundings and 3 products; 16
roundings cover it and the ordinary gates' 8.

Every case prints its name before touching the GPU.
"""

import numpy as np
import pytest
import torch

from implicit_gemm_convolution_conv_amd import binding as B

import token_ref as R

pytestmark = pytest.mark.gpu

DEV = R.DEV


def _gated(gate, up, dtype, kind, name):
    """Codes (as numbers) and scales of the rows silu(gate) * up, after the check against the 64-bit form."""
    x = torch.cat([gate, up], 1).to(dtype).to(DEV)
    rows, cols = gate.shape
    q = torch.empty((rows, B.linear_packed_cols(cols)), dtype=R.TORCH[kind], device=DEV)
    s = torch.empty((rows,), device=DEV)
    B.linear_quant(x, 2 * cols, q, q.stride(0), s, rows, cols, B.IGC_BF16 if dtype == torch.bfloat16 else B.IGC_F32,
                   kind, B.IGC_ACT_SILU_GLU)
    torch.cuda.synchronize()
    codes = q[:, :cols]
    assert torch.isfinite(codes.float()).all() and torch.isfinite(s).all(), name
    with np.errstate(all="ignore"):
        R.check_codes(codes, s, R.silu_glu(R.f64(x), cols), kind, 16, name)
    return codes.float().cpu(), s.cpu()


@pytest.mark.parametrize("kind", [B.IGC_INT8, B.IGC_FP8_E4M3FN])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("cols", [13, 200, 2047, 33001])
def test_gates_far_below_zero(cols, dtype, kind):
    print(f"[case] gates far below zero cols={cols} {dtype} kind={kind}", flush=True)
    g = torch.Generator().manual_seed(cols)
    lowest = torch.finfo(dtype).min
    far = torch.tensor([lowest, -1e36, -1e30, -1e10, -1e5, -1000.0, -200.0, -174.0])

    def some(values):
        return values[torch.randint(0, len(values), (cols,), generator=g)]

    ordinary, up = torch.randn(cols, generator=g), torch.randn(cols, generator=g)
    mixed = torch.where(torch.rand(cols, generator=g) < 0.3, some(far), ordinary)
    mixed[0], up[0] = 0.5, 1.0
    big = torch.full((cols,), 1e38) * (1 + torch.rand(cols, generator=g))
    tail = -88.0 - 16.0 * torch.rand(cols, generator=g)
    edge = -80.0 + torch.randn(cols, generator=g)
    rows = [(mixed, up), (some(far), up), (some(far), big), (tail, big), (edge, big), (edge, up),
            (torch.full((cols,), lowest), torch.full((cols,), lowest)), (ordinary, up)]
    codes, scales = _gated(torch.stack([r[0] for r in rows]), torch.stack([r[1] for r in rows]), dtype, kind, f"cols={cols}")
    for i in (1, 2, 6):  # next to nothing is left of these rows: the least scale, zero codes
        assert abs(float(scales[i]) * R.TOP[kind] / R.TINY - 1) < 1e-6, i
        # (in row 2 a gate of -174 under 1e38 leaves 5e-36, a least code or two in fp8)
        assert i == 2 or bool((codes[i] == 0).all()), i


def test_one_masked_gate_leaves_its_row_alone():
    """The codes of a row do not change when a gate whose value is about zero becomes the type's lowest."""
    print("[case] one masked gate", flush=True)
    g = torch.Generator().manual_seed(4)
    gate, up = torch.randn((4, 640), generator=g), torch.randn((4, 640), generator=g)
    gate[:, 100] = -170.0
    masked = gate.clone()
    masked[:, 100] = torch.finfo(torch.bfloat16).min
    for kind in (B.IGC_INT8, B.IGC_FP8_E4M3FN):
        a, b = (_gated(m, up, torch.bfloat16, kind, "masked") for m in (gate, masked))
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
