"""Token operators in HIP graphs at sizes whose calls are more than one launch: products with a split reduction, gradients
with one workgroup, with few and with many parts of dw. Every replay, with new inputs and eager work between, equals the
eager calls bit for bit.

Every case prints its name before touching the GPU.
"""

import pytest
import torch

from implicit_gemm_convolution_conv_amd import binding as B

import token_ref as R

pytestmark = pytest.mark.gpu

DEV = R.DEV


@pytest.mark.parametrize("kind", [B.IGC_INT8, B.IGC_FP8_E4M3FN])
@pytest.mark.parametrize("dtype", [B.IGC_BF16, B.IGC_F32])
@pytest.mark.parametrize("m,d,n", [(1, 1280, 5120), (100, 8192, 1280), (700, 2049, 129), (2050, 1291, 640), (4200, 96, 33)])
def test_replays_match_eager(m, d, n, dtype, kind):
    print(f"[case] graph {m}x{d} to {n} dtype={dtype} kind={kind}", flush=True)
    g = torch.Generator(device=DEV)
    g.manual_seed(m + d + n)

    def draw(rows, cols):
        return torch.randn((rows, cols), generator=g, device=DEV).to(R.TORCH[dtype])

    x, r, dy, nw = draw(m, d), draw(m, d), draw(m, d), draw(1, d)[0].contiguous()
    kp, hp = B.linear_packed_cols(d), B.linear_packed_cols(n // 2)
    w, sw = torch.empty((n, kp), dtype=R.TORCH[kind], device=DEV), torch.empty((n,), device=DEV)
    B.linear_quant(draw(n, d), d, w, kp, sw, n, d, dtype, kind)
    product, grads = B.linear_fwd_workspace_bytes(m, n, d, kind, dtype), B.norm_bwd_workspace_bytes(m, d)
    assert (m, d) != (100, 8192) or product > 0  # that one splits its reduction
    ws = torch.empty((max(product, grads),), dtype=torch.uint8, device=DEV)

    def outputs():
        return {"h": torch.empty_like(x), "q": torch.empty((m, kp), dtype=R.TORCH[kind], device=DEV),
                "s": torch.empty((m,), device=DEV), "y": torch.empty((m, n), dtype=R.TORCH[dtype], device=DEV),
                "q2": torch.empty((m, hp), dtype=R.TORCH[kind], device=DEV), "s2": torch.empty((m,), device=DEV),
                "dx": torch.empty_like(x), "dw": torch.empty((d,), device=DEV)}

    def calls(o):
        B.norm_fwd(x, d, r, d, nw, o["h"], d, o["q"], kp, o["s"], m, d, 1e-6, dtype, kind)
        B.linear_fwd(o["q"], kp, o["s"], w, kp, sw, None, o["y"], n, m, n, d, kind, dtype, ws)
        B.linear_quant(o["y"], n, o["q2"], hp, o["s2"], m, n // 2, dtype, kind, B.IGC_ACT_SILU_GLU)
        B.norm_bwd(dy, d, o["h"], d, nw, r, d, o["dx"], d, o["dw"], m, d, 1e-6, dtype, ws)

    static, eager = outputs(), outputs()
    calls(static)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls(static)
    for _ in range(3):
        x.copy_(draw(m, d))
        dy.copy_(draw(m, d))
        torch.cuda.synchronize()
        for o in static.values():
            o.view(torch.uint8).fill_(0x5A)
        graph.replay()
        torch.cuda.synchronize()
        calls(eager)
        torch.cuda.synchronize()
        for key in static:
            assert torch.equal(static[key].view(torch.uint8), eager[key].view(torch.uint8)), key
    del graph
