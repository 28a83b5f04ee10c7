"""Buffers of pipeline.py's sequences belong to the stream that their work runs on: a block that came from another
stream's pool would be handed out again, or still be in use there, while that work runs. Without a GPU: the allocator, the
stream context and the library's launches are replaced by ones that record; with one: calls on a side stream, by handle
and by object, while the current stream allocates and fills blocks of the same sizes."""

import contextlib
import inspect

import pytest
import torch

from implicit_gemm_convolution_conv_amd import binding as B
from implicit_gemm_convolution_conv_amd import pipeline as PL

LAUNCHES = ("norm_fwd", "norm_bwd", "linear_quant", "linear_fwd", "conv_pack_w", "conv_pack_x", "conv_amax",
            "conv_fp8_scales", "conv_fwd")


@pytest.fixture
def recorded(monkeypatch):
    """Names of the launches made; each is checked to have got, of the buffers allocated since, only its own stream's."""
    current, kept, made = [None], {}, []

    @contextlib.contextmanager
    def stream(s):
        before, current[0] = current[0], s
        try:
            yield
        finally:
            current[0] = before

    empty = torch.empty

    def recording_empty(*args, **kw):
        t = empty(*args, **kw)
        kept[t.untyped_storage().data_ptr()] = (t, current[0])  # kept alive, so that no address comes back
        return t

    def launch(name):
        signature = inspect.signature(getattr(B, name))

        def call(*args, **kw):
            bound = signature.bind(*args, **kw).arguments
            for arg, value in bound.items():
                if isinstance(value, torch.Tensor) and value.untyped_storage().data_ptr() in kept:
                    owner = kept[value.untyped_storage().data_ptr()][1]
                    assert owner == bound.get("stream"), f"{name}: {arg} was allocated for stream {owner}"
            made.append(name)
        return call

    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: handle)
    monkeypatch.setattr(torch, "empty", recording_empty)
    for name in LAUNCHES:
        monkeypatch.setattr(B, name, launch(name))
    return made


@pytest.mark.parametrize("stream", [None, 4711])
def test_buffers_belong_to_the_stream(recorded, stream):
    x, r = torch.zeros((100, 8192), dtype=torch.bfloat16), torch.zeros((100, 8192), dtype=torch.bfloat16)
    w = torch.ones((8192,), dtype=torch.bfloat16)
    PL.rms_norm(x, w, r, stream=stream)
    q, _ = PL.rms_norm(x, w, kind="int8", stream=stream)
    PL.rms_norm_grad(x, r, w, stream=stream)
    PL.quantised(x, "fp8", glu=True, stream=stream)
    weight = PL.quantised(torch.zeros((1280, 8192), dtype=torch.bfloat16), "int8", stream=stream)
    assert B.linear_fwd_workspace_bytes(100, 1280, 8192, B.IGC_INT8) > 0  # a split: the product takes a workspace
    PL.linear(q, weight, stream=stream)
    image, taps = torch.zeros((1, 64, 2, 16, 16), dtype=torch.bfloat16), torch.zeros((64, 64, 3, 3, 3), dtype=torch.bfloat16)
    for dtype in ("bf16", "fp8"):
        PL.conv3d(image, taps, pad=(1, 1, 1), dtype=dtype, stream=stream)
    patches, filt = torch.zeros((4, 3, 1, 14, 14), dtype=torch.bfloat16), torch.zeros((64, 3, 1, 14, 14), dtype=torch.bfloat16)
    PL.conv3d(patches, filt, (1, 14, 14), stream=stream)
    assert set(recorded) == set(LAUNCHES)


@pytest.mark.gpu
@pytest.mark.parametrize("handle", [False, True])
def test_sequences_on_a_side_stream(handle):
    print(f"[case] sequences on a side stream, handle={handle}", flush=True)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)

    def draw(rows, cols):
        return torch.randn((rows, cols), generator=g, device="cuda").to(torch.bfloat16)

    x, r, dy, w = draw(100, 8192), draw(100, 8192), draw(100, 8192), draw(1, 8192)[0].contiguous()
    weight = PL.quantised(draw(1280, 8192), "int8")

    def work(stream):
        q, h = PL.rms_norm(x, w, r, kind="int8", stream=stream)
        y = PL.linear(q, weight, stream=stream)
        dx, dw = PL.rms_norm_grad(dy, h, w, stream=stream)
        again = PL.linear(q, weight, stream=stream)
        return h, y, dx, dw, again

    want = work(None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    sizes = (B.linear_fwd_workspace_bytes(100, 1280, 8192, B.IGC_INT8), B.norm_bwd_workspace_bytes(100, 8192),
             100 * 8192, 200 * 8192, 2 * 100 * 1280)
    for _ in range(3):
        got = work(side.cuda_stream if handle else side)
        for size in sizes:  # on the current stream, while the side stream may still be at work
            torch.empty((size,), dtype=torch.uint8, device="cuda").fill_(0xFF)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
