"""The 4-bit layer's calls that allocate or copy: their memory belongs to the stream that
they are given (see test_stream_host.py)."""
import pytest
import torch

import gemm_decode_nvfp4_b200 as nv
from test_stream_host import log  # noqa: F401  (the recorders)

BF16, U8, F32 = torch.bfloat16, torch.uint8, torch.float32


@pytest.fixture
def calls(log, monkeypatch):  # noqa: F811
    """The library's calls recorded too, with the checks for CUDA tensors left out."""
    dev = torch.device("cpu")
    monkeypatch.setattr(nv, "_need", lambda *a, **k: None)
    monkeypatch.setattr(nv, "_stream", lambda stream, d: stream)
    monkeypatch.setattr(nv, "_device", lambda *t: dev)
    monkeypatch.setattr(nv, "gemm_workspace_size", lambda M, N, K: 64)

    def call(fn, d, *args):
        torch.empty(0)
        current = log.pop()[1]
        log.append((fn, current if args[-1] is None else args[-1]))
    monkeypatch.setattr(nv, "_call", call)
    return log


W, S, SMX = torch.zeros((64, 128), dtype=BF16), torch.zeros((64, 8), dtype=U8), torch.zeros((64, 4), dtype=U8)
Q, G = torch.zeros((64, 64), dtype=U8), torch.zeros((1,))
CUBE = torch.zeros((8, 4, 16), dtype=BF16).transpose(0, 1)   # reshape copies it
CALLS = {
    "amax": (lambda s: nv.amax(CUBE, G, stream=s), ["copy", "nvfp4_amax"]),
    "quantize_new": (lambda s: nv.quantize_new(W, stream=s), ["empty", "empty", "empty", "nvfp4_quantize"]),
    "linear": (lambda s: nv.linear(W[:3], Q, S, G, stream=s), ["empty", "empty", "nvfp4_gemm_ex"]),
    "mx_quantize_new": (lambda s: nv.mx_quantize_new(W, stream=s), ["empty", "empty", "mxfp4_quantize"]),
    "mx_to_nvfp4": (lambda s: nv.mx_to_nvfp4(Q, SMX, stream=s), ["empty", "empty", "mxfp4_to_nvfp4_scales"]),
    "w4a4_prepare_weights": (lambda s: nv.w4a4_prepare_weights(S, 128, stream=s),
                             ["empty", "nvfp4_w4a4_prepare_weights"]),
    "w4a4_quantize_x": (lambda s: nv.w4a4_quantize_x(W, torch.zeros(260), stream=s),
                        ["empty", "empty", "nvfp4_w4a4_quantize_x"]),
}


@pytest.mark.parametrize("name", CALLS)
def test_memory_belongs_to_the_given_stream(calls, name):
    call, steps = CALLS[name]
    call("side")
    assert calls == [(step, "side") for step in steps]


@pytest.mark.parametrize("name", CALLS)
def test_without_a_stream_the_current_one(calls, name):
    call, steps = CALLS[name]
    call(None)
    assert calls == [(step, "caller's") for step in steps]
