"""Calls that allocate: what they allocate and copy belongs to the stream that they are
given.  Host logic only, with the streams and the library's calls replaced by recorders:
memory of another stream could be handed on while the call's kernels still use it."""
import contextlib

import pytest
import torch

import gemm_decode_nvfp4_b200 as nv

BF16, F8 = torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture
def log(monkeypatch):
    """Names the stream that is current at each allocation, copy and call of the binding."""
    seen, current = [], ["caller's"]

    @contextlib.contextmanager
    def on(stream):
        before, current[0] = current[0], stream
        yield
        current[0] = before

    empty, reshape = torch.empty, torch.Tensor.reshape

    def new(*a, **k):
        seen.append(("empty", current[0]))
        return empty(*a, **k)

    def reshaped(t, *shape):
        out = reshape(t, *shape)
        if out.data_ptr() != t.data_ptr():
            seen.append(("copy", current[0]))
        return out

    def call(name):
        def f(*a, stream=None, **k):
            seen.append((name, current[0] if stream is None else stream))
        return f

    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch, "empty", new)
    monkeypatch.setattr(torch.Tensor, "reshape", reshaped)
    for name in ("fp8_quantize", "fp8_quantize_weights", "fp8_gemm"):
        monkeypatch.setattr(nv, name, call(name))
    return seen


X, W, SW = torch.zeros((4, 128), dtype=BF16), torch.zeros((64, 128), dtype=F8), torch.zeros((1, 1))
CALLS = {
    "fp8_quantize_new": (lambda s: nv.fp8_quantize_new(X, stream=s), ["empty", "empty", "fp8_quantize"]),
    "fp8_quantize_new gated": (lambda s: nv.fp8_quantize_new(X, gated=True, stream=s),
                               ["empty", "empty", "fp8_quantize"]),
    "fp8_quantize_weights_new": (lambda s: nv.fp8_quantize_weights_new(X, stream=s),
                                 ["empty", "empty", "fp8_quantize_weights"]),
    "fp8_linear": (lambda s: nv.fp8_linear(X, W, SW, stream=s),
                   ["empty", "empty", "fp8_quantize", "empty", "fp8_gemm"]),
    "fp8_linear of a row that reshape copies": (
        lambda s: nv.fp8_linear(torch.zeros((8, 16, 1), dtype=BF16).transpose(0, 1), W, SW, stream=s),
        ["copy", "empty", "empty", "fp8_quantize", "empty", "fp8_gemm"]),
}


@pytest.mark.parametrize("name", CALLS)
def test_memory_belongs_to_the_given_stream(log, name):
    call, steps = CALLS[name]
    call("side")
    assert log == [(step, "side") for step in steps]


@pytest.mark.parametrize("name", CALLS)
def test_without_a_stream_the_current_one(log, name):
    call, steps = CALLS[name]
    call(None)
    assert log == [(step, "caller's") for step in steps]
