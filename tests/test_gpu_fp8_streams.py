"""The 8-bit layer's allocating calls on a stream of their own, beside allocations of the
current stream."""
import pytest
import torch

from test_gpu_fp8 import BF16, F32, blocks, nv, randn  # noqa: F401  (nv: the module's fixture)

pytestmark = pytest.mark.gpu


def fill(M, K, N):
    """Blocks of a call's sizes on the current stream, filled and dropped."""
    for shape, dtype in (((M, K), torch.uint8), ((M, blocks(K)), F32), ((M, N), BF16)):
        torch.empty(shape, dtype=dtype, device="cuda").fill_(127)


@pytest.mark.parametrize("M,N,K", [(1, 1024, 5120), (300, 640, 2064), (2000, 4096, 1024)])
def test_linear_on_a_side_stream(nv, M, N, K):  # noqa: F811
    """Nothing that the current stream allocates meanwhile meets the call's codes and scales."""
    xs = [randn((M, K), 100 + i) for i in range(8)]
    w, sw = nv.fp8_quantize_weights_new(randn((N, K), 3, 0.02))
    refs = [nv.fp8_linear(x, w, sw) for x in xs]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for rep in range(4):
        for x in xs:
            got.append(nv.fp8_linear(x, w, sw, stream=side))
            fill(M, K, N)
    side.synchronize()
    for i, y in enumerate(got):
        assert torch.equal(y, refs[i % len(xs)]), i


def test_quantizers_on_a_side_stream(nv):  # noqa: F811
    M, K = 700, 2064
    xs = [randn((M, 2 * K), 200 + i) for i in range(6)]
    refs = [(nv.fp8_quantize_new(x), nv.fp8_quantize_new(x, gated=True), nv.fp8_quantize_weights_new(x)) for x in xs]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for x in xs:
        fill(M, K, 2 * K)
        got.append((nv.fp8_quantize_new(x, stream=side), nv.fp8_quantize_new(x, gated=True, stream=side),
                    nv.fp8_quantize_weights_new(x, stream=side)))
        fill(M, K, 2 * K)
    side.synchronize()
    for a, b in zip(got, refs):
        for (q, s), (q0, s0) in zip(a, b):
            assert torch.equal(q.view(torch.uint8), q0.view(torch.uint8)) and torch.equal(s, s0)


def test_results_are_used_and_dropped_on_the_current_stream(nv):  # noqa: F811
    """Y is read by the current stream, ordered behind the side stream, and dropped at
    once: the next call on the side stream does not write over it."""
    M, N, K = 256, 8192, 1024
    w, sw = nv.fp8_quantize_weights_new(randn((N, K), 3, 0.02))
    xs = [randn((M, K), 300 + i) for i in range(6)]
    refs = [nv.fp8_linear(x, w, sw) for x in xs]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    copies = []
    for x in xs:
        y = nv.fp8_linear(x, w, sw, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        copies.append(y.clone())
        del y
    torch.cuda.synchronize()
    for y, ref in zip(copies, refs):
        assert torch.equal(y, ref)


def test_captured_on_a_side_stream(nv):  # noqa: F811
    M, N, K = 5, 1024, 2048
    w, sw = nv.fp8_quantize_weights_new(randn((N, K), 3, 0.02))
    x = randn((M, K), 1)
    side = torch.cuda.Stream()
    nv.fp8_linear(x, w, sw, stream=side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        y = nv.fp8_linear(x, w, sw, stream=side)
    for i in range(3):
        x.copy_(randn((M, K), 10 + i))
        graph.replay()
        assert torch.equal(y, nv.fp8_linear(x, w, sw))
