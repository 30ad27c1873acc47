"""The 4-bit layer's allocating calls on a stream of their own, beside a current stream
that keeps allocating blocks of the same sizes."""
import pytest
import torch

import workloads

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def nv():
    import gemm_decode_nvfp4_b200 as m
    yield m
    m.check_device_errors()


@pytest.mark.parametrize("M,N,K", [(40, 384, 1024), (256, 1024, 2048)])
def test_allocating_calls_on_a_side_stream(nv, M, N, K):
    w = workloads.random_bf16((N, K), 1, 0.02).cuda()
    xs = [workloads.random_bf16((M, K), 10 + i).cuda() for i in range(6)]
    q, s, g = nv.quantize_new(w)
    refs = [nv.linear(x, q, s, g) for x in xs]
    mq, ms = nv.mx_quantize_new(w)
    nv_s, nv_g = nv.mx_to_nvfp4(mq, ms)
    s_mma = nv.w4a4_prepare_weights(s, K)
    side = torch.cuda.Stream()
    n = max(nv.gemm_workspace_size(M, N, K), 1)
    torch.cuda.synchronize()
    got, again = [], []
    for x in xs:
        got.append(nv.linear(x, q, s, g, stream=side))
        torch.empty(n, dtype=torch.uint8, device="cuda").fill_(127)
        torch.empty((M, N), dtype=BF16, device="cuda").fill_(7)
        again.append([*nv.quantize_new(w, stream=side), *nv.mx_quantize_new(w, stream=side),
                      *nv.mx_to_nvfp4(mq, ms, stream=side), nv.w4a4_prepare_weights(s, K, stream=side)])
        torch.empty((N, K // 2), dtype=torch.uint8, device="cuda").fill_(127)
    side.synchronize()
    for y, ref in zip(got, refs):
        assert torch.equal(y, ref)
    for outs in again:
        for a, b in zip(outs, (q, s, g, mq, ms, nv_s, nv_g, s_mma)):
            assert torch.equal(a, b)
