"""The products at the ends of the scales' range: sx * sw the smallest or a very large
normal fp32 number, and the scales of blocks of zeros."""
import pytest
import torch

from test_gpu_fp8 import BF16, F8, blocks, nv, whole_numbers  # noqa: F401

pytestmark = pytest.mark.gpu

# (M, N, K): one token, a few, a middle batch, and token rows (256 weight rows per tile)
SHAPES = [(1, 300, 2064), (20, 640, 4096), (60, 5120, 2064), (120, 700, 1040), (900, 1100, 2064), (1500, 5125, 528)]


def both(nv, x, sx, w, sw):  # noqa: F811
    """The dense product and the same rows as two experts with these weights."""
    M, N = x.shape[0], w.shape[0]
    Y, Z = (torch.full((M, N), float("nan"), dtype=BF16, device="cuda") for _ in range(2))
    nv.fp8_gemm(x, sx, w, sw, Y)
    nv.fp8_gemm_grouped(x, sx, torch.stack([w.view(torch.uint8)] * 2).view(F8), torch.stack([sw, sw]),
                        torch.tensor([0, M // 3, M], dtype=torch.int32, device="cuda"), Z)
    return Y, Z


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("ex,ew", [(-100, -26), (-26, -100), (-63, -63), (100, 13), (13, 100),
                                   (57, 56), (-120, 120)])
def test_scales_with_a_normal_product(nv, M, N, K, ex, ew):  # noqa: F811
    """Whole-number sums (at most 4 K <= 2^14) times 2^(ex + ew) <= 2^113: exact in fp32,
    rounded once to BF16.  2^(ex + ew) is a normal number, whatever ex and ew are."""
    x, w = whole_numbers((M, K), M + K), whole_numbers((N, K), N + K)
    sx = torch.full((M, blocks(K)), 2.0 ** ex, device="cuda")
    sw = torch.full((blocks(N), blocks(K)), 2.0 ** ew, device="cuda")
    ref = ((x.double() @ w.double().T) * 2.0 ** (ex + ew)).float().to(BF16)
    assert bool(ref.isfinite().all()) and bool((ref != 0).any())
    for Y in both(nv, x, sx, w, sw):
        assert torch.equal(Y, ref)


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_zero_rows_and_zero_blocks_as_the_quantizers_leave_them(nv, M, N, K):  # noqa: F811
    """A row or block of zeros has the scale 2^-126: its products are zeros, not NaN."""
    X = torch.randn((M, K), generator=torch.Generator().manual_seed(1)).to(BF16)
    W = (2.0 ** -60 * torch.randn((N, K), generator=torch.Generator().manual_seed(2))).to(BF16)
    X[M // 2] = 0.0
    W[:128] = 0.0
    q, s = nv.fp8_quantize_new(X.cuda())
    w, sw = nv.fp8_quantize_weights_new(W.cuda())
    assert s[M // 2, 0].item() == 2.0 ** -126 and sw[0, 0].item() == 2.0 ** -126
    for Y in both(nv, q, s, w, sw):
        assert not bool(Y[M // 2].any()) and not bool(Y[:, :128].any()) and bool(Y.isfinite().all())
        assert M == 1 or bool(Y[0, 128:].any())
