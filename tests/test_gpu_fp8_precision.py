"""The products' arithmetic: sums over the blocks of k that need more bits than the
outputs have, and random data against what fp32 sums can be off by."""
import pytest
import torch

from test_gpu_fp8 import BF16, F8, F64, blocks, nv, spread  # noqa: F401
from test_gpu_fp8_range import SHAPES, both

pytestmark = pytest.mark.gpu


def cancelling(M, N, K, seed):
    """Blocks whose sums are one product each, so that row m's block b adds the whole number
    v[m, b] (or its negative, or nothing where w's code is 0): two pairs of blocks with
    v = +-(2^21 + a) for small odd a, small v elsewhere.  Every sum of some of a row's
    blocks, in any order, is a whole number below 2^24; it needs up to 23 bits, and what is
    left in the end about 8."""
    kb = blocks(K)
    g = torch.Generator().manual_seed(seed)
    small = lambda *shape: 2 * torch.randint(0, 4, shape, generator=g).double() + 1  # noqa: E731  (1, 3, 5, 7)
    v = small(M, kb)
    sign = torch.ones(kb, dtype=F64)
    large = torch.randperm(kb, generator=g)[:4]
    v[:, large] += 2.0 ** 21
    sign[large[1::2]] = -1
    x, w = torch.zeros((M, K)), torch.zeros((N, K))
    for b in range(kb):
        at = 128 * b + (37 * b) % min(128, K - 128 * b)
        x[:, at] = sign[b]
        w[:, at] = 1.0 if b in large else (torch.rand((N,), generator=g) < 0.5).float()
    w *= torch.where(torch.rand((N, 1), generator=g) < 0.5, 1.0, -1.0)
    sw = torch.exp2(torch.randint(-2, 3, (blocks(N), 1), generator=g).float()).expand(-1, kb).contiguous()
    return x.to(F8).cuda(), v.float().cuda(), w.to(F8).cuda(), sw.cuda()


@pytest.mark.parametrize("M,N,K", SHAPES + [(1, 17408, 5120), (47, 5120, 17408), (128, 2560, 5120), (4100, 640, 1040)])
def test_sums_over_blocks_keep_24_bits(nv, M, N, K):  # noqa: F811
    """Large sums of blocks cancel exactly: with fewer bits than fp32's the small rest is lost."""
    x, sx, w, sw = cancelling(M, N, K, M + N)
    ref = ((x.double() * spread(sx.double(), 1, M, K)) @ (w.double() * spread(sw.double(), 128, N, K)).T)
    assert float(ref.abs().max()) < 2048
    for Y in both(nv, x, sx, w, sw):
        assert torch.equal(Y, ref.float().to(BF16))


@pytest.mark.parametrize("M,N,K", SHAPES + [(1, 1001, 17408), (47, 640, 17408), (1111, 640, 5120)])
def test_random_data_to_fp32(nv, M, N, K):  # noqa: F811
    """Products of random codes, their sums in fp32: a block is four MMAs of 32 products and
    the accumulator, each addend held to 24 bits of the largest, off by at most 33 * 2^-24 of
    sum |x w| of the block and MMA; over blocks one product of scales, one multiplication and
    addition each, 2^-24 of the sums so far.  (132 + 2 kb) 2^-24 of sum |x w|, and the BF16
    rounding."""
    X = torch.randn((M, K), generator=torch.Generator().manual_seed(M)).to(BF16).cuda()
    W = (0.02 * torch.randn((N, K), generator=torch.Generator().manual_seed(N))).to(BF16).cuda()
    q, s = nv.fp8_quantize_new(X)
    w, sw = nv.fp8_quantize_weights_new(W)
    x64, w64 = q.double() * spread(s.double(), 1, M, K), w.double() * spread(sw.double(), 128, N, K)
    ref, mag = x64 @ w64.T, x64.abs() @ w64.abs().T
    tol = (132 + 2 * blocks(K)) * 2.0 ** -24 * mag + 2.0 ** -8 * ref.abs()
    for Y in both(nv, q, s, w, sw):
        bad = (Y.double() - ref).abs() > tol
        assert not bool(bad.any()), f"{int(bad.sum())} of {bad.numel()} outputs out of tolerance"
