"""The products in every configuration that the launch rule can take: tile width and CTAs
that share a tile's blocks of k.  tests/test_fp8_plan.py holds that each size here takes the
configuration that it stands for, and that there are no others."""
import pytest
import torch

from gpu_util import guarded_empty
from test_gpu_fp8 import BF16, blocks, grouped_ref, nv, powers, values, whole_numbers  # noqa: F401

pytestmark = pytest.mark.gpu

DENSE = {  # (width, split): M, N, K
    (16, 1): (1, 100, 16), (16, 2): (1, 8431, 768), (16, 3): (1, 5637, 672), (16, 4): (1, 4108, 912),
    (16, 5): (1, 121, 608), (16, 6): (6, 2838, 656), (16, 7): (14, 100, 784), (16, 8): (3, 100, 1040),
    (32, 1): (2385, 129, 16), (32, 2): (1148, 129, 3280), (32, 3): (17, 5936, 1984), (32, 4): (568, 132, 2800),
    (32, 5): (767, 133, 1840), (32, 6): (598, 133, 1936), (32, 7): (17, 4623, 1568), (32, 8): (17, 3567, 2704),
    (64, 1): (4740, 129, 16), (64, 2): (34, 14246, 3472), (64, 3): (2405, 130, 1808), (64, 4): (34, 7187, 2976),
    (64, 5): (1512, 129, 2496), (64, 6): (33, 4803, 4272), (64, 7): (1130, 133, 3392), (64, 8): (865, 135, 5712),
    (128, 1): (4790, 137, 544), (128, 2): (3014, 129, 4496), (128, 3): (2394, 129, 12896),
    (128, 4): (1803, 130, 16800), (128, 5): (4769, 135, 7552), (128, 6): (2434, 1, 26208),
    (128, 7): (1688, 1, 32112), (128, 8): (752, 139, 17296), (256, 1): (6307, 257, 16),
}
GROUPED = {  # width: T, E, N, K
    16: (40, 9, 1001, 528), 32: (700, 5, 1001, 1040), 64: (2000, 20, 1536, 144), 128: (1000, 8, 1536, 1040),
    256: (900, 4, 1540, 1040),
}


@pytest.mark.parametrize("M,N,K", DENSE.values(), ids=[f"{w}x{c}" for w, c in DENSE])
def test_gemm_in_every_configuration(nv, M, N, K):  # noqa: F811
    x, w = whole_numbers((M, K), M + K), whole_numbers((N, K), N + K)
    sx, sw = powers((M, blocks(K)), M), powers((blocks(N), blocks(K)), N)
    ref = (values(x, sx, 1) @ values(w, sw, 128).T).float().to(BF16)
    Y, chk = guarded_empty((M, N), BF16)
    for static in (False, True):
        Y.fill_(float("nan"))
        nv.fp8_gemm(x, sx, w, sw, Y, static_weights=static)
        assert torch.equal(Y, ref), f"{int((Y != ref).sum())} of {ref.numel()} differ"
    chk()


@pytest.mark.parametrize("T,E,N,K", GROUPED.values(), ids=map(str, GROUPED))
def test_grouped_in_every_width(nv, T, E, N, K):  # noqa: F811
    g = torch.Generator().manual_seed(T)
    ends = [1, *sorted(torch.randint(1, T - 2, (E - 1,), generator=g).tolist()), T - 2]
    x, w = whole_numbers((T, K), 1), whole_numbers((E, N, K), 2)
    sx, sw = powers((T, blocks(K)), 3), powers((E, blocks(N), blocks(K)), 4)
    Y, chk = guarded_empty((T, N), BF16)
    Y.fill_(5.0)
    ref = grouped_ref(x, sx, w, sw, ends, Y)
    nv.fp8_gemm_grouped(x, sx, w, sw, torch.tensor(ends, dtype=torch.int32, device="cuda"), Y)
    assert torch.equal(Y, ref)
    chk()
