"""The gated quantizer where silu is smallest, and at gates that are not finite.

Tolerance: silu = g * sigma, sigma from 2^x with x = -g log2(e) - 8 and a reciprocal.  For
gates from -91 on, |x| < 128 where 2^x counts, so x is off by at most 2^-18 (rounding)
and 2^-19 (log2(e) in fp32) and 2^x by 2^-18 of itself; the two approximations by 2^-22
and 2^-23; sigma, subnormal down to 2^-131.3, by 2^-150, 2^-18.7 of it; four roundings of
2^-24.  Less than 2^-17 of silu in all; 2^-15 is what fp8.h states."""
import pytest
import torch

from test_gpu_fp8 import BF16, F64, check_quantized, nv  # noqa: F401

pytestmark = pytest.mark.gpu


def gated(g, u):
    return torch.cat([g.to(BF16), u.to(BF16)], 1).cuda()


@pytest.mark.parametrize("up", [1e37, -3e38, 2.0 ** 100])
@pytest.mark.parametrize("K", [128, 144, 2064])
def test_far_gates_with_a_large_up(nv, K, up):  # noqa: F811
    """Gates from -91 to -86: silu is a normal fp32 number (1.4e-38 to 4e-36), which a
    large up value brings back into range."""
    g = torch.linspace(-91, -86, 5 * K, dtype=F64).to(BF16).view(5, K)
    x = gated(g, torch.full((5, K), up, dtype=F64))
    q, s = nv.fp8_quantize_new(x, gated=True)
    gd, ud = x[:, :K].double(), x[:, K:].double()
    v = gd / (1 + torch.exp(-gd)) * ud
    assert bool((v != 0).all())
    check_quantized(v, q, s, 2.0 ** -15)
    assert bool((q.float() != 0).all())     # (within a block the values differ by less than 448)


def test_gates_over_the_whole_range(nv):  # noqa: F811
    """Blocks of neighbouring gates, so that every code and scale depends on its own."""
    g = torch.linspace(-91, 127, 128 * 40, dtype=F64).to(BF16).view(40, 128)
    x = gated(g, torch.linspace(0.5, 2, 128 * 40, dtype=F64).view(40, 128) * 2.0 ** 20)
    q, s = nv.fp8_quantize_new(x, gated=True)
    gd, ud = x[:, :128].double(), x[:, 128:].double()
    check_quantized(gd / (1 + torch.exp(-gd)) * ud, q, s, 2.0 ** -15)


def test_gates_that_are_not_finite(nv):  # noqa: F811
    """silu(inf) = inf takes its block; silu of NaN, and -inf / inf, stay in their element."""
    g, u = torch.full((3, 256), 1.0, dtype=F64), torch.ones((3, 256), dtype=F64)
    clean, sc = nv.fp8_quantize_new(gated(g, u), gated=True)
    g[0, 3], g[1, 130], g[2, 5] = float("nan"), float("inf"), float("-inf")
    q, s = nv.fp8_quantize_new(gated(g, u), gated=True)
    assert bool(q.float()[0, 3].isnan()) and bool(q.float()[1, 130].isnan()) and bool(q.float()[2, 5].isnan())
    assert s[1, 1].item() == float("inf")
    same = torch.ones((3, 256), dtype=torch.bool)
    same[0, 3], same[1, 128:], same[2, 5] = False, False, False
    assert torch.equal(q.float().cpu()[same], clean.float().cpu()[same])
    s[1, 1] = sc[1, 1]
    assert torch.equal(s, sc)
