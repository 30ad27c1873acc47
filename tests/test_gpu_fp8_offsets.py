"""Grouped 8-bit products whose offsets decrease or leave the rows: each call counts
once, and the rows that the clamped offsets give to an expert are its product."""
import pytest
import torch

from test_gpu_fp8 import BF16, blocks, grouped_ref, nv, powers, values, whole_numbers  # noqa: F401

pytestmark = pytest.mark.gpu
INT_MIN, INT_MAX = -(1 << 31), (1 << 31) - 1

BAD = [[0, 30, 10, 40], [-5, 10, 20, 40], [0, 10, 20, 1000], [50, 0, 50, 0], [INT_MIN, INT_MAX, 0, 7],
       [0, 20, 10, 30, 25, 50], [0] * 40 + [7, 3] + [50] * 40]


def make(E, N=136, K=144, T=50):
    x, w = whole_numbers((T, K), 1), whole_numbers((E, N, K), 2)
    return x, powers((T, blocks(K)), 3), w, powers((E, blocks(N), blocks(K)), 4)


def clamped(ends, T):
    """First row and row end of each expert: offsets clamped to the rows, an expert
    starting no earlier than any before it ends."""
    rows, reach = [], 0
    for u, v in zip(ends, ends[1:]):
        lo, hi = min(max(u, 0), T), min(max(v, 0), T)
        lo = max(lo, reach)
        rows.append((lo, max(hi, lo)))
        reach = max(reach, hi)
    return rows


@pytest.mark.parametrize("ends", BAD, ids=range(len(BAD)))
@pytest.mark.parametrize("calls", [1, 3])
def test_a_bad_call_counts_once(nv, ends, calls):  # noqa: F811
    T, N = 50, 136
    x, sx, w, sw = make(len(ends) - 1)
    Y = torch.empty((T, N), dtype=BF16, device="cuda")
    offsets = torch.tensor(ends, dtype=torch.int32, device="cuda")
    nv.check_device_errors()
    for _ in range(calls):
        nv.fp8_gemm_grouped(x, sx, w, sw, offsets, Y)
    torch.cuda.synchronize()
    with pytest.raises(nv.Nvfp4Error, match=rf"\b{calls} grouped fp8 GEMM call\(s\)"):
        nv.check_device_errors()
    nv.check_device_errors()


@pytest.mark.parametrize("ends", BAD, ids=range(len(BAD)))
def test_rows_of_clamped_offsets(nv, ends):  # noqa: F811
    T, N = 50, 136
    x, sx, w, sw = make(len(ends) - 1)
    Y = torch.full((T, N), 5.0, dtype=BF16, device="cuda")
    ref, X = Y.clone(), values(x, sx, 1)
    for e, (a, b) in enumerate(clamped(ends, T)):
        if b > a:
            ref[a:b] = (X[a:b] @ values(w[e], sw[e], 128).T).float().to(BF16)
    nv.fp8_gemm_grouped(x, sx, w, sw, torch.tensor(ends, dtype=torch.int32, device="cuda"), Y)
    torch.cuda.synchronize()
    with pytest.raises(nv.Nvfp4Error, match="offsets"):
        nv.check_device_errors()
    assert torch.equal(Y, ref)


def test_good_offsets_are_not_counted(nv):  # noqa: F811
    ends = [2, 2, 17, 17, 50]
    x, sx, w, sw = make(4)
    Y = torch.full((50, 136), 5.0, dtype=BF16, device="cuda")
    ref = grouped_ref(x, sx, w, sw, ends, Y)
    nv.fp8_gemm_grouped(x, sx, w, sw, torch.tensor(ends, dtype=torch.int32, device="cuda"), Y)
    torch.cuda.synchronize()
    nv.check_device_errors()
    assert torch.equal(Y, ref)
