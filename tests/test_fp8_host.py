"""Host-side checks of the 8-bit entry points (include/fp8.h): every refusal
happens before anything is launched, so none of these calls needs a GPU."""
import pytest
import torch

import gemm_decode_nvfp4_b200 as nv

OK, INVALID, SHAPE, ALIGN = 0, 1, 2, 3
A = 1 << 20  # fake "device addresses": never dereferenced, all calls fail validation or are no-ops
B, C, D, F, G, H = (A + i * (1 << 24) for i in range(1, 7))
NAN, INF = float("nan"), float("inf")


def norm(x=A, ldx=64, w=B, r=None, ldr=0, ro=None, ldro=0, y=None, ldy=0, q=C, s=D, M=4, K=64, eps=1e-6):
    return nv.lib.fp8_rmsnorm(x, ldx, w, r, ldr, ro, ldro, y, ldy, q, s, M, K, eps, None)


def quant(x=A, ldx=64, M=4, K=64, q=C, s=D, flags=0):
    return nv.lib.fp8_quantize(x, ldx, M, K, q, s, flags, None)


def quant_w(w=A, ldw=64, N=4, K=64, q=C, s=D):
    return nv.lib.fp8_quantize_weights(w, ldw, N, K, q, s, None)


def gemm(x=A, sx=B, w=C, sw=D, Y=F, ldy=64, M=4, N=64, K=64, flags=0):
    return nv.lib.fp8_gemm(x, sx, w, sw, Y, ldy, M, N, K, flags, None)


def grouped(x=A, sx=B, w=C, sw=D, off=G, Y=F, ldy=64, T=4, E=2, N=64, K=64, flags=0):
    return nv.lib.fp8_gemm_grouped(x, sx, w, sw, off, Y, ldy, T, E, N, K, flags, None)


def test_symbols_are_declared():
    assert {"fp8_rmsnorm", "fp8_quantize", "fp8_quantize_weights", "fp8_gemm", "fp8_gemm_grouped"} <= \
        set(nv.declared_symbols())


@pytest.mark.parametrize("call", [norm, quant, quant_w, gemm, grouped])
@pytest.mark.parametrize("K", [0, -16, 8, 24, (1 << 24) + 16])
def test_k_is_a_positive_multiple_of_16(call, K):
    assert call(K=K) == SHAPE
    assert b"multiple of 16" in nv.lib.nvfp4_last_error()


@pytest.mark.parametrize("call,rows", [(norm, "M"), (quant, "M"), (quant_w, "N"), (gemm, "M"), (gemm, "N"),
                                       (grouped, "T"), (grouped, "N")])
def test_row_counts(call, rows):
    assert call(**{rows: -1}) == SHAPE
    assert call(**{rows: 1 << 31}) == SHAPE
    assert call(**{rows: 0}) == OK   # a no-op, without a device


def test_norm_refusals():
    assert norm(q=None, s=None) == INVALID          # no output
    assert norm(q=C, s=None) == INVALID
    assert norm(q=None, s=D, y=F, ldy=64) == INVALID
    assert norm(r=F, ldr=64) == INVALID             # residual without residual_out
    assert norm(ro=F, ldro=64) == INVALID
    for eps in (-1e-6, NAN, INF):
        assert norm(eps=eps) == INVALID
    assert norm(x=None) == INVALID and norm(w=None) == INVALID
    assert norm(ldx=48) == INVALID and norm(y=F, ldy=48) == INVALID
    assert norm(r=F, ldr=48, ro=G, ldro=64) == INVALID and norm(r=F, ldr=64, ro=G, ldro=48) == INVALID
    assert norm(ldx=68) == ALIGN and norm(x=A + 8) == ALIGN and norm(w=B + 2) == ALIGN and norm(q=C + 8) == ALIGN
    assert norm(s=D + 2) == ALIGN and norm(y=F + 8, ldy=64) == ALIGN and norm(y=F, ldy=66) == ALIGN
    assert norm(r=F + 8, ldr=64, ro=G, ldro=64) == ALIGN and norm(r=F, ldr=64, ro=G, ldro=66) == ALIGN
    assert norm(q=A + 64) == INVALID and norm(s=A + 64) == INVALID and norm(q=B) == INVALID   # over an input
    assert norm(y=A + 512, ldy=64, q=A + 768) == INVALID                                       # over each other
    assert norm(r=F, ldr=64, ro=F + 16, ldro=64) == INVALID                                    # shifted, not in place
    assert norm(r=F, ldr=64, ro=F, ldro=72) == INVALID


def test_quantize_refusals():
    assert quant(flags=1) == INVALID and quant(flags=4) == INVALID
    assert quant(x=None) == INVALID and quant(q=None) == INVALID and quant(s=None) == INVALID
    assert quant(ldx=48) == INVALID and quant(ldx=64, flags=2) == INVALID   # gated needs 2 K columns
    assert quant(ldx=68) == ALIGN and quant(x=A + 8) == ALIGN and quant(q=C + 4) == ALIGN and quant(s=D + 1) == ALIGN
    assert quant(q=A + 256) == INVALID and quant(s=C + 64) == INVALID
    assert quant(M=1 << 30, K=1 << 10) == SHAPE                             # more than 2^31 blocks
    assert quant_w(w=None) == INVALID and quant_w(ldw=48) == INVALID
    assert quant_w(ldw=68) == ALIGN and quant_w(q=C + 8) == ALIGN and quant_w(s=D + 2) == ALIGN
    assert quant_w(q=A + 256) == INVALID and quant_w(s=C + 64) == INVALID
    assert quant_w(N=1 << 30, K=1 << 16, ldw=1 << 16) == SHAPE


@pytest.mark.parametrize("call", [gemm, grouped])
def test_product_refusals(call):
    rows = "M" if call is gemm else "T"
    assert call(flags=2) == INVALID and call(flags=1 << 8) == INVALID
    for name in ("x", "sx", "w", "sw", "Y"):
        assert call(**{name: None}) == INVALID
    assert call(ldy=63) == INVALID
    assert call(x=A + 8) == ALIGN and call(w=C + 8) == ALIGN
    assert call(sx=B + 2) == ALIGN and call(sw=D + 2) == ALIGN and call(Y=F + 1) == ALIGN
    for over in (A + 16, B, C + 16, D):
        assert call(Y=over) == INVALID
    assert call(**{rows: (1 << 31) - 512, "N": 1 << 20, "ldy": 1 << 20}) == SHAPE   # too many tiles


def test_grouped_refusals():
    assert grouped(off=None) == INVALID and grouped(off=G + 2) == ALIGN and grouped(Y=G) == INVALID
    assert grouped(E=0) == SHAPE and grouped(E=-1) == SHAPE and grouped(E=4097) == SHAPE
    assert grouped(E=4096, N=1 << 20, ldy=1 << 20) == SHAPE


def test_binding_refuses_before_the_library():
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        nv.fp8_quantize(x, x, x)          # CPU tensors
    with pytest.raises(TypeError):
        nv.fp8_rmsnorm(x, x[0])
    with pytest.raises(TypeError):
        nv.fp8_gemm(x, x, x, x, x)
    with pytest.raises(TypeError):
        nv.fp8_gemm_grouped(x, x, x, x, x, x)
