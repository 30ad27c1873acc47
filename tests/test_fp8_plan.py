"""The launch rules of the 8-bit kernels (csrc/fp8_plan.h), run on the host."""
import ctypes
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "gemm_decode_nvfp4_b200", "csrc")
SM_REGISTERS, SM_SMEM, SM_THREADS = 65536, 228 * 1024, 2048


@pytest.fixture(scope="session")
def plan(tmp_path_factory):
    lib = str(tmp_path_factory.mktemp("plan") / "plan.so")
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", f"-I{CSRC}",
                    os.path.join(ROOT, "tests", "fp8_plan_host.cpp"), "-o", lib], check=True)
    return ctypes.CDLL(lib)


def norm_rows(plan, K, residual, regs):
    """regs: registers per thread of the kernels with 2 and 4 vectors per thread."""
    out = (ctypes.c_int * 4)()
    plan.norm_rows(ctypes.c_int64(K), int(residual), *(SM_REGISTERS // 32 // (-(-r // 8) * 8) for r in regs), out)
    return tuple(out)


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("regs", [(55, 64), (64, 64), (40, 48), (32, 32)])
def test_an_sm_holds_the_norm_ctas_planned_for_it(plan, residual, regs):
    """Registers, threads and shared memory of all CTAs planned for an SM are there, every
    column has a thread, and a CTA has two row slots or the rule gives the row up."""
    for K in range(1040, 32768 + 16, 16):
        wide, threads, per_sm, slots = norm_rows(plan, K, residual, regs)
        row = K * (4 if residual else 2)
        if per_sm == 0:
            assert 2 * row + 2048 > 227 * 1024
            continue
        held = -(-regs[wide == 4] // 8) * 8
        assert threads % 32 == 0 and threads <= 1024 and K <= threads * wide * 8 < K + 32 * wide * 8
        assert per_sm * threads * held <= SM_REGISTERS, K
        assert per_sm * threads <= SM_THREADS
        assert per_sm * (slots * row + 1024 + 512) <= SM_SMEM and slots * row + 512 <= 227 * 1024
        assert 2 <= slots <= 8


def test_two_norm_ctas_where_the_registers_hold_them(plan):
    """55 registers: 36 warps, two CTAs of 18 (K = 9216) but not of 19."""
    assert norm_rows(plan, 9216, False, (55, 64))[1:3] == (576, 2)
    assert norm_rows(plan, 9232, False, (55, 64))[1:3] == (608, 1)
    assert norm_rows(plan, 9216, False, (64, 64))[1:3] == (576, 1)
    assert norm_rows(plan, 5120, False, (55, 64))[2:] == (3, 7)
    assert norm_rows(plan, 5120, True, (55, 64))[2:] == (2, 5)


SMS = 148
WIDTHS = (16, 32, 64, 128, 256)


def choice(plan, T, E, N, K, grouped):
    out = (ctypes.c_int * 2)()
    plan.gemm_choice(*(ctypes.c_int64(v) for v in (T, E, N, K)), int(grouped), SMS, out)
    return tuple(out)


def test_gpu_tests_reach_every_configuration_of_the_products(plan):
    """Each size of test_gpu_fp8_choices takes the configuration that it is listed under,
    and over 200000 random shapes no other configuration is chosen."""
    from test_gpu_fp8_choices import DENSE, GROUPED
    assert {s: choice(plan, s[0], 1, s[1], s[2], False) for s in DENSE.values()} == \
        {shape: pair for pair, shape in DENSE.items()}
    assert {w: choice(plan, *s, True) for w, s in GROUPED.items()} == {w: (w, 1) for w in WIDTHS}
    counts, shapes = (ctypes.c_int * 40)(), (ctypes.c_int64 * 120)()
    plan.scan_choices(200000, ctypes.c_uint64(3), SMS, counts, shapes)
    found = {(w, c + 1): tuple(shapes[3 * (8 * i + c):][:3]) for i, w in enumerate(WIDTHS) for c in range(8)
             if counts[8 * i + c]}
    assert not set(found) - set(DENSE), {k: v for k, v in found.items() if k not in DENSE}


def test_a_split_has_a_block_for_every_cta(plan):
    for K in range(16, 1100, 16):
        for M, N in ((1, 64), (33, 640), (120, 5120)):
            assert choice(plan, M, 1, N, K, False)[1] <= -(-K // 128)


def test_grouped_products_are_not_split(plan):
    for T in (1, 7, 64, 1000, 30000):
        for E in (1, 8, 160, 4096):
            width, splits = choice(plan, T, E, 1536, 2048, True)
            assert width in WIDTHS and splits == 1
