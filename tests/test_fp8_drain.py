"""Before a CTA of the 8-bit kernels that gave up on a wait ends, every copy that it asked
for has landed: the kernels' own rule (csrc/fp8_drain.h) on a model of their rings, with
roles that stop at any point.  Host code only."""
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "gemm_decode_nvfp4_b200", "csrc")


@pytest.fixture(scope="module")
def failures(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("drain") / "sim")
    subprocess.run(["g++", "-O1", "-std=c++17", f"-I{CSRC}", os.path.join(ROOT, "tests", "fp8_drain_sim.cpp"),
                    "-o", exe], check=True)
    out = subprocess.run([exe], check=True, capture_output=True, text=True, timeout=120).stdout
    return dict(zip(("product", "norm"), map(int, re.findall(r"\d+", out))))


@pytest.mark.parametrize("ring", ["product", "norm"])
def test_nothing_is_left_in_flight(failures, ring):
    assert failures[ring] == 0


@pytest.mark.parametrize("source", ["fp8_gemm.cu", "fp8_quant.cu"])
def test_the_kernels_drain_by_this_rule(source):
    with open(os.path.join(CSRC, source)) as f:
        assert "drain_ring(" in f.read()
