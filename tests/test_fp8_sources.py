"""What the 8-bit kernels' sources hold themselves to."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gemm_decode_nvfp4_b200", "csrc")


def code(name):
    """A source without its comments."""
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


@pytest.mark.parametrize("name", ["fp8_gemm.cu", "fp8_quant.cu"])
def test_no_read_only_loads(name):
    """The kernels start while the ones before them may still write what they read, so no
    load of theirs is one for data that nothing writes while the kernel runs: neither by
    instruction nor by what `const __restrict__` lets the compiler take for such."""
    text = code(name)
    assert "griddepcontrol.wait" in text
    for word in ("__ldg", "ld.global.nc", "ld_stream"):
        assert word not in text, word
    assert not re.search(r"const \w+\* __restrict__", text)
