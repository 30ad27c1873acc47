"""The 8-bit layer called from host threads side by side, also as a process's first calls."""
import os
import subprocess
import sys
import threading

import pytest
import torch

from test_gpu_fp8 import check_mlp, mlp, mlp_state, nv  # noqa: F401

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def run(*work):
    """Each function on a thread of its own; the first exception is raised here."""
    errors = []

    def guarded(f):
        try:
            f()
        except BaseException as e:  # noqa: BLE001
            errors.append(e)
    threads = [threading.Thread(target=guarded, args=(f,)) for f in work]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    if errors:
        raise errors[0]


@pytest.mark.parametrize("sizes", [(1, 37), (37, 700), (5, 5)])
def test_two_threads_with_streams_of_their_own(nv, sizes):  # noqa: F811
    states = [mlp_state(nv, M, 1024, 1808, 40 + i) for i, M in enumerate(sizes)]
    torch.cuda.synchronize()

    def work(st):
        def f():
            with torch.cuda.stream(torch.cuda.Stream()):
                first = None
                for _ in range(50):
                    mlp(nv, st)
                    y = st["y"].clone()
                    first = y if first is None else first
                    assert torch.equal(y, first)
                torch.cuda.current_stream().synchronize()
        return f
    run(*(work(st) for st in states))
    for st in states:
        check_mlp(st)


def test_a_refused_call_keeps_its_message_to_its_thread(nv):  # noqa: F811
    st = mlp_state(nv, 4, 512, 528, 60)
    X = st["x"]
    torch.cuda.synchronize()

    def refused():
        for _ in range(300):
            with pytest.raises(nv.Nvfp4Error, match="no output"):
                nv.fp8_rmsnorm(X, st["nw"])

    def other():
        for _ in range(300):
            with pytest.raises(nv.Nvfp4Error, match="overlap"):
                nv.fp8_rmsnorm(X, st["nw"], y=X)

    def good():
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(100):
                mlp(nv, st)
            torch.cuda.current_stream().synchronize()
    run(refused, other, good)
    check_mlp(st)


FIRST = """
import sys, threading
sys.path[:0] = [{root!r}, {root!r} + "/tests"]
import torch
import gemm_decode_nvfp4_b200 as nv
from test_gpu_fp8 import check_mlp, mlp, mlp_state
from test_gpu_fp8_threads import run
torch.zeros(1, device="cuda")
sts = [None] * 3
barrier = threading.Barrier(3)
def work(i, M):
    def f():
        with torch.cuda.stream(torch.cuda.Stream()):
            barrier.wait()
            sts[i] = mlp_state(nv, M, 1024, 1808, 70 + i)
            mlp(nv, sts[i])
            torch.cuda.current_stream().synchronize()
    return f
run(work(0, 1), work(1, 700), work(2, 90))
for st in sts:
    check_mlp(st)
nv.check_device_errors()
print("ok")
"""


def test_first_calls_of_a_process_from_three_threads():
    r = subprocess.run([sys.executable, "-c", FIRST.format(root=ROOT)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), r.stdout + r.stderr
