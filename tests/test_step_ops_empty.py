"""Rows by expert where there are no tokens or no rows: a rank that has received nothing
goes through the same calls, forward and backward, and rows that do not exist are still
reported. On the host a stand-in for the CUDA runtime (see test_second_device.py) answers."""
import ctypes
import os
import shutil
import subprocess
import sys

import pytest
import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from nvfp4_w4a4_moe_permute_gb300 import build as B   # noqa: E402
from nvfp4_w4a4_moe_permute_gb300 import minite as M   # noqa: E402

P = 1 << 20   # an address that nothing reads
INVALID = 1
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


def backward(lib, rows=P, drows=2 * P, dweights=P, dy=P, T=8, M_=16, rs=64, drs=64, weights=P, status=None):
    return lib.minite_moe_combine_rows_backward(dy, 0, 64, rows, rs, P, weights, T, M_, 64, 2, drows, drs, dweights, status,
                                                None)


def test_no_tokens_is_nothing_to_do():
    B.build()
    lib = M.load()
    assert backward(lib, T=0, dy=None, dweights=None) == 0               # rows there, [0, k] weights' gradient
    assert backward(lib, T=0, dy=None, rows=None, drows=None, dweights=None, M_=0, rs=0) == 0
    assert backward(lib, T=0, dy=None, rows=None) == 0
    assert backward(lib, T=-1) != 0 and backward(lib, T=0, drs=63) != 0   # shapes are looked at all the same


def child():
    lib, runtime = M.load(), ctypes.CDLL(os.environ["LD_PRELOAD"])

    def launches(call):
        before = runtime.standin_launches()
        assert call() == 0
        return runtime.standin_launches() - before
    for dtype in (0, 1):
        # no rows: every slot is skipped, the weights' gradient is 0 and has to be written
        assert launches(lambda: backward(lib, rows=None, drows=None, M_=0, rs=0)) == 1
        assert launches(lambda: backward(lib, rows=None, drows=None, M_=0, rs=64)) == 1
        assert launches(lambda: backward(lib, rows=None, drows=None, M_=0, rs=0, status=P)) == 1
        # and without one there is nothing to write, but rows that are not there to report
        assert launches(lambda: backward(lib, rows=None, drows=None, dweights=None, M_=0, rs=0, status=P)) == 1
        spread = lambda M_, rows, status: lib.minite_moe_spread_rows(P, dtype, 64, P, 8, M_, 64, 2, rows, 64, status, None)
        assert launches(lambda: spread(0, None, P)) == 1
        assert launches(lambda: spread(0, None, None)) == 0
        assert launches(lambda: spread(16, 2 * P, None)) == 1
        assert spread(16, None, None) == INVALID
    # where there are rows the pair is checked as before
    assert backward(lib, rows=None) == INVALID and backward(lib, dweights=None) == INVALID
    assert backward(lib, drows=None) == INVALID and backward(lib, rows=2 * P, rs=72) == INVALID
    assert backward(lib, weights=None, rows=None, drows=None, M_=0, rs=0) == INVALID
    print("every call went through")


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_no_rows(tmp_path):
    from test_second_device import RUNTIME
    B.build()
    src, lib = tmp_path / "runtime.cpp", tmp_path / "runtime.so"
    src.write_text(RUNTIME)
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(B.nvcc_path()))), "include")
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", include, str(src), "-o", str(lib)], check=True)
    env = {**os.environ, "LD_PRELOAD": str(lib), "PYTHONPATH": B.ROOT}
    r = subprocess.run([sys.executable, os.path.abspath(__file__)], env=env, cwd=B.ROOT, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "every call went through" in r.stdout, r.stdout + r.stderr[-2000:]


if __name__ == "__main__":
    child()
