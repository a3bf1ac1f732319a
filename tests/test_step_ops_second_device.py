"""Rows by expert on a device that is new to them: their launches, with the shared
memory that they ask for, go through there too (see test_second_device.py, whose
stand-in for the CUDA runtime answers here)."""
import ctypes
import os
import shutil
import subprocess
import sys

import pytest

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from nvfp4_w4a4_moe_permute_gb300 import build as B   # noqa: E402

P = 1 << 20   # an address that nothing reads


def steps(lib):
    for dtype in (0, 1):
        yield "combine", lambda: lib.minite_moe_combine_rows(P, dtype, 64, P, P, 8, 16, 64, 2, P, 64, None, None)
        yield "gradient", lambda: lib.minite_moe_combine_rows_backward(P, dtype, 64, P, 64, P, P, 8, 16, 64, 2, 2 * P, 64,
                                                                       P, None, None)
        yield "rows' gradient", lambda: lib.minite_moe_combine_rows_backward(P, dtype, 64, None, 64, P, P, 8, 16, 64, 2,
                                                                             2 * P, 64, None, None, None)
        for T in (4, 4000, 200000):
            yield "permute", lambda: lib.minite_moe_permute_rows(P, dtype, 64, P, T, 64, 1024, 8, 2 * P, 64, P, P, P, P,
                                                                 1 << 30, None, None)


def child():
    from nvfp4_w4a4_moe_permute_gb300 import minite as M
    lib, runtime = M.load(), ctypes.CDLL(os.environ["LD_PRELOAD"])
    for what, call in steps(lib):
        for device in (0, 1, 0, 5):
            runtime.standin_set_device(device)
            before = runtime.standin_launches()
            rc = call()
            assert rc == 0 and runtime.standin_launches() > before, f"{what} on device {device}: status {rc}"
    print("every call went through")


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_every_device_gets_its_shared_memory(tmp_path):
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
