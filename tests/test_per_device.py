"""What a launch sets once per GPU is set on every GPU of the process, and a failure is not kept
(CPU only: the header that the launches use, with outcomes of the test's choice)."""
import ctypes as C
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_each_device_is_set_once(tmp_path):
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    so = str(tmp_path / "per_device.so")
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Wextra", "-Werror", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "quantized_moe_sigmoid_amd", "csrc"), os.path.join(ROOT, "tests", "per_device.cpp"),
                    "-o", so], check=True)
    L = C.CDLL(so)

    def once(device, outcome):
        ran = C.c_int(-1)
        return L.once_on(device, outcome, C.byref(ran)), ran.value

    assert once(0, 0) == (0, 1)
    assert once(0, 98) == (0, 0)   # done: not called again
    assert once(1, 98) == (98, 1)  # another GPU is set by itself; its failure is reported ..
    assert once(1, 0) == (0, 1)    # .. and not kept
    assert once(1, 98) == (0, 0)
    for d in range(2, 64):
        assert once(d, 0) == (0, 1) and once(d, 98) == (0, 0)
    for _ in range(2):
        assert once(64, 0) == (0, 1) and once(-1, 98) == (98, 1)
