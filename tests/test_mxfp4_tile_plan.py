"""The plan of the tiled MXFP4 products, walked on the CPU from the header that the kernels use:
every weight row a workgroup loads lies in the matrix, and no buffer or scale window is filled
again before every wavefront has read it (CPU only, no kernel runs)."""
import ctypes as C
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    so = str(tmp_path_factory.mktemp("plan") / "plan.so")
    subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-Wextra", "-Werror", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "quantized_moe_sigmoid_amd", "csrc"),
                    os.path.join(ROOT, "tests", "mx_tile_walk.cpp"), "-o", so], check=True)
    return C.CDLL(so)


@pytest.mark.parametrize("BN,BM,slots", [(256, 256, 256), (128, 128, 512)])
def test_dense_weight_rows_stay_inside(plan, BN, BM, slots):
    """Every N up to several strips, and larger odd ones, with the strip that the launch takes."""
    sizes = list(range(1, 4200)) + [5000, 9801, 10300, 11003, 12000, 12288, 20001, 50257, 1 << 20]
    for N in sizes:
        for M in (17, 129, 513, 2000, 4096) if N > 1200 else (17, 100000):
            strip = plan.dense_strip_of(N, BN, (M + BM - 1) // BM, slots)
            assert plan.walk_rows(0, N, BN, strip) >= 0, (M, N, strip)


def test_dense_strips_of_several_tiles_are_met(plan):
    """The sizes above do take strips of more than one tile with a short last tile."""
    assert plan.dense_strip_of(5000, 256, 8, 256) > 0
    assert any(plan.dense_strip_of(N, 256, (4096 + 255) // 256, 256) > 1 for N in (5000, 9801, 12000))


@pytest.mark.parametrize("strip", range(1, 9))
def test_expert_weight_rows_stay_inside(plan, strip):
    """hidden and ffn are multiples of 128: down tiles of 256 columns, gate/up tiles of 128 features."""
    for n in range(128, 8192 + 128, 128):
        assert plan.walk_rows(0, n, 256, strip) >= 0, n
        assert plan.walk_rows(1, n, 256, strip) >= 0, n


def test_expert_buffers_and_windows_are_read_before_they_are_refilled(plan):
    """Rows of every multiple of 128 inputs that the experts' products take on the tiled kernel."""
    for nb in range(4, 260, 4):
        nst = (nb + 7) // 8
        if nb >= 16:
            for cols in range(1, plan.strip_experts(nb) + 1):
                assert plan.walk_experts(nst, cols) == 0, (nb, cols)
        else:
            for cols in range(1, plan.strip_experts_short(nb) + 1):
                assert plan.walk_experts_short(nst, cols) == 0, (nb, cols)


def test_walk_sees_a_window_refilled_early(plan):
    """Three buffers, an odd number of stages, two column tiles: the walk reports the conflict."""
    for nst in range(3, 33, 2):
        assert plan.walk_experts(nst, 2) == 5
        assert plan.walk_experts(nst + 1, 2) == 0


@pytest.mark.parametrize("cols", range(1, 9))
def test_dense_buffers_and_windows_are_read_before_they_are_refilled(plan, cols):
    for nst in range(1, 60):
        assert plan.walk_dense(nst, cols) == 0, nst
        assert plan.walk_dense_small(nst, cols) == 0, nst
