"""How the operators of a trainable expert block are launched: host code, no GPU."""
import ctypes
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mxfp4_grouped_gemm_amd", "csrc")


@pytest.fixture(scope="module")
def norm(tmp_path_factory):
    """layer_norm_plan.hpp as a library."""
    d = tmp_path_factory.mktemp("plan")
    (d / "plan.cpp").write_text('#include "layer_norm_plan.hpp"\nextern "C" {\n'
                                "int few(int T, int H) { return moe::layer_norm_few_rows(T, H); }\n"
                                "int groups(int T, int H, int sums) { return moe::layer_norm_row_groups(T, H, sums); }\n"
                                "int parts(int T, int H) { return moe::layer_norm_parts(T, H); }\n}\n")
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", CSRC, str(d / "plan.cpp"), "-o", str(d / "plan.so")], check=True)
    return ctypes.CDLL(str(d / "plan.so"))


WIDTHS = (1, 512, 513, 1024, 2048, 4096, 8192, 8193, 10001, 12288, 16384)
TOKENS = (1, 63, 64, 65, 100, 256, 320, 321, 400, 512, 513, 640, 641, 1000, 1024)


def test_rows_of_few_use_the_device(norm):
    """Row workgroups of the launch of few rows: one a compute unit for dx alone (or
    one a row), and no more than eight rows behind each other beside the sums."""
    for H in WIDTHS:
        for T in TOKENS:
            assert norm.few(T, H)
            rows = -(-T // 4) if H <= 512 else T
            assert norm.groups(T, H, 0) >= min(rows, 256), (T, H)
            assert -(-rows // norm.groups(T, H, 1)) <= 8, (T, H)
            assert norm.groups(T, H, 1) <= rows and norm.groups(T, H, 0) <= rows


def test_parts_are_what_the_workspace_holds(norm):
    """The sums' parts: none for few rows, else a row workgroup's each, or 64 runs."""
    for H in WIDTHS + (16385, 65536):
        assert norm.parts(0, H) == 0
        for T in TOKENS + (1025, 2049, 5000, 1 << 24):
            if norm.few(T, H):
                assert norm.parts(T, H) == 0
            elif H <= 8192:
                assert norm.parts(T, H) == norm.groups(T, H, 1) == norm.groups(T, H, 0)
            else:
                assert norm.parts(T, H) == min(T, 64)
