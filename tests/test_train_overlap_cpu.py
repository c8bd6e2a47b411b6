"""Rows of the layer norm's backward that overlap: refused before anything is
launched (no GPU; made-up device pointers, as in test_train_abi_cpu.py)."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

from tests.test_train_abi_cpu import BAD, P, norm_bwd, said

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mxfp4_grouped_gemm_amd", "csrc")

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="host-only checks pass invalid device "
                                "pointers; never run where a GPU is visible")

T, H = 4000, 64
FAR = 1 << 30
STOP = dict(T=T, ws=None)  # the check behind the overlap's: nothing is launched


def refused(**kw):
    return said(norm_bwd(**{**STOP, **kw}), "must not") == BAD


def passed(**kw):
    return said(norm_bwd(**{**STOP, **kw}), "null workspace") == BAD


@pytest.mark.parametrize("out", ["dx", "dres"])
@pytest.mark.parametrize("into", ["dy", "s"])
def test_outputs_that_share_rows_with_inputs(out, into):
    """At the input's own address, rows into it (forwards and back), inside a row, at
    its last byte and just beyond."""
    other = {"dy": "s", "s": "dy"}[into]
    base = {other: FAR, "dx": 2 * FAR, "dres": 3 * FAR, "dr": 4 * FAR}
    row = 2 * H
    for at in (0, row, 17 * row, -row, -17 * row, 2, -2, row + 6, (T - 1) * row, (T - 1) * row + row - 2, -T * row + 2):
        assert refused(**{**base, into: 8 * P, out: 8 * P + at}), at
    for at in (T * row, T * row + 2, -T * row):
        assert passed(**{**base, into: 8 * P, out: 8 * P + at}), at


def test_columns_of_one_buffer():
    """Rows beside each other in a wider buffer do not overlap; other strides are
    looked at row by row; another type has another row length."""
    far = dict(s=FAR, dx=2 * FAR, dres=3 * FAR, dr=4 * FAR)
    assert passed(**{**far, "dy": 8 * P, "lddy": 2 * H, "dx": 8 * P + 2 * H, "lddx": 2 * H})
    assert passed(**{**far, "dy": 8 * P + 2 * H, "lddy": 2 * H, "dx": 8 * P, "lddx": 2 * H})
    assert refused(**{**far, "dy": 8 * P, "lddy": 2 * H, "dx": 8 * P + 2 * H - 2, "lddx": 2 * H})
    assert refused(**{**far, "dy": 8 * P, "lddy": 2 * H, "dx": 8 * P + 2 * H, "lddx": 3 * H})
    # (rows of 128 bytes 256 apart, and between them rows 512 apart)
    assert passed(**{**far, "dy": 8 * P, "lddy": 2 * H, "dx": 8 * P + 2 * H, "lddx": 4 * H})
    assert refused(**{**far, "s": 8 * P, "lds": 2 * H, "st": 1, "dres": 8 * P + 4 * H, "lddres": 2 * H + 1})
    assert passed(**{**far, "s": 8 * P, "lds": 2 * H, "st": 1, "dres": 8 * P + 4 * H, "lddres": 2 * H})
    assert refused(**{**far, "s": 8 * P, "lds": 2 * H, "st": 1, "dx": 8 * P + 4 * H - 2, "lddx": 4 * H})


def test_the_streams_own_gradient():
    """dresidual_out's rows may be the output's own, not others of them."""
    far = dict(dy=FAR, s=2 * FAR)
    assert passed(**far, dr=8 * P, dx=8 * P, dres=4 * FAR) and passed(**far, dr=8 * P, dres=8 * P, dx=4 * FAR)
    assert refused(**far, dr=8 * P, dx=8 * P + 2 * H, dres=4 * FAR)
    assert refused(**far, dr=8 * P, dres=8 * P - 2 * H, dx=4 * FAR)
    assert refused(**far, dr=8 * P, st=1, dx=8 * P, dres=4 * FAR)  # another element size


def test_overlap_of_rows_against_all_pairs(tmp_path):
    """rows_overlap against every pair of rows."""
    (tmp_path / "o.cpp").write_text('#include "rows_overlap.hpp"\nextern "C" int overlap(int64_t p, int64_t sp, int64_t lp, int64_t q, '
                                    "int64_t sq, int64_t lq, int n) {\n    return moe::abi::rows_overlap(p, sp, lp, q, sq, lq, n);\n}\n")
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", CSRC, str(tmp_path / "o.cpp"), "-o", str(tmp_path / "o.so")],
                   check=True)
    f = ctypes.CDLL(str(tmp_path / "o.so")).overlap
    f.argtypes = [ctypes.c_int64] * 6 + [ctypes.c_int]
    g = np.random.default_rng(1)
    seen = [0, 0]
    for _ in range(20000):
        n = int(g.integers(1, 9))
        lp, lq = (int(v) for v in g.integers(1, 9, 2))
        sp = lp + int(g.integers(0, 9))
        sq = sp if g.random() < 0.4 and sp >= lq else lq + int(g.integers(0, 12))
        p, q = 1000, 1000 + int(g.integers(-100, 100))
        want = any(p + i * sp < q + j * sq + lq and q + j * sq < p + i * sp + lp for i in range(n) for j in range(n))
        assert bool(f(p, sp, lp, q, sq, lq, n)) == want, (p, sp, lp, q, sq, lq, n)
        seen[want] += 1
    assert min(seen) > 2000
