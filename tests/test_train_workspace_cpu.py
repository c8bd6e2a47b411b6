"""Workspaces of the operators of a trainable expert block, and what they say of the
parts that sums are taken in (no GPU; made-up device pointers, as in
test_train_abi_cpu.py)."""
import re

import pytest
import torch

import mxfp4_grouped_gemm_amd as moe
from tests.test_train_abi_cpu import BAD, linear_bwd, permute

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="host-only checks pass invalid device "
                                "pointers; never run where a GPU is visible")


def needed(call, **kw):
    """Bytes that a call asks for."""
    assert call(wsb=0, **kw) == BAD
    return int(re.search(r"< (\d+) needed", moe.moe_last_error()).group(1))


def backward(T, K, N):
    return needed(linear_bwd, T=T, K=K, N=N, ldd=N, ldx=K, lddx=K)


@pytest.mark.parametrize("K,N", [(64, 10240), (128, 5120), (8, 8192), (64, 4096), (128, 4096)])
def test_long_sums_of_both_products(K, N):
    """From 3000 tokens on the sum of dw is taken in parts, unless dx's is as long and
    would be left whole on a few compute units: dx is in parts as with one token fewer
    (its fp32 parts, T * K each, are in the workspace beside dz and the bias sums)."""
    parts = lambda T: backward(T, K, N) - 2 * T * N  # noqa: E731
    assert parts(2999) >= 2 * 2999 * K * 4
    assert abs(parts(3000) - parts(2999)) <= 16 * K * 4 + N * 4 + 512


@pytest.mark.parametrize("T,K,N", [(3000, 64, 2048), (5000, 64, 4096), (8000, 256, 256), (3000, 512, 1280)])
def test_long_sums_of_dw(T, K, N):
    """dx's sum is shorter: dw's is in parts (fp32, N * K each)."""
    assert backward(T, K, N) - 2 * T * N >= 2 * N * K * 4


@pytest.mark.parametrize("T,K,N,n", [(128, 2048, 2048, 8), (129, 2048, 2048, 0), (256, 2048, 2048, 0), (256, 1024, 4096, 4),
                                     (300, 1024, 4104, 3), (256, 2048, 2560, 8), (150, 2048, 2816, 8), (256, 3584, 4096, 4)])
def test_parts_of_few_tokens(T, K, N, n):
    """dx's parts: of 129 to 512 tokens those beside 128 x 128 tiles of dw only where the
    weights are large (5 << 20 of them and more), a workgroup of 128 x 128 a compute unit
    and four steps each at least; else those of 64 x 64 tiles, which leave 256 tokens of
    2048 columns whole. (The bias sums: a part for 16 tokens.)"""
    assert backward(T, K, N) - 2 * T * N - -(-T // 16) * N * 4 - n * T * K * 4 in range(0, 768)


@pytest.mark.parametrize("k,E", [(1, 896), (8, 112), (15, 7), (64, 1024), (3, 1)])
def test_sort_workspace_does_not_shrink(k, E):
    """A buffer for the largest batch holds a smaller one's: its query never decreases
    with T, and no batch asks for more than its own query."""
    last = 0
    tokens = sorted({t for n in (1, 2560, 2561, 4096, 262144, 262145, 524288, 1 << 20, 1 << 22) for t in (n // k, n // k + 1, n)
                     if t <= 1 << 22} | set(range(0, 1 << 22, 99991)))
    for T in tokens:
        size = moe.moe_permute_workspace_size(T, k, E)
        assert size >= last, T
        last = size
        if size and T * k > 4096:
            assert needed(permute, T=T, k=k, E=E) <= size


@pytest.mark.parametrize("H", [8, 512, 520, 1024, 4096, 8192, 8200, 16384, 20000])
def test_layer_norm_workspace_does_not_shrink(H):
    last = 0
    for T in list(range(0, 6000, 7)) + [1 << 20, 1 << 24]:
        size = moe.moe_layer_norm_backward_workspace_size(T, H)
        assert size >= last, T
        last = size
