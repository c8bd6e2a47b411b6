"""Refusals of the dense operators' C ABI (no GPU; nothing is launched). As in
test_abi_cpu.py, the calls pass null or made-up device pointers, so this file
runs only where no GPU is visible."""
import ctypes
import os
import subprocess
import sys

import pytest
import torch

import mxfp4_grouped_gemm_amd as moe

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="host-only checks pass invalid device "
                                "pointers; never run where a GPU is visible")

L = moe.lib
BAD, NOT = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED
P = 1 << 20  # a made-up aligned address
BIG = 1 << 50


def said(status, text):
    assert text in moe.moe_last_error(), moe.moe_last_error()
    return status


def norm(x=P, ldx=64, r=P, ldr=64, rt=0, w=P, wt=0, eps=1e-6, T=4, H=64, ro=P, ldro=64, y=P, ldy=64, q=P, ldq=64,
         qs=P, ldqs=2):
    return L.moe_rms_norm(x, ldx, r, ldr, rt, w, wt, eps, 0.0, T, H, ro, ldro, y, ldy, q, ldq, qs, ldqs, None)


def test_norm_refusals():
    assert said(norm(T=-1), "T=-1") == BAD
    assert norm(T=(1 << 24) + 1) == NOT
    assert norm(H=0) == BAD
    assert norm(H=65568, ldx=65568) == NOT
    assert said(norm(rt=2), "type") == NOT and norm(wt=7) == NOT
    for eps in (-1e-6, float("nan"), float("inf")):
        assert said(norm(eps=eps), "eps") == BAD
    assert said(norm(qs=None), "together") == BAD and norm(q=None) == BAD
    assert said(norm(H=48, ldqs=2), "multiple of 32") == BAD
    for k in ("ldx", "ldr", "ldro", "ldy", "ldq"):
        assert said(norm(**{k: 63}), "stride") == BAD
        assert norm(**{k: (1 << 20) + 1}) == NOT
    assert norm(ldqs=1) == BAD
    assert norm(T=0) == moe.MOE_OK
    assert said(norm(ro=None, y=None, q=None, qs=None), "no output") == BAD
    assert said(norm(x=None), "null") == BAD and norm(w=None) == BAD
    assert said(norm(x=P + 1), "misaligned") == BAD and norm(r=P + 2, rt=1) == BAD and norm(w=P + 2, wt=1) == BAD


def lora(a=P, b=P, index=P, ranks=P, scale=P, n=4, rank=16):
    return moe._CLora(a, b, index, ranks, scale, n, rank)


def linear(x=P, ldx=64, w=P, lo=None, T=100, K=64, N=32, out=P, ldo=32, ot=0, ws=P, wsb=BIG):
    return L.moe_lora_linear(x, ldx, w, lo, T, K, N, out, ldo, ot, ws, wsb, None)


def test_linear_refusals():
    assert linear(T=-1) == BAD and linear(T=(1 << 24) + 1) == NOT
    assert said(linear(K=60), "K=60") == BAD and linear(K=0) == BAD and linear(N=12) == BAD
    assert linear(K=(1 << 18) + 8, ldx=1 << 19) == NOT
    assert linear(ldx=56) == BAD and said(linear(ldx=68), "x_stride") == BAD and linear(ldo=33) == BAD
    assert linear(ldx=(1 << 20) + 8) == NOT
    assert linear(ot=2) == NOT
    assert linear(x=None) == BAD and linear(w=None) == BAD and linear(out=None) == BAD
    assert said(linear(x=P + 8), "16-byte") == BAD
    assert linear(T=0, x=None) == moe.MOE_OK
    for bad in (dict(n=0), dict(rank=0), dict(rank=12), dict(a=None), dict(b=None), dict(index=None), dict(a=P + 8),
                dict(index=P + 2), dict(ranks=P + 1), dict(scale=P + 2)):
        assert said(linear(lo=lora(**bad)), "lora") == BAD, bad
    assert linear(lo=lora(rank=264)) == NOT and linear(lo=lora(n=(1 << 24) + 1)) == NOT
    need = moe.moe_lora_linear_workspace_size(100, 64, 32, 16)
    assert need >= 100 * 32 * 4 and need % 256 == 0
    assert said(linear(lo=lora(), wsb=need - 1), "workspace") == BAD
    assert linear(lo=lora(), ws=None) == BAD and linear(lo=lora(), ws=P + 16) == BAD
    for args in ((-1, 64, 32, 0), (1, 60, 32, 0), (1, 64, 4, 0), (1, 64, 32, 4), (1, 64, 32, 264)):
        assert moe.moe_lora_linear_workspace_size(*args) == -1


def ffn(x=P, ldx=64, w13=P, w2=P, act=0, add=P, lda=64, l13=None, l2=None, T=100, H=64, I=40, out=P, ldo=64, gu=P,
        ws=P, wsb=BIG):
    return L.moe_ffn_forward(x, ldx, w13, w2, act, add, lda, l13, l2, T, H, I, out, ldo, gu, ws, wsb, None)


def test_ffn_refusals():
    assert said(ffn(act=1), "activation") == NOT
    assert ffn(T=-1) == BAD and ffn(T=(1 << 24) + 1) == NOT
    assert ffn(H=60) == BAD and ffn(I=4) == BAD and ffn(I=(1 << 18) + 8) == NOT
    assert ffn(ldx=60) == BAD and ffn(ldo=70) == BAD and ffn(lda=32) == BAD
    for k in ("x", "w13", "w2", "out"):
        assert said(ffn(**{k: None}), "null") == BAD and ffn(**{k: P + 8}) == BAD
    assert ffn(add=P + 2) == BAD and ffn(gu=P + 4) == BAD
    assert said(ffn(l13=lora(n=-1)), "lora13") == BAD and said(ffn(l2=lora(rank=4)), "lora2") == BAD
    assert ffn(T=0, x=None, ws=None) == moe.MOE_OK
    need = moe.moe_ffn_workspace_size(100, 64, 40, 16, 8)
    assert said(ffn(l13=lora(), l2=lora(rank=8), wsb=need - 1), "workspace") == BAD
    assert ffn(ws=None) == BAD and ffn(ws=P + 128) == BAD
    assert moe.moe_ffn_workspace_size(1, 64, 40) >= 80
    for args in ((-1, 64, 40), (1, 62, 40), (1, 64, 0), (1, 64, 40, 9), (1, 64, 40, 0, 512)):
        assert moe.moe_ffn_workspace_size(*args) == -1


def mx(act=0, add=P, lda=64, T=100, H=64, I=96, ldo=64, ws=P, wsb=BIG, **kw):
    p = [kw.get(k, P) for k in ("x", "xs", "w13", "w13s", "w2", "w2s")]
    return L.moe_ffn_forward_mxfp8(*p, act, add, lda, T, H, I, kw.get("out", P), ldo, ws, wsb, None)


def test_ffn_mxfp8_refusals():
    assert mx(act=3) == NOT
    assert mx(T=-1) == BAD and mx(H=48) == BAD and mx(I=40) == BAD and mx(H=(1 << 18) + 32) == NOT
    assert mx(ldo=60) == BAD and mx(lda=60) == BAD
    for k in ("x", "xs", "w13", "w13s", "w2", "w2s", "out"):
        assert said(mx(**{k: None}), "null") == BAD and mx(**{k: P + 8}) == BAD
    assert mx(add=P + 8) == BAD
    need = moe.moe_ffn_mxfp8_workspace_size(100, 64, 96)
    assert said(mx(wsb=need - 1), "workspace") == BAD and mx(ws=None) == BAD
    assert mx(T=0, x=None) == moe.MOE_OK
    assert moe.moe_ffn_mxfp8_workspace_size(1, 64, 40) == -1


def bwd(dout=P, ldd=64, x=P, ldx=64, gu=P, w13=P, w2=P, act=0, T=100, H=64, I=40, dx=P, lddx=64, d13=P, d2=P, ws=P,
        wsb=BIG):
    return L.moe_ffn_backward(dout, ldd, x, ldx, gu, w13, w2, act, T, H, I, dx, lddx, d13, d2, ws, wsb, None)


def test_ffn_backward_refusals():
    assert bwd(act=1) == NOT
    assert bwd(T=-1) == BAD and bwd(H=60) == BAD and bwd(I=44) == BAD
    assert bwd(ldd=60) == BAD and bwd(ldx=65) == BAD and bwd(lddx=8) == BAD
    for k in ("dout", "x", "gu", "w13", "w2"):
        assert said(bwd(**{k: None}), "null") == BAD and bwd(**{k: P + 8}) == BAD
    assert said(bwd(dx=None, d13=None, d2=None), "no output") == BAD
    assert bwd(dx=P + 8) == BAD and bwd(d13=P + 8) == BAD and bwd(d2=P + 2) == BAD
    need = moe.moe_ffn_backward_workspace_size(100, 64, 40)
    assert said(bwd(wsb=need - 1), "workspace") == BAD and bwd(ws=None) == BAD
    assert moe.moe_ffn_backward_workspace_size(1, 60, 40) == -1


def test_binding_refuses_host_tensors():
    x, w = torch.zeros(2, 64, dtype=torch.bfloat16), torch.zeros(64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):
        moe.moe_rms_norm(x, w)
    with pytest.raises(ValueError, match="GPU"):
        moe.moe_lora_linear(x, torch.zeros(8, 64, dtype=torch.bfloat16))
    with pytest.raises(TypeError):
        moe.moe_lora_linear([1.0], x)
    with pytest.raises(ValueError, match="GPU"):
        moe.moe_ffn_forward(x, torch.zeros(16, 64, dtype=torch.bfloat16), torch.zeros(64, 8, dtype=torch.bfloat16))


def test_workspaces_hold_what_the_calls_keep():
    """At least the intermediate tensors of the batch, in whole 256 bytes."""
    H, I = 3584, 2048
    for T in (1, 16, 17, 32, 33, 64, 65, 128, 1000, 8192):
        for need, least in ((moe.moe_ffn_workspace_size(T, H, I), T * I * 2),
                            (moe.moe_ffn_workspace_size(T, H, I, 16, 64), T * I * 2 + T * 64 * 4),
                            (moe.moe_ffn_mxfp8_workspace_size(T, H, I), T * I + T * I // 32),
                            (moe.moe_ffn_backward_workspace_size(T, H, I), T * I * 6),
                            (moe.moe_lora_linear_workspace_size(T, H, I, 8), T * 8 * 4)):
            assert need >= least and need % 256 == 0, (T, need, least)
    assert moe.moe_lora_linear_workspace_size(16, H, I) == 0
    assert ctypes.sizeof(moe._CLora) == 48


@pytest.mark.parametrize("call", [
    "moe_lora_linear_workspace_size(0, 8192, 152064)", "moe_lora_linear_workspace_size(0, 8192, 152064, 16)",
    "moe_ffn_workspace_size(0, 16384, 32768)", "moe_ffn_workspace_size(0, 16384, 32768, 8, 8)",
    "moe_ffn_mxfp8_workspace_size(0, 32768, 65536)", "moe_ffn_backward_workspace_size(0, 16384, 32768)"])
def test_workspaces_of_no_tokens_beside_large_weights(call):
    """Weights above 2 GiB are not for the few-token kernels: the tiles' rule
    for parts of K has to take no tiles too (in a process of its own, since a
    division by zero ends it)."""
    r = subprocess.run([sys.executable, "-c", f"import mxfp4_grouped_gemm_amd as m; print(m.{call})"],
                       capture_output=True, text=True, cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0 and r.stdout.split() == ["0"], (r.returncode, r.stdout, r.stderr[-500:])


def test_ffn_backward_of_no_tokens_with_only_an_empty_dx():
    """An empty tensor's address is null: not a call without outputs."""
    assert bwd(T=0, dout=None, x=None, gu=None, dx=None, d13=None, d2=None, ws=None, wsb=0) == moe.MOE_OK
    assert said(bwd(T=1, dx=None, d13=None, d2=None), "no output") == BAD
    assert bwd(T=0, lddx=8, d13=None, d2=None) == BAD  # what is given is checked as ever
    assert bwd(T=0, dx=None, d13=None, d2=P + 2) == BAD
