"""Refusals of the trainable block's C ABI (no GPU; nothing is launched). As in
test_abi_cpu.py, the calls pass null or made-up device pointers, so this file
runs only where no GPU is visible."""
import pytest
import torch

import mxfp4_grouped_gemm_amd as moe
from tests import train_ref as ref

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="host-only checks pass invalid device "
                                "pointers; never run where a GPU is visible")

L = moe.lib
OK, BAD, NOT = moe.MOE_OK, moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED
P = 1 << 20  # a made-up aligned address
BIG = 1 << 50


def said(status, text):
    assert text in moe.moe_last_error(), moe.moe_last_error()
    return status


def norm(x=P, ldx=64, r=P, ldr=64, rt=0, w=P, b=P, wt=0, eps=1e-5, T=4, H=64, ro=P, ldro=64, y=P, ldy=64, m=P, q=P):
    return L.moe_layer_norm_forward(x, ldx, r, ldr, rt, w, b, wt, eps, T, H, ro, ldro, y, ldy, m, q, None)


def test_layer_norm_refusals():
    assert said(norm(T=-1), "T=-1") == BAD and norm(T=(1 << 24) + 1) == NOT
    assert norm(H=0) == BAD and norm(H=65537, ldx=65537) == NOT
    assert said(norm(rt=2), "type") == NOT and norm(wt=-1) == NOT
    for eps in (-1e-6, float("nan"), float("inf")):
        assert said(norm(eps=eps), "eps") == BAD
    for k in ("ldx", "ldr", "ldro", "ldy"):
        assert said(norm(**{k: 63}), "stride") == BAD and norm(**{k: (1 << 20) + 1}) == NOT
    assert norm(T=0, x=None, w=None) == OK
    assert said(norm(m=None), "together") == BAD and norm(q=None) == BAD
    assert said(norm(ro=None, y=None, m=None, q=None), "no output") == BAD
    assert said(norm(x=None), "null") == BAD and norm(w=None) == BAD
    for k in ("x", "y", "b", "w"):
        assert said(norm(**{k: P + 1}), "misaligned") == BAD
    assert norm(r=P + 2, rt=1) == BAD and norm(w=P + 2, wt=1) == BAD and norm(b=P + 2, wt=1) == BAD
    assert norm(m=P + 2) == BAD and norm(q=P + 1) == BAD


def norm_bwd(dy=P, lddy=64, s=P, lds=64, st=0, m=P, q=P, w=P, wt=0, dr=P, lddr=64, T=4, H=64, dx=2 * P, lddx=64,
             dres=3 * P, lddres=64, dw=P, db=P, ws=P, wsb=BIG):
    return L.moe_layer_norm_backward(dy, lddy, s, lds, st, m, q, w, wt, dr, lddr, T, H, dx, lddx, dres, lddres, dw, db,
                                     ws, wsb, None)


def test_layer_norm_backward_refusals():
    assert norm_bwd(T=-1) == BAD and norm_bwd(T=(1 << 24) + 1) == NOT
    assert norm_bwd(H=0) == BAD and norm_bwd(H=1 << 17, lddy=1 << 17) == NOT
    assert norm_bwd(st=2) == NOT and norm_bwd(wt=3) == NOT
    for k in ("lddy", "lds", "lddr", "lddx", "lddres"):
        assert said(norm_bwd(**{k: 60}), "stride") == BAD and norm_bwd(**{k: (1 << 20) + 1}) == NOT
    assert said(norm_bwd(dx=None, dres=None, dw=None, db=None), "no output") == BAD
    assert norm_bwd(T=0, dy=None, dx=None, dres=None, dw=None, db=None) == OK
    for k in ("dy", "s", "m", "q", "w"):
        assert said(norm_bwd(**{k: None}), "null") == BAD and said(norm_bwd(**{k: P + 1}), "misaligned") == BAD
    for k in ("dx", "dres", "dw", "db"):
        assert said(norm_bwd(**{k: P + 1}), "misaligned output") == BAD
    for k in ("dx", "dres"):
        assert said(norm_bwd(**{k: P}), "must not be dy or s") == BAD
    assert norm_bwd(s=P + 2, st=1) == BAD and norm_bwd(dr=P + 2, st=1) == BAD and norm_bwd(dw=P + 2, wt=1) == BAD
    need = moe.moe_layer_norm_backward_workspace_size(4000, 64)
    assert need > 0 and need % 256 == 0
    assert said(norm_bwd(T=4000, wsb=need - 1), "workspace") == BAD
    assert norm_bwd(T=4000, ws=None) == BAD and norm_bwd(T=4000, ws=P + 64) == BAD
    for args in ((-1, 64), (4, 0), (4, 65537), ((1 << 24) + 1, 64)):
        assert moe.moe_layer_norm_backward_workspace_size(*args) == -1
    assert moe.moe_layer_norm_backward_workspace_size(0, 64) == 0


def permute(x=P, ldx=64, dt=0, ids=P, T=4, k=2, E=8, H=64, out=P, ldo=64, rows=P, off=P, ws=P, wsb=BIG):
    return L.moe_permute(x, ldx, dt, ids, T, k, E, H, out, ldo, rows, off, ws, wsb, None)


def test_permute_refusals():
    assert said(permute(T=-1), "T=-1") == BAD and permute(T=(1 << 22) + 1) == NOT
    assert permute(k=0) == BAD and permute(k=65) == NOT
    assert permute(E=0) == BAD and permute(E=1025) == NOT
    assert permute(H=0) == BAD and permute(H=(1 << 18) + 1, ldx=1 << 19, ldo=1 << 19) == NOT
    assert said(permute(dt=3), "type") == NOT
    assert said(permute(ldx=63), "x_stride") == BAD and permute(ldo=63) == BAD and permute(ldo=(1 << 20) + 1) == NOT
    for k in ("x", "ids", "out", "rows", "off"):
        assert said(permute(**{k: None}), "null") == BAD
    for k in ("x", "out"):
        assert said(permute(**{k: P + 1}), "misaligned") == BAD and permute(dt=1, **{k: P + 2}) == BAD
    for k in ("ids", "rows", "off"):
        assert permute(**{k: P + 2}) == BAD
    need = moe.moe_permute_workspace_size(4000, 8, 64)
    assert need > 0 and need % 256 == 0
    assert said(permute(T=4000, k=8, E=64, wsb=need - 1), "workspace") == BAD and permute(T=4000, k=8, E=64, ws=None) == BAD
    for args in ((-1, 2, 8), (4, 0, 8), (4, 65, 8), (4, 2, 0), (4, 2, 1025), ((1 << 22) + 1, 2, 8)):
        assert moe.moe_permute_workspace_size(*args) == -1


def unpermute(y=P, ldy=64, yt=0, rows=P, w=P, r=P, ldr=64, T=4, k=2, H=64, out=P, ldo=64, ot=0):
    return L.moe_unpermute(y, ldy, yt, rows, w, r, ldr, T, k, H, out, ldo, ot, None)


def test_unpermute_refusals():
    assert unpermute(T=-1) == BAD and unpermute(T=(1 << 22) + 1) == NOT
    assert unpermute(k=0) == BAD and unpermute(k=65) == NOT and unpermute(H=0) == BAD
    assert said(unpermute(yt=2), "type") == NOT and unpermute(ot=2) == NOT
    for k in ("ldy", "ldr", "ldo"):
        assert said(unpermute(**{k: 63}), "stride") == BAD and unpermute(**{k: (1 << 20) + 1}) == NOT
    for k in ("y", "rows", "out"):
        assert said(unpermute(**{k: None}), "null") == BAD
    for k in ("y", "rows", "w", "r", "out"):
        assert said(unpermute(**{k: P + 1}), "misaligned") == BAD
    assert unpermute(y=P + 2, yt=1) == BAD and unpermute(r=P + 2, ot=1) == BAD
    assert unpermute(T=0, y=None, rows=None, out=None) == OK


def unpermute_bwd(d=P, ldd=64, ot=0, rows=P, w=P, y=P, ldy=64, yt=0, T=4, k=2, H=64, dy=P, lddy=64, dw=P):
    return L.moe_unpermute_backward(d, ldd, ot, rows, w, y, ldy, yt, T, k, H, dy, lddy, dw, None)


def test_unpermute_backward_refusals():
    assert unpermute_bwd(T=-1) == BAD and unpermute_bwd(k=0) == BAD and unpermute_bwd(H=0) == BAD
    assert unpermute_bwd(T=(1 << 22) + 1) == NOT and unpermute_bwd(k=65) == NOT
    assert unpermute_bwd(yt=2) == NOT and unpermute_bwd(ot=5) == NOT
    for k in ("ldd", "ldy", "lddy"):
        assert said(unpermute_bwd(**{k: 63}), "stride") == BAD
    assert said(unpermute_bwd(dy=None, dw=None), "no output") == BAD
    for k in ("d", "rows", "y"):
        assert said(unpermute_bwd(**{k: None}), "null") == BAD
    for k in ("d", "rows", "w", "y", "dy", "dw"):
        assert said(unpermute_bwd(**{k: P + 1}), "misaligned") == BAD
    assert unpermute_bwd(T=0, d=None, rows=None, y=None, dy=None, dw=None) == OK


def linear(x=P, ldx=64, w=P, b=P, bt=0, act=3, add=P, lda=32, T=100, K=64, N=32, out=P, ldo=32, ot=0, pre=P, ws=P,
           wsb=BIG):
    return L.moe_linear_forward(x, ldx, w, b, bt, act, add, lda, T, K, N, out, ldo, ot, pre, ws, wsb, None)


def test_linear_refusals():
    assert said(linear(act=5), "activation") == NOT and linear(act=-1) == NOT
    assert linear(T=-1) == BAD and linear(T=(1 << 24) + 1) == NOT
    assert said(linear(K=60), "K=60") == BAD and linear(N=12) == BAD and linear(N=0) == BAD
    assert linear(K=(1 << 18) + 8, ldx=1 << 19) == NOT
    assert linear(bt=2) == NOT and linear(ot=2) == NOT
    assert linear(ldx=56) == BAD and linear(ldo=36) == BAD and said(linear(lda=24), "addend_stride") == BAD
    for k in ("x", "w", "out"):
        assert said(linear(**{k: None}), "null") == BAD and said(linear(**{k: P + 8}), "16-byte") == BAD
    for k in ("b", "add", "pre"):
        assert linear(**{k: P + 8}) == BAD
    assert linear(T=0, x=None) == OK
    need = moe.moe_linear_workspace_size(100, 4096, 64)
    assert need > 0 and need % 256 == 0
    assert said(linear(K=4096, ldx=4096, N=64, ldo=64, lda=64, wsb=need - 1), "workspace") == BAD
    for args in ((-1, 64, 32), (1, 60, 32), (1, 64, 4)):
        assert moe.moe_linear_workspace_size(*args) == -1
        assert moe.moe_linear_backward_workspace_size(*args) == -1


def linear_bwd(d=P, ldd=32, dt=0, x=P, ldx=64, pre=P, w=P, act=3, T=100, K=64, N=32, dx=P, lddx=64, dw=P, db=P, bt=0,
               ws=P, wsb=BIG):
    return L.moe_linear_backward(d, ldd, dt, x, ldx, pre, w, act, T, K, N, dx, lddx, dw, db, bt, ws, wsb, None)


def test_linear_backward_refusals():
    assert linear_bwd(act=7) == NOT and linear_bwd(T=-1) == BAD and linear_bwd(K=60) == BAD and linear_bwd(N=20) == BAD
    assert linear_bwd(dt=2) == NOT and linear_bwd(bt=2) == NOT
    assert linear_bwd(ldd=36) == BAD and linear_bwd(ldx=60) == BAD and linear_bwd(lddx=8) == BAD
    for k in ("d", "x", "pre", "w"):
        assert said(linear_bwd(**{k: None}), "null") == BAD and said(linear_bwd(**{k: P + 8}), "16-byte") == BAD
    for k in ("dx", "dw", "db"):
        assert linear_bwd(**{k: P + 8}) == BAD
    assert said(linear_bwd(dx=None, dw=None, db=None), "no output") == BAD
    assert linear_bwd(T=0, d=None, x=None, pre=None, w=None, dx=None, dw=None, db=None, ws=None, wsb=0) == OK
    need = moe.moe_linear_backward_workspace_size(100, 64, 32)
    assert need >= 100 * 32 * 2 and need % 256 == 0
    assert said(linear_bwd(wsb=need - 1), "workspace") == BAD and linear_bwd(ws=None) == BAD
    # what is not read may be missing, and the next check is reached
    assert said(linear_bwd(act=0, pre=None, wsb=0), "workspace") == BAD
    assert said(linear_bwd(dw=None, x=None, wsb=0), "workspace") == BAD
    assert said(linear_bwd(dx=None, w=None, wsb=0), "workspace") == BAD


def test_binding_refuses_host_tensors():
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    w, v = torch.zeros(8, 64, dtype=torch.bfloat16), torch.zeros(64, dtype=torch.bfloat16)
    ids = torch.zeros(2, 1, dtype=torch.int32)
    for call in (lambda: moe.moe_layer_norm_forward(x, v), lambda: moe.moe_layer_norm(x, v),
                 lambda: moe.moe_permute(x, ids, 4), lambda: moe.moe_dispatch(x, ids, 4), lambda: moe.moe_unpermute(x, ids),
                 lambda: moe.moe_combine(x, ids), lambda: moe.moe_unpermute_backward(x, ids),
                 lambda: moe.moe_linear_forward(x, w), lambda: moe.moe_linear(x, w),
                 lambda: moe.moe_linear_backward(torch.zeros(2, 8, dtype=torch.bfloat16), x, w)):
        with pytest.raises(ValueError, match="GPU"):
            call()
    with pytest.raises(TypeError):
        moe.moe_linear_forward([1.0], w)


def test_reference_permutation():
    """The oracle against a stable sort."""
    g = torch.Generator().manual_seed(1)
    for T, k, E in ((1, 1, 1), (5, 3, 4), (70, 2, 9)):
        ids = torch.randint(-1, E + 1, (T, k), generator=g, dtype=torch.int32)
        x = torch.randn(T, 3, generator=g)
        out, rows, offsets = ref.permute(x, ids, E)
        key = ids.flatten().where((ids.flatten() >= 0) & (ids.flatten() < E), torch.tensor(E, dtype=torch.int32))
        order = torch.sort(key, stable=True).indices
        assert torch.equal(out[:offsets[E]], x[order[:offsets[E]] // k]) and not bool(out[offsets[E]:].any())
        place = torch.where(rows < 0, -1 - rows, rows).flatten().long()
        assert torch.equal(order[place], torch.arange(T * k)) and torch.equal(rows.flatten() < 0, key == E)


@pytest.mark.parametrize("a", range(5))
def test_reference_slopes(a):
    """The oracle's slopes against differences of its activations."""
    z = torch.linspace(-6, 6, 241, dtype=torch.float64) + 0.013
    e = 1e-6
    d = (ref.act(a, z + e)[0] - ref.act(a, z - e)[0]) / (2 * e)
    assert float((d - ref.slope(a, z)[0]).abs().max()) < 1e-8


def test_reference_layer_norm_backward():
    """The oracle's gradients against differences of its forward."""
    g = torch.Generator().manual_seed(2)
    x, w, b, dy = (torch.randn(*s, generator=g, dtype=torch.float64) for s in ((3, 7), (7,), (7,), (3, 7)))
    _, _, mean, rstd = ref.layer_norm(x, None, w, b, 1e-5)
    (ds, dw, db), _ = ref.layer_norm_backward(dy, x, mean, rstd, w)

    def loss(x, w, b):
        return float((ref.layer_norm(x, None, w, b, 1e-5)[1] * dy).sum())
    e = 1e-6
    for k, (t, grad) in enumerate(((x, ds), (w, dw), (b, db))):
        step = torch.randn(*t.shape, generator=g, dtype=torch.float64)
        hi, lo = ([u + s * e * step if i == k else u for i, u in enumerate((x, w, b))] for s in (1, -1))
        assert abs((loss(*hi) - loss(*lo)) / (2 * e) - float((grad * step).sum())) < 1e-7
