"""The operators of a trainable expert block against plain fp64 forms (MI355X).
Tolerances: tests/train_ref.py, tests/dense_ref.py."""
import math

import pytest
import torch

from tests import dense_ref, train_ref as ref

pytestmark = pytest.mark.gpu

B8 = 2.0 ** -8   # half a bf16 step, relative
F24 = 2.0 ** -24
BF, F32, U8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
HALF = {BF: B8, F32: F24}


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import mxfp4_grouped_gemm_amd as m
    return m


def gen(seed):
    return torch.Generator().manual_seed(seed)


def rnd(g, *shape, scale=1.0, dtype=BF):
    return (torch.randn(*shape, generator=g) * scale).to(dtype)


def cuda(v):
    return None if v is None else v.cuda()


def dbl(v):
    return None if v is None else v.double().cpu()


def near(got, want, tol, what=""):
    """|got - want| <= half a step of got's type + tol, element by element."""
    got, half = dbl(got), HALF[got.dtype]
    assert got.shape == want.shape, f"{what}: {tuple(got.shape)}"
    if not want.numel():
        return
    assert bool(torch.isfinite(got).all()), f"{what}: not finite"
    over = (got - want).abs() - (half * (want.abs() + tol) + tol)
    assert float(over.max()) <= 0, f"{what}: {float(over.max()):.3g} over at {int(over.argmax())}"


# ------------------------------------------------------------------ layer norm
# (one row to thousands; widths at the borders of the kernels' row sizes, odd ones)
NORMS = [(1, 1), (3, 7), (1, 3584), (5, 33), (2, 512), (7, 513), (4, 1000), (2050, 520), (2049, 1032), (300, 2793),
         (9, 4096), (3, 4104), (2, 8192), (5, 8193), (3, 16384), (70, 16390), (2, 20000), (1, 65536), (1024, 530), (1025, 529), (2048, 96),
         (2049, 99),
         (640, 8200), (641, 8200), (645, 8203), (1030, 4103)]


@pytest.mark.parametrize("T,H", NORMS)
@pytest.mark.parametrize("res", [None, BF, F32])
def test_layer_norm(moe, T, H, res):
    g = gen(T * 131 + H)
    x = rnd(g, T, H)
    r = None if res is None else (rnd(g, T, H, scale=3, dtype=F32) + 2 * rnd(g, T, 1, dtype=F32)).to(res)
    w = rnd(g, H, dtype=F32 if res == F32 else BF)
    b = None if H % 2 else rnd(g, H, dtype=w.dtype)
    y, ro, mean, rstd = moe.moe_layer_norm_forward(cuda(x), cuda(w), cuda(b), residual=cuda(r), eps=1e-5, save_stats=True)
    s, v, m, q = ref.layer_norm(dbl(x), dbl(r), dbl(w), dbl(b), 1e-5)
    near(y, v, ref.layer_norm_tol(s, m, q, dbl(w), v), "y")
    near(mean, m, F24 * s.abs().mean(1), "mean")
    near(rstd, q, 4 * F24 * q + 2 * F24 * q * q * s.square().mean(1).sqrt(), "rstd")
    if r is None:
        assert ro is None
    else:
        near(ro, s, F24 * s.abs(), "residual_out")
    only = moe.moe_layer_norm_forward(cuda(x), cuda(w), cuda(b), residual=cuda(r))
    assert torch.equal(only[0], y) and only[2] is None and only[3] is None


def test_layer_norm_in_place_strides_and_rows_behind(moe):
    g = gen(3)
    T, H = 5, 96
    big, res = rnd(g, 8, H + 40).cuda(), rnd(g, 8, H + 8, dtype=F32).cuda()
    keep, keep_r = big.clone(), res.clone()
    w, b = rnd(g, H).cuda(), rnd(g, H).cuda()
    x, r = big[1:1 + T, 3:3 + H], res[2:2 + T, :H]  # rows that are not 16-byte aligned
    s, v, m, q = ref.layer_norm(dbl(x), dbl(r), dbl(w), dbl(b), 1e-6)
    stats = torch.full((2, 8), 7.0, device="cuda")
    y, ro, _, _ = moe.moe_layer_norm_forward(x, w, b, residual=r, eps=1e-6, y=x, residual_out=r, mean=stats[0, :T],
                                             rstd=stats[1, :T])
    assert y.data_ptr() == x.data_ptr() and ro.data_ptr() == r.data_ptr()
    near(y, v, ref.layer_norm_tol(s, m, q, dbl(w), v), "y")
    near(ro, s, F24 * s.abs(), "residual")
    assert bool((stats[:, T:] == 7).all())
    keep[1:1 + T, 3:3 + H] = big[1:1 + T, 3:3 + H]
    keep_r[2:2 + T, :H] = res[2:2 + T, :H]
    assert torch.equal(keep, big) and torch.equal(keep_r, res)


def test_layer_norm_far_means_and_special_values(moe):
    """Rows whose mean is large against their deviation, whose squares
    overflow fp32, constant rows, and rows with an infinity or a NaN."""
    g = gen(4)
    T, H = 8, 1000
    r = rnd(g, T, H, dtype=F32)
    r[0] += 3e4
    r[1] = r[1] * 1e30
    r[2] = 5.0
    r[3] *= 1e-20
    x = torch.zeros(T, H, dtype=BF)
    w, b = rnd(g, H, dtype=F32), rnd(g, H, dtype=F32)
    y, _, mean, rstd = moe.moe_layer_norm_forward(cuda(x), cuda(w), cuda(b), residual=cuda(r), eps=1e-5, save_stats=True)
    s, v, m, q = ref.layer_norm(dbl(x), dbl(r), dbl(w), dbl(b), 1e-5)
    # (nothing is rounded in the sum with zeros)
    near(y, v, 8 * F24 * (v.abs() + dbl(b).abs()), "y")
    near(mean, m, F24 * m.abs(), "mean")
    near(rstd, q, 8 * F24 * q, "rstd")
    r[4, 7], r[5, 9] = math.inf, math.nan
    y2 = moe.moe_layer_norm_forward(cuda(x), cuda(w), cuda(b), residual=cuda(r), eps=1e-5)[0]
    assert bool(y2[4].isnan().any()) and bool(y2[5].isnan().all())
    keep = [0, 1, 2, 3, 6, 7]
    assert torch.equal(y2[keep], y[keep])


def test_layer_norm_of_more_rows_than_a_launch(moe):
    T, H = (1 << 21) + 3, 8
    x = torch.ones(T, H, dtype=BF, device="cuda")
    x[:, ::2] = -1.0
    x[-4:] *= 2.0
    one = torch.ones(H, dtype=BF, device="cuda")
    y, _, mean, rstd = moe.moe_layer_norm_forward(x, one, eps=0.0, save_stats=True)
    assert bool((y.abs() == 1).all()) and not bool(mean.any()) and bool((rstd[-4:] == 0.5).all())
    dx, _, dw, db = moe.moe_layer_norm_backward(x, x, mean, rstd, one)
    assert not bool(dx.any())  # a gradient along the row itself
    # (an odd number of thousands: bf16 of 2^21 - 1 and 4 rows of 4 / 2)
    assert bool((dw.float() - (T - 4 + 8)).abs().max() <= T * B8) and bool((db.float().abs() - (T + 4)).abs().max() <= T * B8)


@pytest.mark.parametrize("T,H", NORMS)
@pytest.mark.parametrize("kind", [(BF, False), (BF, True), (F32, False), (F32, True)])
def test_layer_norm_backward(moe, T, H, kind):
    dt, has = kind
    g = gen(T * 7 + H)
    s = (rnd(g, T, H, scale=2, dtype=F32) + rnd(g, T, 1, dtype=F32)).to(dt)
    _, _, mean, rstd = ref.layer_norm(dbl(s), None, torch.ones(H, dtype=torch.float64), None, 1e-5)
    mean, rstd = mean.float(), rstd.float()
    dy, w = rnd(g, T, H), rnd(g, H, dtype=F32 if H % 3 == 0 else BF)
    dres = rnd(g, T, H, dtype=dt) if has else None
    args = [cuda(t) for t in (dy, s, mean, rstd, w)]
    got = moe.moe_layer_norm_backward(*args, dresidual_out=cuda(dres), need_dresidual=True)
    want, tols = ref.layer_norm_backward(dbl(dy), dbl(s), dbl(mean), dbl(rstd), dbl(w), dbl(dres))
    near(got[0], want[0], tols[0], "dx")
    near(got[1], want[0], tols[0], "dresidual")
    assert got[1].dtype == dt and (dt == F32 or torch.equal(got[0], got[1]))
    near(got[2], want[1], tols[1], "dweight")
    near(got[3], want[2], tols[2], "dbias")
    for k in range(4):
        need = dict(need_dx=k == 0, need_dresidual=k == 1, need_dweight=k == 2, need_dbias=k == 3)
        one = moe.moe_layer_norm_backward(*args, dresidual_out=cuda(dres), **need)
        assert [t is not None for t in one] == [i == k for i in range(4)] and torch.equal(one[k], got[k])


def test_layer_norm_backward_strides_and_rows_behind(moe):
    g = gen(8)
    for T, H in ((5, 96), (3, 301), (40, 2056)):
        dy, s, dr = rnd(g, T + 2, H + 9), rnd(g, T + 2, H + 8, dtype=F32), rnd(g, T + 2, H + 8, dtype=F32)
        st = torch.rand(2, T, generator=g) + 0.5
        w = rnd(g, H)
        dx, dres = torch.full((T + 3, H + 3), 7, dtype=BF).cuda(), torch.full((T + 3, H + 4), 7, dtype=F32).cuda()
        v = (dy[1:1 + T, 3:3 + H], s[:T, :H], st[0], st[1], w)
        out = moe.moe_layer_norm_backward(cuda(dy)[1:1 + T, 3:3 + H], cuda(s)[:T, :H], *(cuda(t) for t in v[2:]),
                                          dresidual_out=cuda(dr)[2:, 8:], need_dresidual=True, dx=dx[1:1 + T, 1:1 + H],
                                          dresidual=dres[:T, :H])
        want, tols = ref.layer_norm_backward(*(dbl(t) for t in v), dbl(dr[2:, 8:]))
        near(out[0], want[0], tols[0], "dx")
        near(out[1], want[0], tols[0], "dresidual")
        near(out[2], want[1], tols[1], "dweight")
        dx[1:1 + T, 1:1 + H] = 7
        dres[:T, :H] = 7
        assert bool((dx == 7).all()) and bool((dres == 7).all())


def test_layer_norm_backward_of_no_rows(moe):
    H = 72
    e, v = torch.empty(0, H, dtype=BF, device="cuda"), torch.empty(0, dtype=F32, device="cuda")
    w = torch.ones(H, dtype=BF, device="cuda")
    dw, db = torch.full_like(w, math.nan), torch.full_like(w, math.nan)
    dx, _, _, _ = moe.moe_layer_norm_backward(e, e, v, v, w, dweight=dw, dbias=db)
    assert dx.shape == (0, H) and not bool(dw.any()) and not bool(db.any())
    x = torch.empty(0, H, dtype=BF, device="cuda", requires_grad=True)
    w.requires_grad_()
    y, s = moe.moe_layer_norm(x, w)
    y.sum().backward()
    assert x.grad.shape == (0, H) and not bool(w.grad.any()) and s is None


@pytest.mark.parametrize("res", [None, BF, F32])
def test_layer_norm_gradients(moe, res):
    """The differentiable form against the formula and against differences of
    the fp64 forward."""
    g = gen(11)
    T, H = 37, 264
    x, w, b = rnd(g, T, H), rnd(g, H), rnd(g, H)
    r = None if res is None else rnd(g, T, H, scale=2, dtype=res)
    leaves = [cuda(t).requires_grad_() for t in (x, w, b)] + ([] if r is None else [cuda(r).requires_grad_()])
    y, s = moe.moe_layer_norm(*leaves, eps=1e-5)
    py, ps = rnd(g, T, H), None if r is None else rnd(g, T, H, dtype=res)
    if r is None:
        assert s is None
        y.backward(cuda(py))
    else:
        torch.autograd.backward([y, s], [cuda(py), cuda(ps)])
    stream = dbl(x) if r is None else dbl(s.detach())
    s64, _, mean, rstd = ref.layer_norm(dbl(x), dbl(r), dbl(w), dbl(b), 1e-5)
    want, tols = ref.layer_norm_backward(dbl(py), stream, mean, rstd, dbl(w), dbl(ps))
    # (mean and rstd are fp32: two more roundings of n)
    slack = 4 * F24 * (1 + s64.abs().max() * rstd.max()) * dbl(py).abs().max() * dbl(w).abs().max() * rstd.max() * 4
    near(leaves[0].grad, want[0], tols[0] + slack, "dx")
    near(leaves[1].grad, want[1], tols[1] + T * slack, "dweight")
    near(leaves[2].grad, want[2], tols[2], "dbias")
    if r is not None:
        assert leaves[3].grad.dtype == res
        near(leaves[3].grad, want[0], tols[0] + slack, "dresidual")

    def loss(x, w, b, r=None):
        s, y, _, _ = ref.layer_norm(x, r, w, b, 1e-5)
        return float((y * dbl(py)).sum() + (0 if r is None else (s * dbl(ps)).sum()))

    d = [dbl(t.detach()) for t in leaves]
    for k, leaf in enumerate(leaves):
        step = rnd(g, *leaf.shape, dtype=torch.float64)
        e = 1e-5
        hi, lo = (loss(*(u + c * e * step if i == k else u for i, u in enumerate(d))) for c in (1, -1))
        # the gradient's rounding (and a bf16 stream's, 2^-8 |s| r of n), summed at random
        tol = 6 * B8 * float((leaf.grad.double().cpu() * step).norm()) + (
            6 * B8 * float((want[0].abs() + rstd.unsqueeze(1) * 4).mul(step if step.dim() == 2 else 1).norm()) if res == BF else 0)
        assert abs((hi - lo) / (2 * e) - float((dbl(leaf.grad) * step).sum())) <= tol + 1e-5 * abs(hi), k


def test_layer_norm_partial_gradients(moe):
    """Outputs that are not used, expanded gradients, frozen inputs."""
    g = gen(12)
    T, H = 6, 64
    x, r = cuda(rnd(g, T, H)).requires_grad_(), cuda(rnd(g, T, H, dtype=F32)).requires_grad_()
    w = cuda(rnd(g, H))
    y, s = moe.moe_layer_norm(x, w, residual=r)
    s.sum().backward(retain_graph=True)  # the stream alone
    assert bool((r.grad == 1).all()) and bool((x.grad == 1).all())
    x.grad = r.grad = None
    y.sum().backward()  # the norm alone, with an expanded gradient
    _, _, mean, rstd = moe.moe_layer_norm_forward(x.detach(), w, residual=r.detach(), save_stats=True)
    one = torch.ones(T, H, dtype=BF, device="cuda")
    dx, dr, _, _ = moe.moe_layer_norm_backward(one, s.detach(), mean, rstd, w, need_dresidual=True)
    assert torch.equal(x.grad, dx) and torch.equal(r.grad, dr)
    y, s = moe.moe_layer_norm(x.detach(), w, residual=r.detach())
    assert not y.requires_grad


# ------------------------------------------------------------------ permute
def routing(g, T, k, E, how):
    if how == "one":
        return torch.full((T, k), E - 1, dtype=torch.int32)
    if how == "none":
        return torch.full((T, k), -1, dtype=torch.int32)
    ids = torch.randint(0, E, (T, k), generator=g, dtype=torch.int32)  # (an expert may come twice)
    if how == "absent":
        bad = torch.tensor([-1, E, -(1 << 31), (1 << 31) - 1], dtype=torch.int32)
        pick = torch.rand(T, k, generator=g) < 0.4
        ids = torch.where(pick, bad[torch.randint(0, 4, (T, k), generator=g)], ids)
    return ids


def values(g, T, H, dt):
    return rnd(g, T, H, dtype=F32).to(dt)


# pairs below and above what one launch takes, whole slices of 1024 and one
# more, more slices than chunks
PAIRS = [(1, 1, 1), (1, 15, 112), (16, 15, 112), (3, 64, 1000), (128, 16, 64), (2048, 1, 5), (2049, 1, 1024), (1024, 3, 1),
         (1025, 2, 1023), (700, 8, 257), (5000, 4, 64), (1365, 3, 70),
         (4096, 1, 70), (4097, 1, 70), (1024, 8, 1024), (8193, 1, 1024)]


@pytest.mark.parametrize("T,k,E", PAIRS)
@pytest.mark.parametrize("how", ["all", "absent", "one", "none"])
def test_permute(moe, T, k, E, how):
    g = gen(T + k + E)
    ids = routing(g, T, k, E, how)
    x = values(g, T, 24, BF)
    out, rows, offsets = moe.moe_permute(cuda(x), cuda(ids), E)
    want = ref.permute(x, ids, E)
    assert torch.equal(offsets.cpu(), want[2]) and torch.equal(rows.cpu(), want[1])
    assert torch.equal(out.cpu(), want[0])


@pytest.mark.parametrize("H", [1, 3, 7, 8, 15, 64, 100, 2793, 3584, 4097])
@pytest.mark.parametrize("dt", [BF, F32, U8, torch.uint8])
@pytest.mark.parametrize("T,k", [(5, 3), (1100, 2), (1300, 2)])
def test_permute_widths_and_types(moe, H, dt, T, k):
    g = gen(H + T)
    E = 7
    ids = routing(g, T, k, E, "absent")
    x = torch.randint(0, 256, (T, H), generator=g, dtype=torch.uint8) if dt == torch.uint8 else values(g, T, H, dt)
    out, rows, offsets = moe.moe_permute(cuda(x), cuda(ids), E)
    bits = {2: torch.int16, 4: torch.int32, 1: torch.uint8}[x.element_size()]
    want = ref.permute(x.view(bits), ids, E)
    assert torch.equal(rows.cpu(), want[1]) and torch.equal(out.cpu().view(bits), want[0])


def test_permute_strides_and_rows_behind(moe):
    g = gen(1)
    for T, k, H in ((9, 4, 37), (900, 3, 40)):
        ids = routing(g, T, k, 6, "absent")
        x = values(g, T + 2, H + 5, BF)
        out = torch.full((T * k + 2, H + 6), 7, dtype=BF, device="cuda")
        rows, off = torch.full((T + 1, k), 9, dtype=torch.int32, device="cuda"), torch.full((9,), 9, dtype=torch.int32, device="cuda")
        moe.moe_permute(cuda(x)[1:1 + T, 3:3 + H], cuda(ids), 6, out=out[1:-1, 1:1 + H], rows=rows[:T], expert_offsets=off[:7])
        want = ref.permute(x[1:1 + T, 3:3 + H], ids, 6)
        assert torch.equal(out[1:-1, 1:1 + H].cpu(), want[0]) and torch.equal(rows[:T].cpu(), want[1])
        assert torch.equal(off[:7].cpu(), want[2]) and bool((rows[T:] == 9).all()) and bool((off[7:] == 9).all())
        out[1:-1, 1:1 + H] = 7
        assert bool((out == 7).all())


def test_permute_many_pairs(moe):
    """More slices than chunks (a chunk ranks several): against a stable sort."""
    T, k, E = 70001, 4, 300
    g = gen(2)
    ids = routing(g, T, k, E, "absent").cuda()
    x = torch.arange(T, device="cuda", dtype=torch.int32).view(F32).unsqueeze(1).contiguous()
    out, rows, offsets = moe.moe_permute(x, ids, E)
    key = ids.flatten().long()
    key = torch.where((key >= 0) & (key < E), key, torch.full_like(key, E))
    order = torch.sort(key, stable=True).indices
    n = int((key < E).sum())
    assert torch.equal(out.view(torch.int32).flatten()[:n].long(), order[:n] // k) and not bool(out.view(torch.int32)[n:].any())
    place = torch.where(rows < 0, -1 - rows, rows).flatten().long()
    assert torch.equal(order[place], torch.arange(T * k, device="cuda")) and torch.equal(rows.flatten() < 0, key == E)
    assert offsets.tolist() == [0] + torch.bincount(key, minlength=E + 1)[:E].cumsum(0).tolist()


def test_permute_above_4_gib(moe):
    """Offsets that pass 32 bits, in elements too."""
    T, k, H = 70000, 8, 8192  # out: 8.5 GiB of bf16, 4.6e9 elements
    x = torch.empty(T, H, dtype=BF, device="cuda")
    x[:] = (torch.arange(T, device="cuda") % 251).to(BF).unsqueeze(1)
    ids = ((torch.arange(T * k, device="cuda") * 7) % 40).to(torch.int32).view(T, k)
    out, rows, offsets = moe.moe_permute(x, ids, 40)
    token = torch.empty(T * k, dtype=torch.long, device="cuda")
    token[rows.flatten().long()] = torch.arange(T * k, device="cuda") // k
    for c in (0, 4095, H - 1):
        assert torch.equal(out[:, c], (token % 251).to(BF))
    del x
    back = moe.moe_unpermute(out, rows)
    for c in (0, H - 1):
        assert torch.equal(back[:, c], ((torch.arange(T, device="cuda") % 251) * k).float().to(BF))
    del out
    dy, _ = moe.moe_unpermute_backward(back, rows)
    for c in (0, H - 1):
        assert torch.equal(dy[:, c], back[token, c])


def test_layer_norm_above_4_gib(moe):
    T, H = 300_000, 8192  # 4.6 GiB of bf16, 9.2 of fp32
    x = torch.empty(T, H, dtype=BF, device="cuda").normal_()
    r = torch.empty(T, H, device="cuda").normal_()
    w, b = (torch.empty(H, device="cuda").normal_() for _ in range(2))
    y, s, mean, rstd = moe.moe_layer_norm_forward(x, w, b, residual=r, save_stats=True)
    rows = [0, 131071, 262143, 262144, 299_999]
    s64, v, m, q = ref.layer_norm(dbl(x[rows]), dbl(r[rows]), dbl(w), dbl(b), 1e-5)
    near(y[rows], v, ref.layer_norm_tol(s64, m, q, dbl(w), v), "y")
    near(s[rows], s64, F24 * s64.abs(), "s")
    del r
    dx, ds, dw, db = moe.moe_layer_norm_backward(x, s, mean, rstd, w, dresidual_out=s, need_dresidual=True)
    want, tols = ref.layer_norm_backward(dbl(x[rows]), dbl(s[rows]), dbl(mean[rows]), dbl(rstd[rows]), dbl(w), dbl(s[rows]))
    near(dx[rows], want[0], tols[0], "dx")
    near(ds[rows], want[0], tols[0], "dresidual")
    # (T / 256 rows a workgroup, 128 runs of those)
    for c in (0, H - 1):
        d = dbl(x[:, c])
        n = (dbl(s[:, c]) - dbl(mean)) * dbl(rstd)
        near(db[c:c + 1], d.sum().view(1), (T / 256 + 70) * F24 * d.abs().sum(), "dbias")
        near(dw[c:c + 1], (d * n).sum().view(1), (T / 256 + 80) * F24 * (d * n).abs().sum(), "dweight")


def test_linear_above_4_gib(moe):
    T, K, N = 300_000, 64, 8192  # out, pre and dout of 4.6 GiB
    g = gen(9)
    x = torch.empty(T, K, dtype=BF, device="cuda").normal_()
    w, b = cuda(rnd(g, N, K, scale=K ** -0.5)), cuda(rnd(g, N))
    out, pre = moe.moe_linear_forward(x, w, b, act=ref.GELU, save_pre=True)
    rows = [0, 131071, 262143, 262144, 299_999]
    check_linear(moe, ref.GELU, x[rows].cpu(), w.cpu(), b.cpu(), None, out[rows], pre[rows])
    dx, dw, db = moe.moe_linear_backward(out, x, w, pre=pre, act=ref.GELU)
    check_linear_bwd(ref.GELU, out[rows].cpu(), x[rows].cpu(), pre[rows].cpu(), w.cpu(), (dx[rows], None, None))
    for c in (0, N - 1):
        s64, t = ref.slope(ref.GELU, dbl(pre[:, c]))
        full = dbl(out[:, c]) * s64
        near(db[c:c + 1], full.sum().view(1), (T / 64 + 300) * F24 * full.abs().sum() + (dbl(out[:, c]).abs() * t).sum(), "dbias")
        dz = dense_ref.bf16(full)
        want = dz @ dbl(x)
        # (sums of T / 8 terms in a row at most, and dz on the other side of a tie)
        tol = (T / 8 + 64) * F24 * (dz.abs() @ dbl(x).abs()) + dense_ref.FLIPS * want.square().mean().sqrt()
        near(dw[c], want, tol, "dw")


def plan(g, T, k, E=9, how="absent"):
    return ref.permute(torch.zeros(T, 1), routing(g, T, k, E, how), E)[1]


COMBINE = [(1, 1, 1), (3, 2, 7), (1, 15, 3584), (37, 4, 1001), (300, 5, 264), (40, 9, 520), (5, 16, 4100), (4, 17, 96), (70, 2, 16),
           (33, 6, 257),
           (3, 64, 72), (2, 3, 20000)]


@pytest.mark.parametrize("T,k,H", COMBINE)
@pytest.mark.parametrize("types", [(BF, BF), (BF, F32), (F32, F32), (F32, BF)])
@pytest.mark.parametrize("full", [True, False])
def test_unpermute(moe, T, k, H, types, full):
    g = gen(T + k + H)
    rows = plan(g, T, k)
    y = rnd(g, T * k, H, dtype=types[0])
    y[torch.where(rows < 0, -1 - rows, 0).flatten().long()[rows.flatten() < 0]] = math.nan  # rows of no expert
    w = torch.randn(T, k, generator=g) if full else None
    if full:
        w[rows < 0] = math.inf
    r = rnd(g, T, H, dtype=types[1]) if full else None
    out = moe.moe_unpermute(cuda(y), cuda(rows), cuda(w), cuda(r), out_dtype=types[1])
    want, size = ref.unpermute(dbl(y), rows, dbl(w), dbl(r))
    assert out.dtype == types[1]
    near(out, want, (k + 2) * F24 * size, "out")


@pytest.mark.parametrize("T,k,H", COMBINE)
@pytest.mark.parametrize("types", [(BF, BF), (BF, F32), (F32, F32), (F32, BF)])
def test_unpermute_backward(moe, T, k, H, types):
    g = gen(T + k + H + 1)
    rows = plan(g, T, k)
    y, dout, w = rnd(g, T * k, H, dtype=types[0]), rnd(g, T, H, dtype=types[1]), torch.randn(T, k, generator=g)
    y[torch.where(rows < 0, -1 - rows, 0).flatten().long()[rows.flatten() < 0]] = math.nan
    w[rows < 0] = math.nan
    args = cuda(dout), cuda(rows)
    dy, dw = moe.moe_unpermute_backward(*args, y=cuda(y), weights=cuda(w))
    want, dots, size = ref.unpermute_backward(dbl(dout), rows, dbl(y), dbl(w))
    near(dy, want, F24 * want.abs(), "dy")
    near(dw, dots, (H / 64 + 40) * F24 * size, "dweights")
    assert not bool(dw.cpu()[rows < 0].any())
    one, none = moe.moe_unpermute_backward(*args, y=cuda(y), weights=cuda(w), need_dweights=False)
    assert torch.equal(one, dy) and none is None
    none, one = moe.moe_unpermute_backward(*args, y=cuda(y), weights=cuda(w), need_dy=False)
    assert torch.equal(one, dw) and none is None
    plain, none = moe.moe_unpermute_backward(*args, y_dtype=types[0])
    want, _, _ = ref.unpermute_backward(dbl(dout), rows, None, None)
    assert none is None and torch.equal(dbl(plain), want.to(types[0]).double())


def test_unpermute_strides_in_place_and_rows_behind(moe):
    g = gen(5)
    for T, k, H in ((7, 3, 37), (9, 9, 2048)):
        rows = plan(g, T, k)
        y, w = rnd(g, T * k + 3, H + 9), torch.randn(T, k, generator=g)
        out = rnd(g, T + 2, H + 5, dtype=F32).cuda()
        keep = out.clone()
        res = out[1:1 + T, 2:2 + H]
        want, size = ref.unpermute(dbl(y[2:-1, 4:4 + H]), rows, dbl(w), dbl(res))
        got = moe.moe_unpermute(cuda(y)[2:-1, 4:4 + H], cuda(rows), cuda(w), res, out=res)
        near(got, want, (k + 2) * F24 * size, "out")
        keep[1:1 + T, 2:2 + H] = out[1:1 + T, 2:2 + H]
        assert torch.equal(keep, out)
        dy = torch.full((T * k + 2, H + 3), 7, dtype=BF, device="cuda")
        dw = torch.full((T + 1, k), 7.0, device="cuda")
        moe.moe_unpermute_backward(out[1:1 + T, 2:2 + H], cuda(rows), y=cuda(y)[2:-1, 4:4 + H], weights=cuda(w),
                                   dy=dy[1:-1, 1:1 + H], dweights=dw[:T])
        want, dots, size = ref.unpermute_backward(dbl(out[1:1 + T, 2:2 + H]), rows, dbl(y[2:-1, 4:4 + H]), dbl(w))
        near(dy[1:-1, 1:1 + H], want, F24 * want.abs(), "dy")
        near(dw[:T], dots, (H / 64 + 40) * F24 * size, "dweights")
        dy[1:-1, 1:1 + H] = 7
        assert bool((dy == 7).all()) and bool((dw[T:] == 7).all())


def test_unpermute_rows_outside_are_skipped(moe):
    T, k, H = 3, 2, 40
    y = torch.ones(T * k, H, dtype=BF, device="cuda")
    rows = torch.tensor([[0, 6], [1 << 30, 5], [-1 - (1 << 30), -(1 << 31)]], dtype=torch.int32, device="cuda")
    assert torch.equal(moe.moe_unpermute(y, rows), y[:3] * torch.tensor([[1], [1], [0]], dtype=BF, device="cuda"))
    dy = torch.full((T * k, H), 7, dtype=BF, device="cuda")
    _, dw = moe.moe_unpermute_backward(y[:3], rows, y=y, dy=dy)
    assert bool((dy[[0, 5]] == 1).all()) and bool((dy[1:5] == 7).all())
    assert torch.equal(dw, torch.tensor([[H, 0], [0, H], [0, 0]], dtype=F32, device="cuda"))


def test_rows_of_no_tokens(moe):
    e = torch.empty(0, 40, dtype=BF, device="cuda", requires_grad=True)
    ids = torch.empty(0, 4, dtype=torch.int32, device="cuda")
    off = torch.full((1025,), 9, dtype=torch.int32, device="cuda")
    moe.moe_permute(e, ids, 1024, expert_offsets=off)
    assert not bool(off.any())
    out, rows, offsets = moe.moe_dispatch(e, ids, 6)
    assert out.shape == (0, 40) and rows.shape == (0, 4) and not bool(offsets.any())
    back = moe.moe_combine(out, rows, torch.empty(0, 4, device="cuda"))
    back.sum().backward()
    assert back.shape == (0, 40) and e.grad.shape == (0, 40)


@pytest.mark.parametrize("dt,st", [(BF, BF), (BF, F32), (F32, F32)])
def test_dispatch_and_combine_gradients(moe, dt, st):
    """Against the formula, and (they are linear in each input) against the
    forward itself."""
    g = gen(21)
    T, k, E, H = 23, 3, 5, 72
    ids = routing(g, T, k, E, "absent")
    x, w, r, scale = rnd(g, T, H, dtype=dt), torch.rand(T, k, generator=g), rnd(g, T, H, dtype=st), rnd(g, T * k, H, dtype=dt)
    lx, lw, lr = (cuda(t).requires_grad_() for t in (x, w, r))
    xs, rows, offsets = moe.moe_dispatch(lx, cuda(ids), E)
    y = xs * cuda(scale)  # what the experts do with their rows
    out = moe.moe_combine(y, rows, lw, lr)
    probe = rnd(g, T, H, dtype=st)
    out.backward(cuda(probe))
    rows = rows.cpu()
    dy, dots, size = ref.unpermute_backward(dbl(probe), rows, dbl(y.detach()), dbl(w))
    near(lw.grad, dots, (H / 64 + 40) * F24 * size, "dweights")
    assert torch.equal(lr.grad.cpu(), probe)
    # dy and its product with the experts' factors are rounded on the way
    want, size = ref.unpermute(dy * dbl(scale), rows, None, None)
    near(lx.grad, want, 2.1 * HALF[dt] * size + (k + 2) * F24 * size, "dx")

    def loss(x, w, r):
        y = ref.permute(x, ids, E)[0] * dbl(scale)
        return float((ref.unpermute(y, rows, w, r)[0] * dbl(probe)).sum())
    d = [dbl(t) for t in (x, w, r)]
    for i, leaf in enumerate((lx, lw, lr)):
        step = rnd(g, *leaf.shape, dtype=torch.float64)
        hi, lo = (loss(*(u + c * step if j == i else u for j, u in enumerate(d))) for c in (1, -1))
        tol = 8 * B8 * float((dbl(leaf.grad) * step).norm()) + 4 * B8 * float(size.norm())
        assert abs((hi - lo) / 2 - float((dbl(leaf.grad) * step).sum())) <= tol, i


# ------------------------------------------------------------------ linear
def sum_tol(x, w):
    """Bound of the fp32 sums of x @ w.T, per element."""
    return (x.shape[1] / 8 + 64) * F24 * (x.abs() @ w.abs().t())


ACTS = range(5)
LINEAR = [(1, 64, 8), (1, 3584, 512), (3, 72, 104), (16, 264, 2056), (17, 1000, 40), (33, 520, 2064), (64, 136, 264),
          (65, 1032, 392), (200, 4096, 136), (777, 1000, 520), (130, 64, 16),
          (70, 8200, 200), (600, 520, 2056), (32, 512, 5000)]


def linear_case(g, T, K, N, bias=BF, add=BF):
    x, w = rnd(g, T, K), rnd(g, N, K, scale=1.2 / math.sqrt(K))
    b = None if bias is None else rnd(g, N, dtype=bias)
    return x, w, b, None if add is None else rnd(g, T, N, dtype=add)


def check_linear(moe, a, x, w, b, add, out, pre):
    z = dbl(x) @ dbl(w).t()
    tol = sum_tol(dbl(x), dbl(w))
    if b is not None:
        z = z + dbl(b)
        tol = tol + 2 * F24 * (z.abs() + dbl(b).abs())
    if pre is not None:
        near(pre, z, tol, "pre")
    v, t = ref.act(a, z)
    t = t + ref.slope_of_act(a, z) * tol
    if add is not None:
        v = v + dbl(add)
        t = t + 2 * F24 * (v.abs() + dbl(add).abs())
    near(out, v, t, "out")


@pytest.mark.parametrize("T,K,N", LINEAR)
@pytest.mark.parametrize("a", ACTS)
def test_linear(moe, T, K, N, a):
    g = gen(T + K + N + a)
    f32 = (T + a) % 2 == 0
    x, w, b, add = linear_case(g, T, K, N, F32 if a % 2 else BF, F32 if f32 else BF)
    out, pre = moe.moe_linear_forward(cuda(x), cuda(w), cuda(b), act=a, addend=cuda(add), out_dtype=F32 if f32 else BF,
                                      save_pre=True)
    assert out.dtype == (F32 if f32 else BF)
    check_linear(moe, a, x, w, b, add, out, pre)
    # without an addend or a saved argument; the same twice
    one = moe.moe_linear_forward(cuda(x), cuda(w), cuda(b), act=a)
    check_linear(moe, a, x, w, b, None, one, None)
    assert torch.equal(one, moe.moe_linear_forward(cuda(x), cuda(w), cuda(b), act=a))


@pytest.mark.parametrize("T,K,N", [(5, 72, 40), (40, 2048, 2048), (300, 136, 264)])
def test_linear_parts_absent(moe, T, K, N):
    g = gen(T)
    for bias in (None, BF, F32):
        for add in (None, BF, F32):
            x, w, b, d = linear_case(g, T, K, N, bias, add)
            out = moe.moe_linear_forward(cuda(x), cuda(w), cuda(b), addend=cuda(d), out_dtype=add or F32)
            check_linear(moe, ref.NONE, x, w, b, d, out, None)
    check_linear(moe, ref.NONE, x, w, None, None, moe.moe_linear_forward(cuda(x), cuda(w)), None)


@pytest.mark.parametrize("T,K,N", [(2048, 520, 5128), (4100, 136, 2600)])
def test_linear_large_tiles(moe, T, K, N):
    g = gen(T)
    for a, add in ((ref.GELU, F32), (ref.SILU, BF)):
        x, w, b, d = linear_case(g, T, K, N, BF, add)
        out, pre = moe.moe_linear_forward(cuda(x), cuda(w), cuda(b), act=a, addend=cuda(d), out_dtype=add, save_pre=True)
        check_linear(moe, a, x, w, b, d, out, pre)


@pytest.mark.parametrize("T", [9, 48, 300])
def test_linear_strides_in_place_and_rows_behind(moe, T):
    g = gen(T)
    K, N = 264, 136
    x, w, b, add = linear_case(g, T + 3, K + 16, N + 24)
    w, b = w[:N, :K].contiguous(), b[:N].contiguous()
    buf = cuda(add)
    keep = buf.clone()
    at = buf[1:1 + T, 8:8 + N]
    pre = torch.full((T + 1, N), 7, dtype=BF, device="cuda")
    d = at.cpu().clone()
    out, _ = moe.moe_linear_forward(cuda(x)[2:2 + T, 8:8 + K], cuda(w), cuda(b), act=ref.GELU, addend=at, out=at, pre=pre[:T])
    check_linear(moe, ref.GELU, x[2:2 + T, 8:8 + K], w, b, d, out, pre[:T])
    keep[1:1 + T, 8:8 + N] = buf[1:1 + T, 8:8 + N]
    assert torch.equal(keep, buf) and bool((pre[T:] == 7).all())


@pytest.mark.parametrize("a", ACTS)
def test_linear_special_values(moe, a):
    """Far arguments, infinities and NaN of one token stay its own; the limits
    are met."""
    for T in (4, 40, 200):
        K, N = 64, 16
        x = torch.zeros(T, K, dtype=BF)
        x[:, 0] = 1
        z = torch.tensor([0.0, 1e-30, -1e-30, 5, -5, 30, -30, 1e4, -1e4, 1e30, -1e30, 3e38, -3e38, math.inf, -math.inf, math.nan])
        w = torch.zeros(N, K, dtype=BF)
        b = z.clone()
        out = moe.moe_linear_forward(cuda(x), cuda(w), cuda(b), act=a, out_dtype=F32).cpu()
        want = {ref.NONE: z, ref.RELU: z.clamp_min(0)}.get(a)
        if want is None:
            fine = ref.act(a, z[:13].double().clamp(-1e5, 1e5))[0].float()
            fine[9:13] = torch.tensor([z[9], 0.0, z[11], 0.0])
            want = torch.cat([fine, torch.tensor([math.inf, 0.0, math.nan])])
        assert torch.allclose(out, want.expand(T, N), rtol=1e-5, atol=1e-30, equal_nan=True), (a, out[0], want)
        x[2] = math.nan
        x[3, 5] = math.inf
        w[:, 5] = 1
        out2 = moe.moe_linear_forward(cuda(x), cuda(w), cuda(b), act=a, out_dtype=F32).cpu()
        assert bool(out2[2].isnan().all())
        assert torch.allclose(out2[[0, 1, *range(4, T)]], want.expand(T - 2, N), rtol=1e-5, atol=1e-30, equal_nan=True)


def check_linear_bwd(a, dout, x, pre, w, got):
    s, ts = ref.slope(a, dbl(pre)) if pre is not None else (1.0, 0.0)
    full = dbl(dout) * s
    exact = a == ref.NONE and dout.dtype == BF
    dz = full if exact else dense_ref.bf16(full)
    T = len(dout)
    # (the slope's error can move dz over a tie: FLIPS and one step, as in dense_ref)
    for name, v, r, st in (("dx", got[0], dz @ dbl(w), dense_ref.step_tol(dz, dbl(w).t())),
                           ("dw", got[1], dz.t() @ dbl(x), dense_ref.step_tol(dz.t(), dbl(x).t()))):
        if v is not None:
            dense_ref.check(v, r, B8, rms=2e-5 if exact else dense_ref.FLIPS, absolute=0.0 if exact else st, what=name,
                            norm=dense_ref.NORM)
    if got[2] is not None:
        near(got[2], full.sum(0), (T + 70) * F24 * full.abs().sum(0) + (dbl(dout).abs() * ts).sum(0), "dbias")


BACKWARD = [(1, 64, 8), (2, 1024, 4096), (3, 72, 104), (40, 264, 520), (150, 136, 2064), (777, 1000, 520), (512, 2048, 264),
            (2100, 392, 136)]


@pytest.mark.parametrize("T,K,N", BACKWARD)
@pytest.mark.parametrize("a", ACTS)
def test_linear_backward(moe, T, K, N, a):
    g = gen(T + K + N + a)
    dt = F32 if (T + a) % 3 == 0 else BF
    dout, x, pre = rnd(g, T, N, dtype=dt), rnd(g, T, K), rnd(g, T, N, scale=1.5)
    w = rnd(g, N, K, scale=1 / math.sqrt(K))
    args = [cuda(t) for t in (dout, x, w)]
    opts = dict(pre=cuda(pre), act=a, bias_dtype=F32 if a % 2 else BF)
    got = moe.moe_linear_backward(*args, **opts)
    check_linear_bwd(a, dout, x, pre, w, got)
    assert all(torch.equal(p, q) for p, q in zip(got, moe.moe_linear_backward(*args, **opts)))
    for k in range(3):
        one = moe.moe_linear_backward(*args, need_dx=k == 0, need_dw=k == 1, need_dbias=k == 2, **opts)
        assert [t is not None for t in one] == [i == k for i in range(3)] and torch.equal(one[k], got[k])


@pytest.mark.parametrize("T,K,N", [(2048, 1800, 3600), (4096, 1408, 2048)])
def test_linear_backward_large_tiles(moe, T, K, N):
    g = gen(T)
    dout, x, pre, w = rnd(g, T, N), rnd(g, T, K), rnd(g, T, N), rnd(g, N, K, scale=1 / math.sqrt(K))
    got = moe.moe_linear_backward(*(cuda(t) for t in (dout, x, w)), pre=cuda(pre), act=ref.GELU)
    check_linear_bwd(ref.GELU, dout, x, pre, w, got)


# (sums of few tokens beside weights of many tiles: in one launch, dx in parts
# and whole)
@pytest.mark.parametrize("T,K,N", [(1, 4096, 520), (5, 1032, 4104), (33, 8192, 264), (100, 1032, 2056), (128, 2056, 1288),
                                   (129, 2056, 1288), (300, 1024, 4104), (512, 1024, 4104), (117, 216, 1376), (346, 120, 2184),
                                   (64, 8, 8192)])
@pytest.mark.parametrize("a,dt", [(ref.GELU, BF), (ref.NONE, BF), (ref.SILU, F32)])
def test_linear_backward_of_few_tokens(moe, T, K, N, a, dt):
    g = gen(T + K)
    dout, x, pre, w = rnd(g, T, N + 8, dtype=dt), rnd(g, T, K), rnd(g, T, N), rnd(g, N, K, scale=1 / math.sqrt(K))
    args = [cuda(dout)[:, 8:], cuda(x), cuda(w)]
    got = moe.moe_linear_backward(*args, pre=cuda(pre), act=a)
    check_linear_bwd(a, dout[:, 8:], x, pre, w, got)
    for k in range(3):
        one = moe.moe_linear_backward(*args, pre=cuda(pre), act=a, need_dx=k == 0, need_dw=k == 1, need_dbias=k == 2)
        assert [t is not None for t in one] == [i == k for i in range(3)] and torch.equal(one[k], got[k])


# (the sum over the tokens in parts)
@pytest.mark.parametrize("T,K,N", [(3000, 264, 136), (3001, 64, 8), (4100, 520, 264), (3333, 768, 768)])
@pytest.mark.parametrize("a,dt", [(ref.GELU, BF), (ref.NONE, BF), (ref.RELU, F32)])
def test_linear_backward_of_many_tokens(moe, T, K, N, a, dt):
    g = gen(T + K)
    dout, x, pre = rnd(g, T, N, dtype=dt), rnd(g, T, K + 8), rnd(g, T, N)
    w = rnd(g, N, K, scale=1 / math.sqrt(K))
    args = [cuda(dout), cuda(x)[:, :K], cuda(w)]
    got = moe.moe_linear_backward(*args, pre=cuda(pre), act=a)
    check_linear_bwd(a, dout, x[:, :K], pre, w, got)
    for k in range(3):
        one = moe.moe_linear_backward(*args, pre=cuda(pre), act=a, need_dx=k == 0, need_dw=k == 1, need_dbias=k == 2)
        assert [t is not None for t in one] == [i == k for i in range(3)] and torch.equal(one[k], got[k])


@pytest.mark.parametrize("a", [ref.NONE, ref.GELU])
def test_linear_backward_strides_and_rows_behind(moe, a):
    g = gen(3)
    T, K, N = 70, 136, 72
    dout, x, pre = rnd(g, T + 2, N + 16), rnd(g, T + 1, K + 8), rnd(g, T, N)
    w = rnd(g, N, K, scale=1 / math.sqrt(K))
    dx = torch.full((T + 2, K + 8), 7, dtype=BF, device="cuda")
    got = moe.moe_linear_backward(cuda(dout)[1:1 + T, 8:8 + N], cuda(x)[1:, :K], cuda(w), pre=cuda(pre), act=a,
                                  dx=dx[1:1 + T, :K])
    check_linear_bwd(a, dout[1:1 + T, 8:8 + N], x[1:, :K], pre, w, got)
    dx[1:1 + T, :K] = 7
    assert bool((dx == 7).all())


def test_linear_backward_special_slopes(moe):
    """Limits far out, NaN where the argument is one."""
    z = torch.tensor([3e38, -3e38, math.inf, -math.inf, 1e4, -1e4, 300, -300], dtype=BF)
    x, w = torch.ones(1, 8, dtype=BF, device="cuda"), torch.ones(8, 8, dtype=BF, device="cuda")
    one = torch.ones(1, 8, dtype=BF, device="cuda")
    for a in (ref.RELU, ref.SILU, ref.GELU, ref.GELU_TANH):
        db = moe.moe_linear_backward(one, x, w, pre=cuda(z.unsqueeze(0)), act=a)[2].cpu()
        assert torch.equal(db, torch.tensor([1, 0] * 4, dtype=BF)), (a, db)
        nan = torch.full((1, 8), math.nan, dtype=BF, device="cuda")
        assert bool(moe.moe_linear_backward(one, x, w, pre=nan, act=a)[2].isnan().all())


@pytest.mark.parametrize("K,N", [(64, 96), (3584, 2048)])
def test_linear_of_no_tokens(moe, K, N):
    e, d = torch.empty(0, K, dtype=BF, device="cuda"), torch.empty(0, N, dtype=BF, device="cuda")
    w = torch.ones(N, K, dtype=BF, device="cuda")
    dw, db = torch.full_like(w, math.nan), torch.full((N,), math.nan, device="cuda")
    assert moe.moe_linear_forward(e, w, act=ref.GELU).shape == (0, N)
    dx, _, _ = moe.moe_linear_backward(d, e, w, pre=d, act=ref.GELU, dw=dw, dbias=db)
    assert dx.shape == (0, K) and not bool(dw.any()) and not bool(db.any())
    x = e.clone().requires_grad_()
    w.requires_grad_()
    moe.moe_linear(x, w, act=ref.SILU).sum().backward()
    assert x.grad.shape == (0, K) and not bool(w.grad.any())


@pytest.mark.parametrize("a", ACTS)
@pytest.mark.parametrize("T,out_dtype", [(4, BF), (150, F32)])
def test_linear_gradients(moe, a, T, out_dtype):
    """The differentiable form against the formula and against differences of
    the fp64 forward."""
    g = gen(T + a)
    K, N = 136, 200
    x, w, b, add = linear_case(g, T, K, N, F32, out_dtype)
    leaves = [cuda(t).requires_grad_() for t in (x, w, b, add)]
    out = moe.moe_linear(*leaves[:3], act=a, addend=leaves[3], out_dtype=out_dtype)
    probe = rnd(g, T, N, dtype=out_dtype)
    out.backward(cuda(probe))
    pre = moe.moe_linear_forward(*(t.detach() for t in leaves[:3]), save_pre=True)[1]
    check_linear_bwd(a, probe, x, pre.cpu(), w, [t.grad for t in leaves[:3]])
    assert torch.equal(leaves[3].grad.cpu(), probe)

    def loss(x, w, b, add):
        return float(((ref.act(a, x @ w.t() + b)[0] + add) * dbl(probe)).sum())
    d = [dbl(t) for t in (x, w, b, add)]
    z = d[0] @ d[1].t() + d[2]
    for k, leaf in enumerate(leaves):
        step = rnd(g, *leaf.shape, dtype=torch.float64)
        e = 1e-6
        hi, lo = (loss(*(u + c * e * step if i == k else u for i, u in enumerate(d))) for c in (1, -1))
        # what dz is off by: its rounding and z's (times the second slope, at most
        # 2; a relu's slope jumps where z rounds to 0, which no z here does),
        # summed at random through the step
        dzs = {0: step @ d[1].t() if k == 0 else None, 1: d[0] @ step.t() if k == 1 else None,
               2: step.expand(T, N) if k == 2 else None, 3: None}[k]
        tol = 6 * B8 * float((dbl(leaf.grad) * step).norm())
        if dzs is not None:
            tol += 6 * B8 * float((dzs * dbl(probe).abs() * (1.2 + 2 * z.abs())).norm())
        assert abs((hi - lo) / (2 * e) - float((dbl(leaf.grad) * step).sum())) <= tol + 1e-6 * abs(hi), k


def test_linear_partial_gradients(moe):
    g = gen(31)
    x, w, b, add = (cuda(t) for t in linear_case(g, 5, 64, 40))
    x.requires_grad_()
    moe.moe_linear(x, w, b, act=ref.GELU, addend=add).sum().backward()  # an expanded gradient
    pre = moe.moe_linear_forward(x.detach(), w, b, save_pre=True)[1]
    dx, _, _ = moe.moe_linear_backward(torch.ones(5, 40, dtype=BF, device="cuda"), x.detach(), w, pre=pre, act=ref.GELU)
    assert torch.equal(x.grad, dx)
    add.requires_grad_()
    moe.moe_linear(x.detach(), w, b, act=ref.GELU, addend=add).sum().backward()  # the addend alone
    assert bool((add.grad == 1).all())
    with pytest.raises(ValueError, match="pre"):
        moe.moe_linear_backward(add.detach(), x.detach(), w, act=ref.GELU)


# ---------------------------------------------- together
def block(moe, x, stream, p, ids, weights, E):
    """Layer norm, rows to their experts (two products each, by the host's
    offsets), back with the weights into the stream."""
    y, s = moe.moe_layer_norm(x, p["g"], p["b"], residual=stream)
    xs, rows, offsets = moe.moe_dispatch(y, ids, E)
    parts = []
    off = offsets.tolist()
    for e in range(E):
        h = moe.moe_linear(xs[off[e]:off[e + 1]], p["w1"][e], p["b1"][e], act=moe.MOE_LINEAR_GELU)
        parts.append(moe.moe_linear(h, p["w2"][e], p["b2"][e]))
    parts.append(xs[off[E]:])
    return moe.moe_combine(torch.cat(parts), rows, weights, s)


def test_block_of_experts(moe):
    """The operators together, forward and gradients, against fp64 autograd of
    the same block. Each value on the way (y, h, the experts' outputs and their
    gradients) is rounded to bf16, at most half a step of 2^-8: some ten such
    roundings in a row, summed at random, are 10 B8 of the 2-norm at most."""
    g = gen(41)
    T, H, I, E, k = 90, 128, 192, 4, 2
    ids = torch.rand(T, E + 1, generator=g).topk(k, 1).indices.to(torch.int32)  # (expert E: elsewhere)
    weights = torch.rand(T, k, generator=g)
    x, stream = rnd(g, T, H), rnd(g, T, H, dtype=F32)
    p = dict(g=1 + rnd(g, H, scale=0.1), b=rnd(g, H, scale=0.1), w1=rnd(g, E, I, H, scale=H ** -0.5), b1=rnd(g, E, I, scale=0.2),
             w2=rnd(g, E, H, I, scale=I ** -0.5), b2=rnd(g, E, H, scale=0.2))
    probe = rnd(g, T, H, dtype=F32)
    dev = {n: cuda(t).requires_grad_() for n, t in dict(p, x=x, stream=stream, weights=weights).items()}
    out = block(moe, dev["x"], dev["stream"], dev, cuda(ids), dev["weights"], E)
    out.backward(cuda(probe))
    d = {n: dbl(t).requires_grad_() for n, t in dict(p, x=x, stream=stream, weights=weights).items()}
    s, y, _, _ = ref.layer_norm(d["x"], d["stream"], d["g"], d["b"], 1e-5)
    want = s
    for e in range(E):
        h = y @ d["w1"][e].t() + d["b1"][e]
        v = (h * torch.special.ndtr(h)) @ d["w2"][e].t() + d["b2"][e]
        want = want + v * (d["weights"] * (ids == e)).sum(1, keepdim=True)
    want.backward(dbl(probe))
    far = lambda a, b: float((dbl(a.detach()) - b.detach()).norm() / b.detach().norm())  # noqa: E731
    assert far(out, want) <= 10 * B8
    for n in d:
        assert far(dev[n].grad, d[n].grad) <= 10 * B8, n
        assert dev[n].grad.dtype == dev[n].dtype


# ------------------------------------------- streams, graphs, two at once
def everything(moe, x, r, ids, wt, w, b, E, ws=None, stream=None):
    """Every call once, on one stream."""
    y, s, mean, rstd = moe.moe_layer_norm_forward(x, b["g"], b["b"], residual=r, save_stats=True, stream=stream)
    xs, rows, off = moe.moe_permute(y, ids, E, stream=stream)
    h, pre = moe.moe_linear_forward(xs, w, b["bias"], act=moe.MOE_LINEAR_GELU, addend=xs, save_pre=True, stream=stream)
    o = moe.moe_unpermute(h, rows, weights=wt, residual=s, stream=stream)
    dh, dwt = moe.moe_unpermute_backward(o, rows, y=h, weights=wt, stream=stream)
    dxs, dw, db = moe.moe_linear_backward(dh, xs, w, pre=pre, act=moe.MOE_LINEAR_GELU, stream=stream)
    dy = moe.moe_unpermute(dxs, rows, stream=stream)
    dx, dr, dg, dbn = moe.moe_layer_norm_backward(dy, s, mean, rstd, b["g"], dresidual_out=o, need_dresidual=True,
                                                  stream=stream)
    return y, s, mean, rstd, xs, rows, off, h, pre, o, dh, dwt, dxs, dw, db, dy, dx, dr, dg, dbn


def everything_inputs(g, T, k, H, E):
    ids = routing(g, T, k, E, "absent")
    return (cuda(rnd(g, T, H)), cuda(rnd(g, T, H, dtype=F32)), cuda(ids), cuda(torch.rand(T, k, generator=g)),
            cuda(rnd(g, H, H, scale=H ** -0.5)), {n: cuda(rnd(g, H)) for n in ("g", "b", "bias")}, E)


@pytest.mark.parametrize("T,k", [(5, 3), (700, 4)])
def test_in_a_graph(moe, T, k):
    """Two captured graphs, replayed in turn with eager work between."""
    g = gen(T)
    H, E = 136, 6
    ins = [everything_inputs(g, T, k, H, E) for _ in range(2)]
    everything(moe, *ins[0])
    torch.cuda.synchronize()
    graphs = []
    for i in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            graphs.append((gr, everything(moe, *ins[i])))
    for _ in range(3):
        for i in range(2):
            ins[i][0].copy_(cuda(rnd(g, T, H)))
            ins[i][2].copy_(cuda(routing(g, T, k, E, "absent")))
        for gr, _ in graphs:
            gr.replay()
        torch.cuda.synchronize()
        for i in range(2):
            want = everything(moe, *ins[i])
            assert all(torch.equal(a, b) for a, b in zip(graphs[i][1], want))


def test_gradients_in_a_graph(moe):
    g = gen(6)
    T, k, E, H = 130, 2, 4, 136
    x, stream, probe = cuda(rnd(g, T, H)).requires_grad_(), cuda(rnd(g, T, H, dtype=F32)).requires_grad_(), cuda(rnd(g, T, H, dtype=F32))
    ids, wt = cuda(routing(g, T, k, E, "all")), cuda(torch.rand(T, k, generator=g)).requires_grad_()
    w, b = cuda(rnd(g, H, H, scale=H ** -0.5)).requires_grad_(), [cuda(rnd(g, H)).requires_grad_() for _ in range(3)]
    leaves = (x, stream, wt, w, *b)

    def step():
        y, s = moe.moe_layer_norm(x, b[0], b[1], residual=stream)
        xs, rows, _ = moe.moe_dispatch(y, ids, E)
        out = moe.moe_combine(moe.moe_linear(xs, w, b[2], act=moe.MOE_LINEAR_SILU), rows, wt, s)
        return (out.detach(), *torch.autograd.grad(out, leaves, probe))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        o = step()
    for _ in range(3):
        with torch.no_grad():
            x.copy_(cuda(rnd(g, T, H)))
            probe.copy_(cuda(rnd(g, T, H, dtype=F32)))
            ids.copy_(cuda(routing(g, T, k, E, "all")))
        gr.replay()
        torch.cuda.synchronize()
        want = step()
        assert all(torch.equal(p, q) for p, q in zip(o, want))


def test_two_streams_at_once(moe):
    g = gen(5)
    ins = [everything_inputs(g, 900, 4, 264, 7) for _ in range(2)]
    want = [everything(moe, *i) for i in ins]
    torch.cuda.synchronize()
    st = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(6):
        for i in range(2):
            got[i].append(everything(moe, *ins[i], stream=st[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for o in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(o, want[i]))


# ---------------------------------------------- the block with 4-bit experts
@pytest.mark.parametrize("T", [1, 40])
@pytest.mark.parametrize("E", [8, 13])
def test_quantised_block_with_layer_norm_and_router_bias(moe, T, E):
    """moe_a16w4_block with norm_bias and router_bias is its parts in turn."""
    g = gen(T + E)
    H, I, k = 256, 128, 4
    x, r = cuda(rnd(g, T, H)), cuda(rnd(g, T, H, dtype=F32))
    nw, nb, rw, rb = cuda(rnd(g, H)), cuda(rnd(g, H)), cuda(rnd(g, E, H, scale=H ** -0.5)), cuda(rnd(g, E, dtype=F32))
    w13 = torch.randint(0, 256, (E, 2 * I, H // 2), generator=g, dtype=torch.uint8).cuda()
    w2 = torch.randint(0, 256, (E, H, I // 2), generator=g, dtype=torch.uint8).cuda()
    s13 = torch.randint(118, 122, (E, 2 * I, H // 32), generator=g, dtype=torch.uint8).cuda()
    s2 = torch.randint(118, 122, (E, H, I // 32), generator=g, dtype=torch.uint8).cuda()
    out, res = moe.moe_a16w4_block(x, nw, rw, w13, s13, w2, s2, k, residual=r, eps=1e-5, norm_bias=nb, router_bias=rb)
    y, s, _, _ = moe.moe_layer_norm_forward(x, nw, nb, residual=r, eps=1e-5)
    pad = torch.nn.functional.pad
    logits = moe.moe_linear_forward(y, pad(rw, (0, 0, 0, -E % 8)), bias=pad(rb, (0, -E % 8)), out_dtype=F32)[:, :E].contiguous()
    assert torch.equal(out, moe.moe_a16w4_layer(y, logits, w13, s13, w2, s2, k)) and torch.equal(res, s)
    want = dbl(y) @ dbl(rw).t() + dbl(rb)
    near(logits, want, sum_tol(dbl(y), dbl(rw)) + 2 * F24 * (want.abs() + dbl(rb).abs()), "logits")
    with pytest.raises(ValueError, match="layer norm"):
        moe.moe_a16w4_block(x, nw, rw, w13, s13, w2, s2, k, weight_offset=1.0, norm_bias=nb)
    with pytest.raises(ValueError, match="router_bias"):
        moe.moe_a16w4_block(x, nw, rw, w13, s13, w2, s2, k, router_bias=rb[1:])
