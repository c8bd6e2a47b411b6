"""More sizes, layouts and far values of the operators of a trainable expert block
(MI355X); forms and tolerances as in test_train_gpu.py."""
import pytest
import torch

from tests import test_train_gpu as base, train_ref as ref
from tests.test_train_gpu import BF, F24, F32, cuda, dbl, gen, moe, near, rnd  # noqa: F401

pytestmark = pytest.mark.gpu


# (rows of more than 8192 columns: the borders of the row workgroups and of one launch)
@pytest.mark.parametrize("T,H", [(64, 8200), (320, 10001), (321, 10001), (512, 12288), (513, 12288), (1000, 16384), (1024, 8201), (1025, 8200)])
@pytest.mark.parametrize("kind", [(BF, True), (F32, False)])
def test_layer_norm_backward_of_wide_rows(moe, T, H, kind):  # noqa: F811
    base.test_layer_norm_backward(moe, T, H, kind)


@pytest.mark.parametrize("T,H", [(6, 7), (40, 301), (1500, 96), (1100, 1032), (1030, 8201), (30, 16400)])
def test_layer_norm_backward_in_columns_of_its_inputs_buffer(moe, T, H):  # noqa: F811
    """dx beside dy in one buffer, and dresidual in dresidual_out's own rows; rows of
    dy or s are refused."""
    g = gen(T + H)
    both, s, dr = cuda(rnd(g, T, 2 * H)), cuda(rnd(g, T + 1, H, dtype=F32)), cuda(rnd(g, T, H, dtype=F32))
    w = cuda(rnd(g, H))
    _, _, mean, rstd = (cuda(t.float()) for t in ref.layer_norm(dbl(s[:T]), None, torch.ones(H).double(), None, 1e-5))
    dy, dx = both[:, :H], both[:, H:]
    keep = dr.clone()
    want = moe.moe_layer_norm_backward(dy.clone(), s[:T], mean, rstd, w, dresidual_out=keep, need_dresidual=True)
    got = moe.moe_layer_norm_backward(dy, s[:T], mean, rstd, w, dresidual_out=dr, need_dresidual=True, dx=dx, dresidual=dr)
    assert got[0].data_ptr() == dx.data_ptr() and got[1].data_ptr() == dr.data_ptr()
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    with pytest.raises(moe.MoeError, match="share rows"):
        moe.moe_layer_norm_backward(dy, s[:T], mean, rstd, w, need_dx=False, need_dresidual=True, dresidual=s[1:])
    with pytest.raises(moe.MoeError, match="share rows"):
        moe.moe_layer_norm_backward(dy, s[:T], mean, rstd, w, dx=both[:, H - 1:2 * H - 1])


# (sums of thousands of tokens beside sums as long over the columns)
@pytest.mark.parametrize("T,K,N", [(3000, 64, 4096), (3001, 8, 8192), (3500, 136, 4104), (5000, 64, 4096)])
@pytest.mark.parametrize("a,dt", [(ref.GELU, BF), (ref.NONE, F32)])
def test_linear_backward_of_two_long_sums(moe, T, K, N, a, dt):  # noqa: F811
    base.test_linear_backward_of_many_tokens(moe, T, K, N, a, dt)


@pytest.mark.parametrize("T,K,N", [(129, 2056, 2816), (300, 2056, 2816), (512, 1408, 4104), (256, 2048, 2048), (400, 1032, 4096)])
@pytest.mark.parametrize("a,dt", [(ref.GELU, BF), (ref.NONE, BF), (ref.SILU, F32)])
def test_linear_backward_of_few_tokens_of_large_weights(moe, T, K, N, a, dt):  # noqa: F811
    base.test_linear_backward_of_few_tokens(moe, T, K, N, a, dt)


def test_one_buffer_for_several_sizes(moe):  # noqa: F811
    """A workspace of the largest batch (of the sort), or of the largest query, for
    smaller ones."""
    E = 896
    ws = torch.empty(moe.moe_permute_workspace_size(262145, 1, E), dtype=torch.uint8, device="cuda")
    for T in (262145, 262144, 131073, 5000, 2561, 3):
        x, ids = torch.arange(T, device="cuda", dtype=torch.int32).view(F32).unsqueeze(1), torch.arange(T, device="cuda", dtype=torch.int32) * 7 % (E + 1)
        out, rows, off = moe.moe_permute(x.contiguous(), ids.unsqueeze(1).contiguous(), E, workspace=ws)
        order = torch.sort(ids, stable=True).indices
        n = int((ids < E).sum())
        assert torch.equal(out.view(torch.int32).flatten()[:n].long(), order[:n]) and int(off[E]) == n
    g = gen(1)
    K = N = 512
    ws = torch.empty(max(moe.moe_linear_backward_workspace_size(T, K, N) for T in (64, 512, 4096)), dtype=torch.uint8, device="cuda")
    w = cuda(rnd(g, N, K))
    for T in (4096, 512, 64):
        d, x = cuda(rnd(g, T, N)), cuda(rnd(g, T, K))
        assert all(torch.equal(p, q) for p, q in zip(moe.moe_linear_backward(d, x, w, workspace=ws), moe.moe_linear_backward(d, x, w)))


@pytest.mark.parametrize("T,H", [(40, 264), (300, 4104), (1030, 96), (1100, 1001), (30, 16400)])
def test_layer_norm_backward_of_far_means(moe, T, H):  # noqa: F811
    """The forward's statistics and the gradients from them against fp64 with the mean
    as it is: what the saved mean loses is F |mean| r of n, which train_ref's tolerance
    has (its F (|s| + |mean|) r), and rstd is within 8 F of itself, as in the forward's
    test of such rows."""
    g = gen(T + H)
    s = rnd(g, T, H, dtype=F32) + torch.tensor([0.0, 1e3, -3e4, 3e4])[torch.arange(T) % 4].unsqueeze(1)
    dy, w = rnd(g, T, H), rnd(g, H, dtype=F32)
    zero = torch.zeros(T, H, dtype=BF)
    _, s2, mean, rstd = moe.moe_layer_norm_forward(cuda(zero), cuda(w), residual=cuda(s), save_stats=True)
    assert torch.equal(s2.cpu(), s)
    _, dres, dw, db = moe.moe_layer_norm_backward(cuda(dy), s2, mean, rstd, cuda(w), need_dx=False, need_dresidual=True)
    _, _, m, q = ref.layer_norm(dbl(s), None, dbl(w), None, 1e-5)
    want, tols = ref.layer_norm_backward(dbl(dy), dbl(s), m, q, dbl(w))
    n, gr = (dbl(s) - m.unsqueeze(1)) * q.unsqueeze(1), dbl(dy) * dbl(w)
    gn = (gr * n).abs().mean(1, keepdim=True)
    near(dres, want[0], tols[0] + 8 * F24 * (want[0].abs() + 2 * q.unsqueeze(1) * n.abs() * gn), "dresidual")
    near(dw, want[1], tols[1] + 8 * F24 * (dbl(dy) * n).abs().sum(0), "dweight")
    near(db, want[2], tols[2], "dbias")


def test_layer_norm_sums_of_more_rows_than_a_launch_exactly(moe):  # noqa: F811
    """Sums over more rows than a launch of the forward takes, to the last row: every
    term and every partial sum is a whole number below 2^24, so fp32 holds them."""
    T, H = (1 << 21) + 3, 8
    x = torch.ones(T, H, dtype=BF, device="cuda")
    x[:, ::2] = -1.0
    x[-4:] *= 2.0
    one = torch.ones(H, device="cuda")
    y, _, mean, rstd = moe.moe_layer_norm_forward(x, one, eps=0.0, save_stats=True)
    assert torch.equal(y, x.sign()) and not bool(mean.any())
    assert bool((rstd[:-4] == 1).all()) and bool((rstd[-4:] == 0.5).all())
    _, _, dw, db = moe.moe_layer_norm_backward(x, x, mean, rstd, one, need_dx=False)
    # (dy n is 1 a row, 2 in the last four)
    assert bool((dw == T + 4).all()) and torch.equal(db, x[0].float() * (T + 4))


@pytest.mark.parametrize("T,H", [(300_000, 8200), (5001, 9000), (4100, 3000), (1024, 16384), (1030, 300), (100, 520)])
def test_layer_norm_sums_exactly(moe, T, H):  # noqa: F811
    """Each row once and no row twice, in the kernels of few, many and wide rows: whole
    numbers, as above."""
    x = torch.ones(T, H, dtype=BF, device="cuda")
    one, mean, rstd = torch.ones(H, device="cuda"), torch.zeros(T, device="cuda"), torch.ones(T, device="cuda")
    rstd[::7] = 2.0
    _, _, dw, db = moe.moe_layer_norm_backward(x, x, mean, rstd, one, need_dx=False)
    assert bool((db == T).all()) and bool((dw == T + -(-T // 7)).all())


# (tiles of 128 and 256 columns, whose lanes trade halves of a row before they store)
@pytest.mark.parametrize("T,K,N", [(1400, 136, 2600), (900, 72, 4104), (4100, 136, 2600), (2048, 520, 5128), (2000, 4104, 1032), (1500, 4104, 1032)])
@pytest.mark.parametrize("a,dt", [(ref.GELU, BF), (ref.NONE, F32), (ref.SILU, BF), (ref.RELU, F32)])
def test_linear_large_tiles_strides_in_place_and_rows_behind(moe, T, K, N, a, dt):  # noqa: F811
    """A strided out in the addend's own rows, and a pre whose rows behind stay."""
    g = gen(T + N + a)
    x, w, b, add = base.linear_case(g, T + 3, K + 16, N + 24, F32, dt)
    w, b = w[:N, :K].contiguous(), b[:N].contiguous()
    buf = cuda(add)
    keep, at = buf.clone(), buf[1:1 + T, 16:16 + N]
    d = at.cpu().clone()
    pre = torch.full((T + 1, N), 7, dtype=BF, device="cuda")
    args = cuda(x)[2:2 + T, 8:8 + K], cuda(w), cuda(b)
    out, _ = moe.moe_linear_forward(*args, act=a, addend=at, out=at, pre=pre[:T])
    assert out.data_ptr() == at.data_ptr()
    base.check_linear(moe, a, x[2:2 + T, 8:8 + K], w, b, d, out, pre[:T])
    keep[1:1 + T, 16:16 + N] = buf[1:1 + T, 16:16 + N]
    assert torch.equal(keep, buf) and bool((pre[T:] == 7).all())
    # the same bits apart, and without a saved argument
    apart = moe.moe_linear_forward(*args, act=a, addend=cuda(d), out_dtype=dt)
    assert torch.equal(apart, out)
