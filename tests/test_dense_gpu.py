"""The dense operators around the routed experts against plain fp64 forms
(MI355X). Tolerances: tests/dense_ref.py."""
import math

import pytest
import torch

from tests import dense_ref as ref

pytestmark = pytest.mark.gpu

B8 = 2.0 ** -8   # half a bf16 step, relative
F24 = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32


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


def weight(g, n, k):
    return rnd(g, n, k, scale=1 / math.sqrt(k))


def adapters(g, T, K, N, n, rank, ranks=True, scale=True, runs=False):
    a = rnd(g, n, rank, K, scale=1 / math.sqrt(K))
    b = rnd(g, n, N, rank, scale=0.5 / math.sqrt(rank))
    index = torch.randint(-1, n, (T,), generator=g, dtype=torch.int32)
    if runs:
        index = index.sort().values
    r = torch.randint(0, rank + 1, (n,), generator=g, dtype=torch.int32) if ranks else None
    s = torch.rand(n, generator=g) + 0.5 if scale else None
    return a, b, index, r, s


def cuda(v):
    if v is None:
        return None
    if isinstance(v, tuple):
        return tuple(cuda(t) for t in v)
    return v.cuda()


def sum_tol(x, w):
    """Bound of the fp32 sums of x @ w.T, per element."""
    return (x.shape[1] / 8 + 64) * F24 * (x.abs() @ w.abs().t())


# ------------------------------------------------------------------ norm
@pytest.mark.parametrize("T,H", [(1, 1), (3, 7), (1, 3584), (5, 33), (2, 64), (4, 1000), (7, 2784), (2050, 520),
                                 (2049, 1032), (2051, 3584), (3, 4104), (2, 8192), (3, 16384), (2, 20000),
                                 (1, 65536)])
@pytest.mark.parametrize("res", [None, BF, F32])
def test_norm(moe, T, H, res):
    g = gen(T * 131 + H)
    x = rnd(g, T, H)
    r = None if res is None else rnd(g, T, H, scale=3, dtype=res)
    w = rnd(g, H, dtype=F32 if res == F32 else BF)
    mx = H % 32 == 0
    y, ro, q, qs = moe.moe_rms_norm(cuda(x), cuda(w), residual=cuda(r), eps=1e-5, weight_offset=1.0, mxfp8=mx)
    s, v = ref.norm(x.double(), None if r is None else r.double(), w.double(), 1e-5, 1.0)
    # fp32: the sum, its root, the quotient and two products, each 2^-24, and
    # the squares' sum of at most 64 + 10 terms in a row
    f = 90 * F24
    # offset + weight cancels where weight is near -1: 2^-24 of the offset
    k = f * (s / torch.sqrt((s * s).mean(-1, keepdim=True) + 1e-5)).abs()
    ref.check(y, v, B8 * (1 + 2 ** -7) + f, absolute=float(k.max()), what="y")
    if r is None:
        assert ro is None
    else:
        ref.check(ro, s, B8 if res == BF else F24, what="residual_out")
    if mx:
        qf, sf = q.double().cpu(), qs.double().cpu()
        want = ref.mx_scale(v)
        # equal, but where the block's maximum is at the border of two scales
        amax = v.unflatten(-1, (-1, 32)).abs().amax(-1)
        border = (ref.mx_scale(v * (1 + 1e-4)) != ref.mx_scale(v * (1 - 1e-4)))
        assert bool(((sf == want) | border).all()) and float(amax.min()) > 0
        got = ref.mx_wide(qf, sf)
        tol = torch.maximum(2.0 ** -4 * v.abs(), 2.0 ** -10 * sf.repeat_interleave(32, -1)) + k + 1e-5 * v.abs()
        assert bool(((got - v).abs() <= tol).all())


def test_norm_in_place_strides_and_rows_behind(moe):
    g = gen(3)
    T, H = 5, 96
    big = rnd(g, 8, H + 40).cuda()
    res = rnd(g, 8, H + 8, dtype=F32).cuda()
    keep, keep_r = big.clone(), res.clone()
    w = rnd(g, H).cuda()
    x, r = big[1:1 + T, 3:3 + H], res[2:2 + T, :H]  # rows that are not 16-byte aligned
    s, v = ref.norm(x.double().cpu(), r.double().cpu(), w.double().cpu(), 1e-6, 0.0)
    q = torch.full((8, H + 5), 77, dtype=torch.uint8, device="cuda")
    y, ro, _, qs = moe.moe_rms_norm(x, w, residual=r, y=x, residual_out=r, q=q[:T, 1:1 + H], mxfp8=True)
    assert y.data_ptr() == x.data_ptr() and ro.data_ptr() == r.data_ptr()
    ref.check(y, v, B8 * 1.01, what="y")
    ref.check(ro, s, F24, what="residual")
    got = ref.mx_wide(q[:T, 1:1 + H].view(torch.float8_e4m3fn).double().cpu(), qs.double().cpu())
    tol = torch.maximum(2.0 ** -4 * v.abs(), 2.0 ** -10 * qs.double().cpu().repeat_interleave(32, -1))
    assert bool(((got - v).abs() <= tol * 1.001).all())
    keep[1:1 + T, 3:3 + H] = big[1:1 + T, 3:3 + H]
    keep_r[2:2 + T, :H] = res[2:2 + T, :H]
    assert torch.equal(keep, big) and torch.equal(keep_r, res)
    assert bool((q[T:] == 77).all()) and bool((q[:, 0] == 77).all()) and bool((q[:, 1 + H:] == 77).all())


def test_norm_of_more_rows_than_a_launch(moe):
    T, H = (1 << 21) + 3, 8
    x = torch.ones(T, H, dtype=BF, device="cuda")
    x[-4:] = 2.0
    x[: 1 << 21] *= 3.0
    y, _, _, _ = moe.moe_rms_norm(x, torch.ones(H, dtype=BF, device="cuda"), eps=0.0)
    assert bool((y == 1).all())


@pytest.mark.parametrize("H", [1536, 2784])
@pytest.mark.parametrize("res", [None, BF, F32])
def test_norm_codes_are_exact(moe, H, res):
    """A code is the one of the exact value: the product is carried to 2^-45,
    so of 2^22 elements none is expected within that of a tie."""
    g = gen(H)
    T = (1 << 22) // H
    x, w = rnd(g, T, H), rnd(g, H)
    r = None if res is None else rnd(g, T, H, scale=3, dtype=res)
    _, _, q, qs = moe.moe_rms_norm(cuda(x), cuda(w), residual=cuda(r), mxfp8=True)
    _, v = ref.norm(x.double(), None if r is None else r.double(), w.double(), 1e-6, 0.0)
    want, scale = ref.mx_quant(v)
    assert torch.equal(qs.double().cpu(), scale)
    assert torch.equal(q.double().cpu(), want)


def _just_above_448():
    """(s, w) with s w / 2 above 1.75 by less than half an fp32 step there, so
    that it rounds to it."""
    for m in range(129, 256):
        s = m / 128  # a bf16 number
        w = torch.tensor(3.5 / s, dtype=torch.float64).float().double()
        for w in (w, torch.nextafter(w.float(), torch.tensor(9.0)).double()):
            if 0 < float(s * w / 2) - 1.75 < 2.0 ** -24:
                yield s, float(w)


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("far", [0, 31])
def test_norm_scale_of_a_value_that_rounds_to_the_border(moe, sign, far):
    """The largest e4m3 is 448 = 1.75 * 2^8: a block whose exact maximum is
    above 1.75 takes the next scale, though its fp32 number is 1.75."""
    H, seen = 64, 0
    for s, w in _just_above_448():
        x, wt = torch.ones(1, H), torch.full((H,), 0.25)
        x[0, 32 + far], wt[32 + far] = s * sign, w
        eps = 4 - float(x.double().square().mean())
        assert torch.tensor(eps).double() == eps
        _, v = ref.norm(x.double(), None, wt.double(), eps, 0.0)
        assert float(v.abs().max()) > 1.75 and float(v.abs().max().float()) == 1.75
        want, scale = ref.mx_quant(v)
        _, _, q, qs = moe.moe_rms_norm(cuda(x.bfloat16()), cuda(wt), eps=eps, mxfp8=True)
        assert torch.equal(qs.double().cpu(), scale) and torch.equal(q.double().cpu(), want), (s, w)
        # and not above: the smaller scale
        wt[32 + far] = 1.75 / (s / 2)
        _, v = ref.norm(x.double(), None, wt.double(), eps, 0.0)
        if float(v.abs().max()) <= 1.75:
            want, scale = ref.mx_quant(v)
            _, _, q, qs = moe.moe_rms_norm(cuda(x.bfloat16()), cuda(wt), eps=eps, mxfp8=True)
            assert torch.equal(qs.double().cpu(), scale) and torch.equal(q.double().cpu(), want), (s, w)
        seen += 1
    assert seen >= 5


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("k", [-10, -9, -8, -7, -6, -5, 0, 4])
def test_norm_codes_next_to_ties(moe, sign, k):
    """Exact values next to a tie of two codes that round to it in fp32, in the
    normal range of e4m3 (2^-6 and more) and below it (steps of 2^-9). r = 1/2
    exactly, and the block's scale is 1."""
    H, seen = 64, 0
    x, wt = torch.ones(1, H), torch.full((H,), 1.0)
    wt[32] = 2.0 * 448
    step = 2.0 ** (max(k, -6) - 3)
    for n in range(int(2.0 ** k / step), int(2.0 ** (k + 1) / step)) if k > -10 else [0]:
        tie = (n + 0.5) * step  # its fp32 neighbours are 2^-24 of it or more apart
        for m in range(129, 256, 2):
            s = m / 128
            w = float(torch.tensor(2 * tie / s, dtype=torch.float64).float())
            v = s * w / 2  # 8 and 24 bits: exact in fp64
            if v != tie and float(torch.tensor(v, dtype=torch.float64).float()) == tie:
                x[0, 40], wt[40] = s * sign, w
                eps = 4 - float(x.double().square().mean())
                _, v = ref.norm(x.double(), None, wt.double(), eps, 0.0)
                want, scale = ref.mx_quant(v)
                _, _, q, qs = moe.moe_rms_norm(cuda(x.bfloat16()), cuda(wt), eps=eps, mxfp8=True)
                assert torch.equal(qs.double().cpu(), scale) and torch.equal(q.double().cpu(), want), (n, s, w)
                seen += 1
    assert seen >= 3


def test_norm_special_values(moe):
    H = 64
    x = torch.zeros(6, H)
    x[1] = 1e-30        # squares vanish next to eps
    x[2, 5] = math.nan  # the row, and only the row
    x[3, 40] = math.inf
    x[4] = 3e38
    x[5] = 2.0
    w = torch.ones(H)
    w[33] = math.nan    # one element of every row, not its block
    y, _, q, qs = moe.moe_rms_norm(x.bfloat16().cuda(), w.cuda(), eps=1e-6, mxfp8=True)
    y, q, qs = y.float().cpu(), q.float().cpu(), qs.float().cpu()
    other = torch.arange(H) != 33
    assert bool(y[:, 33].isnan().all()) and bool(q[:, 33].isnan().all())
    assert bool((y[0][other] == 0).all()) and bool((q[0][other] == 0).all())
    assert float(qs[0, 0]) == 2.0 ** -127
    assert bool(y[2].isnan().all()) and bool(q[2].isnan().all())
    assert bool(y[3][other & (torch.arange(H) != 40)].eq(0).all()) and bool(y[3, 40].isnan())
    assert bool(y[4][other].eq(1).all())  # fp32 squares would overflow: by the formula each is 1
    assert bool((y[5][other] == 1).all())
    assert bool((q[5][other] * qs[5].repeat_interleave(32)[other] == 1).all())


# ---------------------------------------------------------------- linear
LINEAR = [(1, 8, 8), (1, 3584, 112), (3, 72, 40), (16, 520, 1000), (17, 136, 24), (33, 3584, 384), (64, 64, 72),
          (65, 72, 136), (130, 1000, 520), (300, 3584, 896), (777, 264, 1032), (2100, 192, 4104), (4200, 200, 64)]


@pytest.mark.parametrize("T,K,N", LINEAR)
def test_linear(moe, T, K, N):
    g = gen(T + K + N)
    x, w = rnd(g, T, K), weight(g, N, K)
    want = x.double() @ w.double().t()
    tol = sum_tol(x.double(), w.double())
    got = moe.moe_lora_linear(cuda(x), cuda(w), out_dtype=F32)
    assert got.dtype == F32
    assert bool(((got.double().cpu() - want).abs() <= tol).all())
    got = moe.moe_lora_linear(cuda(x), cuda(w))
    assert bool(((got.double().cpu() - want).abs() <= tol * 1.01 + B8 * want.abs()).all())


@pytest.mark.parametrize("T,K,N", LINEAR)
@pytest.mark.parametrize("n,rank,runs", [(1, 8, False), (5, 40, True), (40, 16, False)])
def test_linear_adapters(moe, T, K, N, n, rank, runs):
    g = gen(T + K + N + n)
    x, w = rnd(g, T, K), weight(g, N, K)
    lo = adapters(g, T, K, N, n, rank, runs=runs)
    # what lies beyond an adapter's rank is never read as numbers
    for i in range(n):
        lo[0][i, int(lo[3][i]):] = math.nan
        lo[1][i, :, int(lo[3][i]):] = math.inf
    xd = x.double()
    want = xd @ w.double().t() + ref.lora(xd, lo)
    # the narrow product's sum, and two bf16 halves of v: 2^-16 of |B| |v|
    wide = tuple(t if t is None or not t.is_floating_point() else torch.nan_to_num(t.double(), 0, 0, 0).abs() for t in lo)
    extra = ref.lora(xd.abs(), wide)
    tol = sum_tol(xd, w.double()) + extra * (2.0 ** -16 + (K / 8 + 128) * F24)
    got = moe.moe_lora_linear(cuda(x), cuda(w), lora=cuda(lo), out_dtype=F32)
    assert bool(((got.double().cpu() - want).abs() <= tol).all())
    got = moe.moe_lora_linear(cuda(x), cuda(w), lora=moe.LoraAdapters(*cuda(lo)))
    assert bool(((got.double().cpu() - want).abs() <= tol * 1.01 + B8 * want.abs()).all())


@pytest.mark.parametrize("T,K,N,n,runs", [
    (257, 72, 304, 3, False),      # a tile's own rows
    (300, 1032, 264, 40, False),   # K in parts, joined token by token
    (1500, 264, 2056, 30, False),  # tiles side by side
    (1500, 264, 2056, 30, True),
    (9000, 136, 1160, 5, False),   # a sort in more than one batch, large tiles
    (400, 64, 128, 1023, False),   # the most adapters of a sort
    (400, 64, 128, 1024, False),   # and one more
])
def test_linear_adapters_by_order(moe, T, K, N, n, runs):
    """Many tokens are taken adapter by adapter; x and out have rows of their
    own strides, and what lies behind them stays."""
    g = gen(T + n)
    rank = 72
    xb, w = rnd(g, T, K + 8), weight(g, N, K)
    lo = adapters(g, T, K, N, n, rank, runs=runs)
    for i in range(n):
        lo[0][i, int(lo[3][i]):] = math.nan
        lo[1][i, :, int(lo[3][i]):] = math.inf
    xd = xb[:, :K].double()
    want = xd @ w.double().t() + ref.lora(xd, lo)
    wide = tuple(t if t is None or not t.is_floating_point() else torch.nan_to_num(t.double(), 0, 0, 0).abs() for t in lo)
    extra = ref.lora(xd.abs(), wide)
    tol = sum_tol(xd, w.double()) + extra * (2.0 ** -16 + (K / 8 + 128) * F24)
    out = torch.full((T + 2, N + 8), 5.0, dtype=F32, device="cuda")
    moe.moe_lora_linear(cuda(xb)[:, :K], cuda(w), lora=cuda(lo), out=out[:T, :N])
    assert bool(((out[:T, :N].double().cpu() - want).abs() <= tol).all())
    assert bool((out[T:] == 5).all()) and bool((out[:, N:] == 5).all())
    # a token's result does not depend on its place
    p = torch.randperm(T, generator=g)
    lo2 = (lo[0], lo[1], lo[2][p], lo[3], lo[4])
    got = moe.moe_lora_linear(cuda(xb[p])[:, :K], cuda(w), lora=cuda(lo2), out_dtype=F32)
    assert torch.equal(got, out[:T, :N][p.cuda()])


@pytest.mark.parametrize("same", [True, False])
@pytest.mark.parametrize("T,H,I", [(700, 264, 392), (3000, 136, 2056)])
def test_ffn_adapters_by_order(moe, T, H, I, same):
    g = gen(T + I)
    x, w13, w2, add = rnd(g, T, H), weight(g, 2 * I, H), weight(g, H, I), rnd(g, T, H)
    l13 = adapters(g, T, H, 2 * I, 7, 24)
    l2 = adapters(g, T, I, H, 7, 16)
    c13, c2 = cuda(l13), cuda(l2)
    if same:  # one index tensor for both
        l2 = (l2[0], l2[1], l13[2], l2[3], l2[4])
        c2 = (c2[0], c2[1], c13[2], c2[3], c2[4])
    want, gu, h = ref.ffn(x.double(), w13.double(), w2.double(), add.double(), l13, l2)
    out = cuda(add)  # the addend's own buffer
    _, saved = moe.moe_ffn_forward(cuda(x), cuda(w13), cuda(w2), addend=out, lora13=c13, lora2=c2, out=out,
                                   save_gate_up=True)
    ref.check(saved, gu, B8, rms=1e-4, what="gate_up")
    ref.check(out, want, B8, rms=ref.FLIPS, absolute=ref.step_tol(h, w2.double()), what="out", norm=ref.NORM)


@pytest.mark.parametrize("T,K,N", [(17, 72, 4096), (25, 264, 4104), (25, 2056, 4624), (40, 136, 16400), (20, 72, 20000),
                                   (64, 520, 8200), (33, 72, 2040), (33, 72, 2048)])
@pytest.mark.parametrize("n", [0, 3])
def test_linear_few_tokens_many_rows(moe, T, K, N, n):
    g = gen(T + N + n)
    x, w = rnd(g, T, K), weight(g, N, K)
    xd, wd = x.double(), w.double()
    want, tol = xd @ wd.t(), sum_tol(xd, wd)
    lo = None
    if n:
        lo = adapters(g, T, K, N, n, 16, ranks=False)
        want += ref.lora(xd, lo)
        wide = tuple(t if t is None or not t.is_floating_point() else t.double().abs() for t in lo)
        tol += ref.lora(xd.abs(), wide) * (2.0 ** -16 + (K / 8 + 128) * F24)
    got = moe.moe_lora_linear(cuda(x), cuda(w), lora=cuda(lo), out_dtype=F32)
    assert bool(((got.double().cpu() - want).abs() <= tol).all())
    assert torch.equal(moe.moe_lora_linear(cuda(x), cuda(w), lora=cuda(lo)), got.bfloat16())


@pytest.mark.parametrize("T", [9, 200, 500])
def test_linear_tokens_do_not_meet(moe, T):
    """A NaN in one token, or in one adapter, stays with its tokens."""
    g = gen(T)
    K, N, n = 136, 72, 3
    x, w = rnd(g, T, K), weight(g, N, K)
    lo = adapters(g, T, K, N, n, 16, ranks=False, scale=False)
    clean = moe.moe_lora_linear(cuda(x), cuda(w), lora=cuda(lo))
    x[4, 7] = math.nan
    lo[0][1, 3, 5] = math.inf
    lo[1][1, 2, 3] = math.nan
    got = moe.moe_lora_linear(cuda(x), cuda(w), lora=cuda(lo))
    hit = (lo[2] == 1) | (torch.arange(T) == 4)
    assert torch.equal(got[~hit.cuda()], clean[~hit.cuda()])
    assert bool(got[4].isnan().all())


@pytest.mark.parametrize("T", [5, 70, 200, 400])
def test_linear_infinite_scale(moe, T):
    """An infinite scale takes part in the adapter's own rank alone."""
    g = gen(T)
    K, N, n = 64, 96, 4
    x, w = rnd(g, T, K).abs(), weight(g, N, K)
    a, b, index, _, _ = adapters(g, T, K, N, n, 24, ranks=False, scale=False)
    lo = (a.abs() + 0.01, b.abs() + 0.01, index, torch.tensor([8, 24, 0, 13], dtype=torch.int32),
          torch.tensor([math.inf, 1.0, math.inf, math.inf]))
    got = moe.moe_lora_linear(cuda(x), cuda(w), lora=cuda(lo)).cpu()
    hit = (index == 0) | (index == 3)
    assert bool(got[hit].isinf().all()) and bool(got[~hit].isfinite().all())


# One part of K; parts joined token by token (tokens in their own order, and by
# adapter); parts that the tiles read (N of more rows than are split over).
@pytest.mark.parametrize("T,K,N", [(5, 64, 96), (40, 1024, 96), (70, 64, 96), (70, 1024, 96), (200, 64, 96), (200, 1024, 96), (400, 1024, 96),
                                   (200, 264, 2056), (400, 264, 2056), (2100, 264, 4104), (5000, 64, 96)])
@pytest.mark.parametrize("ranks", [True, False])
def test_linear_infinite_scale_over_parts(moe, T, K, N, ranks):
    """An infinite scale acts within the rank alone, on every path: an adapter
    of rank 0 adds nothing, A x of 0 within the rank becomes a NaN, other
    values infinities."""
    g = gen(T + K)
    n, rank = 5, 24
    x, w = rnd(g, T, K).abs(), weight(g, N, K)
    a, b, index, _, _ = adapters(g, T, K, N, n, rank, ranks=False, scale=False)
    a, b = a.abs() + 0.01, b.abs() + 0.01
    a[4, 5] = 0
    r = torch.tensor([8, 24, 0, 13, 8], dtype=torch.int32) if ranks else None
    scale = torch.tensor([math.inf, 1.0, math.inf if ranks else 2.0, math.inf, math.inf])
    plain = moe.moe_lora_linear(cuda(x), cuda(w)).cpu()
    got = moe.moe_lora_linear(cuda(x), cuda(w), lora=cuda((a, b, index, r, scale))).cpu()
    assert bool(got[(index == 0) | (index == 3)].isinf().all()) and bool(got[index == 4].isnan().all())
    assert bool(got[(index < 0) | (index == 1) | (index == 2)].isfinite().all())
    same = (index < 0) | (index == 2) if ranks else index < 0
    assert torch.equal(got[same], plain[same])


@pytest.mark.parametrize("T", [5, 70, 300])
def test_linear_index_outside_and_defaults(moe, T):
    g = gen(T)
    K, N, n = 64, 96, 4
    x, w = rnd(g, T, K), weight(g, N, K)
    lo = list(adapters(g, T, K, N, n, 8, ranks=False, scale=False))
    plain = moe.moe_lora_linear(cuda(x), cuda(w))
    for bad in (-1, n, 2 ** 31 - 1, -2 ** 31):
        lo[2] = torch.full((T,), bad, dtype=torch.int32)
        assert torch.equal(moe.moe_lora_linear(cuda(x), cuda(w), lora=cuda(tuple(lo))), plain)
    lo[2] = torch.full((T,), 2, dtype=torch.int32)
    lo[3] = torch.tensor([8, 8, 1000, 8], dtype=torch.int32)  # clamped to the stack's rank
    a = moe.moe_lora_linear(cuda(x), cuda(w), lora=cuda(tuple(lo)))
    lo[3] = None
    assert torch.equal(a, moe.moe_lora_linear(cuda(x), cuda(w), lora=cuda(tuple(lo))))


@pytest.mark.parametrize("T,K,N", [(5, 64, 96), (40, 1024, 96), (70, 64, 96), (200, 1024, 96), (200, 264, 2056),
                                   (400, 264, 2056), (5000, 64, 96)])
def test_linear_ranks_outside_are_clamped(moe, T, K, N):
    """Any int32 below 0 is rank 0, any above the stack's rank is the stack's."""
    g = gen(T + N)
    n, rank = 5, 40
    x, w = rnd(g, T, K), weight(g, N, K)
    a, b, index, _, scale = adapters(g, T, K, N, n, rank, ranks=False)
    want = moe.moe_lora_linear(cuda(x), cuda(w), lora=cuda((a, b, index, torch.tensor([0, 40, 0, 0, 40], dtype=torch.int32), scale)))
    r = torch.tensor([-2 ** 31, 2 ** 31 - 1, -2 ** 31 + 1, -1, 41], dtype=torch.int32)
    b[0], b[2], b[3] = math.inf, math.nan, math.inf
    got = moe.moe_lora_linear(cuda(x), cuda(w), lora=cuda((a, b, index, r, scale)))
    assert torch.equal(got, want)


@pytest.mark.parametrize("T", [6, 90, 260])
def test_linear_strides_and_rows_behind(moe, T):
    g = gen(T)
    K, N = 72, 40
    xb, w = rnd(g, T + 2, K + 24), weight(g, N, K)
    out = torch.full((T + 3, N + 16), 5.0, dtype=F32, device="cuda")
    x = cuda(xb)[1:1 + T, 8:8 + K]
    moe.moe_lora_linear(x, cuda(w), out=out[:T, 8:8 + N])
    want = xb[1:1 + T, 8:8 + K].double() @ w.double().t()
    tol = sum_tol(xb[1:1 + T, 8:8 + K].double(), w.double())
    assert bool(((out[:T, 8:8 + N].double().cpu() - want).abs() <= tol).all())
    assert bool((out[T:] == 5).all()) and bool((out[:, :8] == 5).all()) and bool((out[:, 8 + N:] == 5).all())


# ------------------------------------------------------------------- ffn
FFN = [(20, 72, 4200), (50, 4200, 72), (1, 8, 8), (1, 3584, 384), (2, 40, 72), (16, 520, 136), (17, 264, 1000), (37, 3584, 128), (64, 96, 64),
       (65, 136, 72), (129, 520, 264), (300, 1032, 1000), (1030, 264, 392), (2200, 136, 2056)]


@pytest.mark.parametrize("T,H,I", FFN)
@pytest.mark.parametrize("lora", [False, True])
def test_ffn_forward(moe, T, H, I, lora):
    g = gen(T + H + I)
    x, w13, w2, add = rnd(g, T, H), weight(g, 2 * I, H), weight(g, H, I), rnd(g, T, H)
    l13 = adapters(g, T, H, 2 * I, 6, 24) if lora else None
    l2 = adapters(g, T, I, H, 6, 16) if lora else None
    want, gu, h = ref.ffn(x.double(), w13.double(), w2.double(), add.double(), l13, l2)
    step = ref.step_tol(h, w2.double())
    got, saved = moe.moe_ffn_forward(cuda(x), cuda(w13), cuda(w2), addend=cuda(add), lora13=cuda(l13),
                                     lora2=cuda(l2), save_gate_up=True)
    ref.check(saved, gu, B8, rms=1e-4, what="gate_up")
    ref.check(got, want, B8, rms=ref.FLIPS, absolute=step, what="out", norm=ref.NORM)
    assert torch.equal(moe.moe_ffn_forward(cuda(x), cuda(w13), cuda(w2), addend=cuda(add), lora13=cuda(l13),
                                           lora2=cuda(l2)), got)
    if not lora:
        want, _, _ = ref.ffn(x.double(), w13.double(), w2.double())
        ref.check(moe.moe_ffn_forward(cuda(x), cuda(w13), cuda(w2)), want, B8, rms=ref.FLIPS, absolute=step,
                  what="no addend", norm=ref.NORM)


@pytest.mark.parametrize("T,H,I", [(1, 32, 32), (20, 64, 2080), (32, 4128, 64), (1, 3584, 384), (5, 96, 160), (16, 544, 128), (20, 128, 1024),
                                   (40, 256, 96), (64, 1056, 64), (65, 96, 160), (130, 544, 288), (300, 1024, 1056),
                                   (1030, 288, 384), (2200, 160, 2080)])
def test_ffn_forward_mxfp8(moe, T, H, I):
    g = gen(T + H + I)
    mats = []
    for n, k, s in ((T, H, 1.0), (2 * I, H, 1 / math.sqrt(H)), (H, I, 1 / math.sqrt(I))):
        q, sc = ref.mx_quant(rnd(g, n, k, scale=s).double())
        mats += [q.float().to(torch.float8_e4m3fn), sc.float().to(torch.float8_e8m0fnu)]
    add = rnd(g, T, H)
    x, w13, w2 = (ref.mx_wide(mats[i].float(), mats[i + 1].float()) for i in (0, 2, 4))
    gu = x @ w13.t()
    h = ref.mx_wide(*ref.mx_quant(ref.silu(gu[:, :I]) * gu[:, I:]))
    want = h @ w2.t()
    dev = [cuda(m) for m in mats]
    got = moe.moe_ffn_forward_mxfp8(*dev, addend=cuda(add))
    step = ref.step_tol(h, w2, 2.0 ** -3)
    ref.check(got, want + add.double(), B8, rms=ref.MXFLIPS, absolute=step, what="out", norm=ref.MXNORM)
    as_bytes = [m.view(torch.uint8) for m in dev]
    ref.check(moe.moe_ffn_forward_mxfp8(*as_bytes), want, B8, rms=ref.MXFLIPS, absolute=step, what="no addend",
              norm=ref.MXNORM)


def test_ffn_addend_in_place_and_strides(moe):
    g = gen(11)
    for T in (3, 100, 280):
        H, I = 136, 72
        x, w13, w2 = rnd(g, T, H + 8), weight(g, 2 * I, H), weight(g, H, I)
        buf = rnd(g, T + 2, H + 32)
        want, _, h = ref.ffn(x[:, 8:].double(), w13.double(), w2.double(), buf[:T, 16:16 + H].double())
        b = cuda(buf)
        moe.moe_ffn_forward(cuda(x)[:, 8:], cuda(w13), cuda(w2), addend=b[:T, 16:16 + H], out=b[:T, 16:16 + H])
        ref.check(b[:T, 16:16 + H], want, B8, rms=ref.FLIPS, absolute=ref.step_tol(h, w2.double()), what="out")
        after = b.cpu()
        after[:T, 16:16 + H] = buf[:T, 16:16 + H]
        assert torch.equal(after, buf)


@pytest.mark.parametrize("T", [3, 200])
def test_ffn_tokens_do_not_meet(moe, T):
    g = gen(T)
    H, I = 72, 264
    x, w13, w2 = rnd(g, T, H), weight(g, 2 * I, H), weight(g, H, I)
    clean = moe.moe_ffn_forward(cuda(x), cuda(w13), cuda(w2))
    x[1, 9] = math.inf
    got = moe.moe_ffn_forward(cuda(x), cuda(w13), cuda(w2))
    rows = torch.arange(T, device="cuda") != 1
    assert torch.equal(got[rows], clean[rows]) and not bool(torch.isfinite(got[1]).any())


# -------------------------------------------------------------- backward
@pytest.mark.parametrize("T,H,I", [(1, 8, 8), (2, 40, 72), (16, 520, 136), (63, 264, 1000), (64, 96, 64), (65, 136, 72),
                                   (129, 520, 264), (300, 1032, 520), (777, 264, 392), (2200, 1032, 2056),
                                   # parts of K for dh and dx, dx alone, 128 x 128 tiles
                                   (1, 2056, 1032), (130, 264, 4104), (200, 2056, 2760), (520, 1032, 1032)])
def test_ffn_backward(moe, T, H, I):
    g = gen(T + H + I)
    dout, x, gu = rnd(g, T, H), rnd(g, T, H), rnd(g, T, 2 * I)
    w13, w2 = weight(g, 2 * I, H), weight(g, H, I)
    want, steps = ref.ffn_backward(*(t.double() for t in (dout, x, gu, w13, w2)))
    got = moe.moe_ffn_backward(*(cuda(t) for t in (dout, x, gu, w13, w2)))
    for name, a, b, st in zip(("dx", "dw13", "dw2"), got, want, steps):
        ref.check(a, b, B8, rms=ref.FLIPS, absolute=st, what=name, norm=ref.NORM)
    again = moe.moe_ffn_backward(*(cuda(t) for t in (dout, x, gu, w13, w2)))
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    # each gradient alone is the same
    for k in range(3):
        need = [i == k for i in range(3)]
        one = moe.moe_ffn_backward(*(cuda(t) for t in (dout, x, gu, w13, w2)), *need)
        assert [t is not None for t in one] == need and torch.equal(one[k], got[k])


def test_ffn_backward_of_no_tokens(moe):
    H, I = 64, 96
    e = torch.empty(0, H, dtype=BF, device="cuda")
    w13, w2 = torch.ones(2 * I, H, dtype=BF, device="cuda"), torch.ones(H, I, dtype=BF, device="cuda")
    d13, d2 = torch.full_like(w13, math.nan), torch.full_like(w2, math.nan)
    dx, _, _ = moe.moe_ffn_backward(e, e, torch.empty(0, 2 * I, dtype=BF, device="cuda"), w13, w2, dw13=d13, dw2=d2)
    assert dx.shape == (0, H) and not bool(d13.any()) and not bool(d2.any())


@pytest.mark.parametrize("H,I", [(64, 96), (1024, 1024), (3584, 2048)])  # tiles of 64, 128 and 256
@pytest.mark.parametrize("given", [(True, True, True), (True, True, False), (True, False, False)])
def test_ffn_backward_of_no_tokens_with_addresses(moe, H, I, given):
    """From C an empty dx may have an address: nothing is written there, and
    the weights' gradients are zeros."""
    w13, w2 = torch.ones(2 * I, H, dtype=BF, device="cuda"), torch.ones(H, I, dtype=BF, device="cuda")
    grads = [torch.full_like(t, math.nan) if on else None
             for t, on in zip((torch.empty(8, H, dtype=BF, device="cuda"), w13, w2), given)]
    ptrs = [None if t is None else t.data_ptr() for t in grads]
    p, s = w13.data_ptr(), torch.cuda.current_stream().cuda_stream
    status = moe.lib.moe_ffn_backward(p, H, p, H, p, p, w2.data_ptr(), 0, 0, H, I, ptrs[0], H, ptrs[1], ptrs[2], None, 0, s)
    assert status == moe.MOE_OK, moe.moe_last_error()
    torch.cuda.synchronize()
    assert bool(grads[0].isnan().all())
    assert all(not bool(t.any()) for t in grads[1:] if t is not None)


@pytest.mark.parametrize("frozen", [True, False])
def test_moe_ffn_gradients_of_no_tokens(moe, frozen):
    H, I = 64, 96
    x = torch.empty(0, H, dtype=BF, device="cuda", requires_grad=True)
    w13 = torch.ones(2 * I, H, dtype=BF, device="cuda", requires_grad=not frozen)
    w2 = torch.ones(H, I, dtype=BF, device="cuda", requires_grad=not frozen)
    moe.moe_ffn(x, w13, w2).sum().backward()
    assert x.grad.shape == (0, H)
    if not frozen:
        assert not bool(w13.grad.any()) and not bool(w2.grad.any())


@pytest.mark.parametrize("T", [4, 150])
def test_moe_ffn_gradients(moe, T):
    """The differentiable form against the formula and against differences of
    the fp64 forward."""
    g = gen(T)
    H, I = 136, 200
    x, w13, w2, add = rnd(g, T, H), weight(g, 2 * I, H), weight(g, H, I), rnd(g, T, H)
    leaves = [cuda(t).requires_grad_() for t in (x, w13, w2, add)]
    out = moe.moe_ffn(*leaves)
    probe = rnd(g, T, H)
    out.backward(cuda(probe))
    d = [t.double() for t in (x, w13, w2, add)]
    gu = moe.moe_ffn_forward(*(t.detach() for t in leaves[:3]), save_gate_up=True)[1].double().cpu()
    want, steps = ref.ffn_backward(probe.double(), d[0], gu, d[1], d[2])
    for name, leaf, b, st in zip(("dx", "dw13", "dw2"), leaves, want, steps):
        ref.check(leaf.grad, b, B8, rms=ref.FLIPS, absolute=st, what=name, norm=ref.NORM)
    assert torch.equal(leaves[3].grad.cpu(), probe)

    def loss(x, w13, w2, add):
        gu = x @ w13.t()
        return float((((ref.silu(gu[:, :I]) * gu[:, I:]) @ w2.t() + add) * probe.double()).sum())

    for k, leaf in enumerate(leaves):
        step = rnd(g, *leaf.shape, dtype=torch.float64)
        e = 1e-5
        plus, minus = list(d), list(d)
        plus[k], minus[k] = d[k] + e * step, d[k] - e * step
        slope = (loss(*plus) - loss(*minus)) / (2 * e)
        grad = leaf.grad.double().cpu()
        # Each element of the gradient is off by at most about three bf16
        # roundings (saved gate_up, operand, result); over a random direction
        # they add like independent errors of 3 * 2^-8: six of their sums.
        tol = 6 * 3 * B8 * float((grad * step).square().sum().sqrt())
        assert abs(float((grad * step).sum()) - slope) <= tol, (k, slope)


def test_moe_ffn_partial_and_expanded_gradients(moe):
    g = gen(8)
    T, H, I = 20, 64, 96
    x, w13, w2 = cuda(rnd(g, T, H)), cuda(weight(g, 2 * I, H)), cuda(weight(g, H, I))
    xr = x.clone().requires_grad_()
    moe.moe_ffn(xr, w13, w2).sum().backward()  # the gradient is one expanded value
    _, gu = moe.moe_ffn_forward(x, w13, w2, save_gate_up=True)
    dx, _, _ = moe.moe_ffn_backward(torch.ones(T, H, dtype=BF, device="cuda"), x, gu, w13, w2)
    assert torch.equal(xr.grad, dx)
    assert not moe.moe_ffn(x, w13, w2).requires_grad
    a = torch.zeros(T, H, dtype=BF, device="cuda", requires_grad=True)
    moe.moe_ffn(x, w13, w2, a).sum().backward()
    assert bool((a.grad == 1).all())
    # a leaf used twice
    w = w2.clone().requires_grad_()
    (moe.moe_ffn(x, w13, w) + moe.moe_ffn(x, w13, w)).sum().backward()
    v = w2.clone().requires_grad_()
    moe.moe_ffn(x, w13, v).sum().backward()
    assert torch.equal(w.grad, v.grad + v.grad)


@pytest.mark.parametrize("T,H,I", [(5, 72, 40), (200, 136, 264), (700, 264, 392), (2400, 136, 4104)])
def test_ffn_backward_strides_and_rows_behind(moe, T, H, I):
    """dout, x and dx with rows of their own strides; what lies between and
    behind the rows of dx stays."""
    g = gen(T + H)
    dout, x, gu = rnd(g, T + 1, H + 24), rnd(g, T + 2, H + 8), rnd(g, T, 2 * I)
    w13, w2 = weight(g, 2 * I, H), weight(g, H, I)
    dx = torch.full((T + 3, H + 40), 5.0, dtype=BF, device="cuda")
    got = moe.moe_ffn_backward(cuda(dout)[1:, 8:8 + H], cuda(x)[2:, :H], cuda(gu), cuda(w13), cuda(w2),
                               dx=dx[1:1 + T, 16:16 + H])
    plain = moe.moe_ffn_backward(cuda(dout[1:, 8:8 + H].contiguous()), cuda(x[2:, :H].contiguous()), cuda(gu),
                                 cuda(w13), cuda(w2))
    assert all(torch.equal(a, b) for a, b in zip(got, plain))
    want, steps = ref.ffn_backward(*(t.double() for t in (dout[1:, 8:8 + H], x[2:, :H], gu, w13, w2)))
    for name, a, b, st in zip(("dx", "dw13", "dw2"), got, want, steps):
        ref.check(a, b, B8, rms=ref.FLIPS, absolute=st, what=name, norm=ref.NORM)
    dx[1:1 + T, 16:16 + H] = 5.0
    assert bool((dx == 5).all())


# -------------------------------------------- tiles of 256 x 256 (160 of them)
@pytest.mark.parametrize("T,K,N", [(2400, 192, 4104), (2561, 72, 4096)])
def test_linear_large_tiles(moe, T, K, N):
    g = gen(T + K + N)
    xb, w = rnd(g, T, K + 8), weight(g, N, K)
    x = xb[:, 8:]
    want = x.double() @ w.double().t()
    tol = sum_tol(x.double(), w.double())
    out = torch.full((T + 1, N + 8), 5.0, dtype=F32, device="cuda")
    moe.moe_lora_linear(cuda(xb)[:, 8:], cuda(w), out=out[:T, :N])
    assert bool(((out[:T, :N].double().cpu() - want).abs() <= tol).all())
    assert bool((out[T:] == 5).all()) and bool((out[:, N:] == 5).all())
    assert torch.equal(moe.moe_lora_linear(cuda(x.contiguous()), cuda(w)), out[:T, :N].bfloat16())


# gate_up, down, and both in large tiles
@pytest.mark.parametrize("T,H,I", [(2400, 136, 2056), (2400, 4104, 72), (2561, 4096, 2048)])
def test_ffn_forward_large_tiles(moe, T, H, I):
    g = gen(T + H + I)
    x, w13, w2, add = rnd(g, T, H), weight(g, 2 * I, H), weight(g, H, I), rnd(g, T, H)
    want, gu, h = ref.ffn(x.double(), w13.double(), w2.double(), add.double())
    got, saved = moe.moe_ffn_forward(cuda(x), cuda(w13), cuda(w2), addend=cuda(add), save_gate_up=True)
    ref.check(saved, gu, B8, rms=1e-4, what="gate_up")
    ref.check(got, want, B8, rms=ref.FLIPS, absolute=ref.step_tol(h, w2.double()), what="out", norm=ref.NORM)
    assert torch.equal(moe.moe_ffn_forward(cuda(x), cuda(w13), cuda(w2), addend=cuda(add)), got)


@pytest.mark.parametrize("T,H,I", [(2400, 160, 2080), (2400, 4128, 160), (2561, 4096, 2048), (3, 64, 96), (40, 96, 160),
                                   (130, 544, 288)])
def test_ffn_mxfp8_large_tiles_and_strides(moe, T, H, I):
    g = gen(T + H + I)
    mats = []
    for n, k, s in ((T, H, 1.0), (2 * I, H, 1 / math.sqrt(H)), (H, I, 1 / math.sqrt(I))):
        q, sc = ref.mx_quant(rnd(g, n, k, scale=s).double())
        mats += [q.float().to(torch.float8_e4m3fn), sc.float().to(torch.float8_e8m0fnu)]
    add = rnd(g, T + 1, H + 16)
    x, w13, w2 = (ref.mx_wide(mats[i].float(), mats[i + 1].float()) for i in (0, 2, 4))
    gu = x @ w13.t()
    h = ref.mx_wide(*ref.mx_quant(ref.silu(gu[:, :I]) * gu[:, I:]))
    want = h @ w2.t() + add[1:, 8:8 + H].double()
    out = torch.full((T + 2, H + 24), 5.0, dtype=BF, device="cuda")
    moe.moe_ffn_forward_mxfp8(*(cuda(m) for m in mats), addend=cuda(add)[1:, 8:8 + H], out=out[1:1 + T, 16:16 + H])
    ref.check(out[1:1 + T, 16:16 + H], want, B8, rms=ref.MXFLIPS, absolute=ref.step_tol(h, w2, 2.0 ** -3), what="out",
              norm=ref.MXNORM)
    out[1:1 + T, 16:16 + H] = 5.0
    assert bool((out == 5).all())


# dh in large tiles; all of the backward; dx alone in more 128 x 128 tiles than compute units
@pytest.mark.parametrize("T,H,I,need", [(2400, 136, 4104, (True, True, True)), (2561, 1032, 4096, (True, True, True)),
                                        (129, 16512, 256, (True, True, False))])
def test_ffn_backward_large_tiles(moe, T, H, I, need):
    g = gen(T + H + I)
    dout, x, gu = rnd(g, T, H), rnd(g, T, H), rnd(g, T, 2 * I)
    w13, w2 = weight(g, 2 * I, H), weight(g, H, I)
    want, steps = ref.ffn_backward(*(t.double() for t in (dout, x, gu, w13, w2)))
    got = moe.moe_ffn_backward(*(cuda(t) for t in (dout, x, gu, w13, w2)), *need)
    for name, a, b, st, on in zip(("dx", "dw13", "dw2"), got, want, steps, need):
        assert (a is not None) == on
        if on:
            ref.check(a, b, B8, rms=ref.FLIPS, absolute=st, what=name, norm=ref.NORM)


# ------------------------------------------------------------- a block
def _experts(moe, H, I, E, seed):
    g = gen(seed)
    def u8(*s, lo=0, hi=256):
        return torch.randint(lo, hi, s, generator=g, dtype=torch.int32).to(torch.uint8).cuda()
    return (u8(E, 2 * I, H // 2), u8(E, 2 * I, H // 32, lo=118, hi=124), u8(E, H, I // 2),
            u8(E, H, I // 32, lo=118, hi=124))


@pytest.mark.parametrize("T", [1, 5, 70])
@pytest.mark.parametrize("shared", ["none", "bf16", "lora", "mxfp8"])
def test_block(moe, T, shared):
    """norm -> router -> routed experts + shared expert, against the steps."""
    H, I, E, k = 256, 128, 8, 2
    g = gen(T)
    x, res, nw = cuda(rnd(g, T, H)), cuda(rnd(g, T, H, dtype=F32)), cuda(rnd(g, H))
    rw = cuda(weight(g, E, H))
    ex = _experts(moe, H, I, E, T)
    w13, w2 = weight(g, 2 * I, H), weight(g, H, I)
    kw = {}
    if shared in ("bf16", "lora"):
        kw["shared"] = (cuda(w13), cuda(w2))
    if shared == "lora":
        kw["lora13"], kw["lora2"] = cuda(adapters(g, T, H, 2 * I, 3, 16)), cuda(adapters(g, T, I, H, 3, 8))
    if shared == "mxfp8":
        mx = []
        for m in (w13, w2):
            q, s = ref.mx_quant(m.double())
            mx += [cuda(q.float().to(torch.float8_e4m3fn)), cuda(s.float().to(torch.float8_e8m0fnu))]
        kw["shared_mxfp8"] = tuple(mx)
    out, new_res = moe.moe_a16w4_block(x, nw, rw, *ex, k, residual=res, eps=1e-5, **kw)
    y, ro, q, qs = moe.moe_rms_norm(x, nw, residual=res, eps=1e-5, mxfp8=True)
    s, v = ref.norm(x.double().cpu(), res.double().cpu(), nw.double().cpu(), 1e-5, 0.0)
    ref.check(y, v, B8 * 1.01, what="y")
    assert torch.equal(new_res, ro)
    logits = moe.moe_lora_linear(y, rw, out_dtype=F32)
    routed = moe.moe_a16w4_layer(y, logits, *ex, k)
    if shared == "none":
        assert torch.equal(out, routed)
        return
    yd, rd = y.double().cpu(), routed.double().cpu()
    if shared == "mxfp8":
        gu = ref.mx_wide(q.double().cpu(), qs.double().cpu()) @ ref.mx_wide(mx[0].double().cpu(), mx[1].double().cpu()).t()
        h = ref.mx_wide(*ref.mx_quant(ref.silu(gu[:, :I]) * gu[:, I:]))
        wide2 = ref.mx_wide(mx[2].double().cpu(), mx[3].double().cpu())
        ref.check(out, h @ wide2.t() + rd, B8, rms=ref.MXFLIPS, absolute=ref.step_tol(h, wide2, 2.0 ** -3), what="out")
    else:
        want, _, h = ref.ffn(yd, w13.double(), w2.double(), rd, kw.get("lora13"), kw.get("lora2"))
        ref.check(out, want, B8, rms=ref.FLIPS, absolute=ref.step_tol(h, w2.double()), what="out")


@pytest.mark.parametrize("T", [1, 5, 70])
@pytest.mark.parametrize("E,k", [(1, 1), (4, 2), (130, 3), (300, 6)])
def test_block_any_number_of_experts(moe, T, E, k):
    """The router takes every E that the routed layer takes, with its weights
    as they are or already padded to eights."""
    H, I = 256, 128
    g = gen(T + E)
    x, res, nw = cuda(rnd(g, T, H)), cuda(rnd(g, T, H)), cuda(rnd(g, H))
    rw, ex = weight(g, E, H), _experts(moe, H, I, E, T)
    sh = (cuda(weight(g, 2 * I, H)), cuda(weight(g, H, I)))
    out, new_res = moe.moe_a16w4_block(x, nw, cuda(rw), *ex, k, residual=res, shared=sh)
    y, ro, _, _ = moe.moe_rms_norm(x, nw, residual=res)
    padded = torch.full(((E + 7) // 8 * 8, H), math.nan, dtype=BF)
    padded[:E] = rw
    logits = moe.moe_lora_linear(y, cuda(padded), out_dtype=F32)[:, :E].contiguous()
    yd, wd = y.double().cpu(), rw.double()
    assert bool(((logits.double().cpu() - yd @ wd.t()).abs() <= sum_tol(yd, wd)).all())
    want = moe.moe_ffn_forward(y, *sh, addend=moe.moe_a16w4_layer(y, logits, *ex, k))
    assert torch.equal(out, want) and torch.equal(new_res, ro)
    again, _ = moe.moe_a16w4_block(x, nw, cuda(padded), *ex, k, residual=res, shared=sh)
    assert torch.equal(again, want)


def test_block_refuses_a_router_of_other_experts(moe):
    H, I, E, T = 256, 128, 12, 3
    x, nw = cuda(rnd(gen(1), T, H)), cuda(rnd(gen(2), H))
    ex = _experts(moe, H, I, E, T)
    for rows in (8, 11, 13, 24):
        with pytest.raises(ValueError, match="router_w"):
            moe.moe_a16w4_block(x, nw, cuda(weight(gen(3), rows, H)), *ex, 2)


@pytest.mark.parametrize("T", [1, 5, 70])
def test_block_biases_and_limit(moe, T):
    H, I, E, k = 256, 128, 8, 2
    g = gen(T)
    x, nw, rw, ex = cuda(rnd(g, T, H)), cuda(rnd(g, H)), cuda(weight(g, E, H)), _experts(moe, H, I, E, T)
    sh = (cuda(weight(g, 2 * I, H)), cuda(weight(g, H, I)))
    kw = dict(w13_bias=cuda(rnd(g, E, 2 * I)), w2_bias=cuda(rnd(g, E, H)), swiglu_limit=1.5)
    out, _ = moe.moe_a16w4_block(x, nw, rw, *ex, k, shared=sh, **kw)
    y = moe.moe_rms_norm(x, nw)[0]
    logits = moe.moe_lora_linear(y, rw, out_dtype=F32)
    assert torch.equal(out, moe.moe_ffn_forward(y, *sh, addend=moe.moe_a16w4_layer(y, logits, *ex, k, **kw)))
    for name in kw:  # each of them takes part
        other, _ = moe.moe_a16w4_block(x, nw, rw, *ex, k, shared=sh, **{n: v for n, v in kw.items() if n != name})
        assert not torch.equal(other, out)


def test_block_of_no_tokens(moe):
    H, I, E = 256, 128, 5
    x, res, nw = (torch.empty(0, H, dtype=BF, device="cuda") for _ in range(3))
    nw = torch.ones(H, dtype=BF, device="cuda")
    ex = _experts(moe, H, I, E, 1)
    sh = tuple(torch.ones(s, dtype=BF, device="cuda") for s in ((2 * I, H), (H, I)))
    out, new_res = moe.moe_a16w4_block(x, nw, torch.ones(E, H, dtype=BF, device="cuda"), *ex, 2, residual=res, shared=sh)
    assert out.shape == (0, H) and new_res.shape == (0, H)


# --------------------------------------------------- the ends of the ranges
@pytest.mark.parametrize("T", [0, 3, 70])
def test_linear_weights_above_2_gib(moe, T):
    """Rows that 32-bit byte offsets from the first do not reach."""
    K, N = 8192, 152064
    dev = torch.Generator(device="cuda").manual_seed(T)
    w = torch.empty(N, K, dtype=BF, device="cuda").normal_(0, 1 / math.sqrt(K), generator=dev)
    x = torch.randn(T, K, generator=dev, device="cuda").bfloat16()
    got = moe.moe_lora_linear(x, w, out_dtype=F32)
    assert got.shape == (T, N)
    for rows in (slice(0, 40), slice(131040, 131110), slice(N - 40, N)):  # 131072 rows are 2 GiB
        xd, wd = x.double().cpu(), w[rows].double().cpu()
        assert bool(((got[:, rows].double().cpu() - xd @ wd.t()).abs() <= sum_tol(xd, wd)).all())


@pytest.mark.parametrize("n", [0, 5])
def test_linear_tokens_above_2_gib(moe, n):
    T, K, N = 140001, 8192, 72
    dev = torch.Generator(device="cuda").manual_seed(n)
    x = torch.empty(T, K, dtype=BF, device="cuda").normal_(0, 1, generator=dev)
    w = weight(gen(1), N, K)
    lo = adapters(gen(2), T, K, N, n, 16, ranks=False) if n else None
    got = moe.moe_lora_linear(x, cuda(w), lora=cuda(lo), out_dtype=F32)
    for rows in (slice(0, 40), slice(131040, 131110), slice(T - 40, T)):
        xd, wd = x[rows].double().cpu(), w.double()
        want, tol = xd @ wd.t(), sum_tol(xd, wd)
        if n:
            part = (lo[0], lo[1], lo[2][rows], None, lo[4])
            want += ref.lora(xd, part)
            tol += ref.lora(xd.abs(), (lo[0].double().abs(), lo[1].double().abs(), *part[2:])) * (2.0 ** -16 + (K / 8 + 128) * F24)
        assert bool(((got[rows].double().cpu() - want).abs() <= tol).all())


def test_norm_above_4_gib(moe):
    T, H = 530001, 4128
    x = torch.empty(T, H, dtype=BF, device="cuda").normal_(0, 1, generator=torch.Generator(device="cuda").manual_seed(1))
    w = rnd(gen(1), H)
    y, _, q, qs = moe.moe_rms_norm(x, cuda(w), mxfp8=True)
    for rows in (slice(0, 3), slice(260110, 260120), slice(520220, 520230), slice(T - 3, T)):  # of 2 and 4 GiB
        _, v = ref.norm(x[rows].double().cpu(), None, w.double(), 1e-6, 0.0)
        ref.check(y[rows], v, B8 * 1.01, what="y")
        want, scale = ref.mx_quant(v)
        assert torch.equal(qs[rows].double().cpu(), scale) and torch.equal(q[rows].double().cpu(), want)


@pytest.mark.parametrize("T,K,N", [(1, 72, 40), (5, 1032, 264), (40, 1032, 264), (70, 72, 2056), (200, 1032, 264), (300, 264, 4104),
                                   (700, 264, 520)])
def test_linear_adapters_of_the_largest_rank(moe, T, K, N):
    g = gen(T + K + N)
    n, rank = 4, 256
    x, w = rnd(g, T, K), weight(g, N, K)
    lo = adapters(g, T, K, N, n, rank)
    lo[3][0], lo[3][1] = 256, 255
    for i in range(n):
        lo[0][i, int(lo[3][i]):] = math.nan
        lo[1][i, :, int(lo[3][i]):] = math.inf
    xd = x.double()
    want = xd @ w.double().t() + ref.lora(xd, lo)
    wide = tuple(t if t is None or not t.is_floating_point() else torch.nan_to_num(t.double(), 0, 0, 0).abs() for t in lo)
    tol = sum_tol(xd, w.double()) + ref.lora(xd.abs(), wide) * (2.0 ** -16 + (K / 8 + 256) * F24)
    got = moe.moe_lora_linear(cuda(x), cuda(w), lora=cuda(lo), out_dtype=F32)
    assert bool(((got.double().cpu() - want).abs() <= tol).all())


# ---------------------------------------------- streams, graphs, two at once
def test_block_in_a_graph(moe):
    """Captured once and replayed, with new inputs and eager work between the
    replays; a second graph has its own workspaces."""
    H, I, E, k, T = 256, 128, 8, 2, 70
    g = gen(1)
    nw, rw, ex = cuda(rnd(g, H)), cuda(weight(g, E, H)), _experts(moe, H, I, E, 1)
    sh = (cuda(weight(g, 2 * I, H)), cuda(weight(g, H, I)))
    lo = cuda(adapters(g, T, H, 2 * I, 3, 16))

    def step(x, res):
        return moe.moe_a16w4_block(x, nw, rw, *ex, k, residual=res, shared=sh, lora13=lo)

    xs = [cuda(rnd(g, T, H)) for _ in range(4)]
    rs = [cuda(rnd(g, T, H, dtype=F32)) for _ in range(4)]
    want = [step(x, r) for x, r in zip(xs, rs)]
    graphs = []
    for _ in range(2):
        x, r = xs[0].clone(), rs[0].clone()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step(x, r)
        torch.cuda.current_stream().wait_stream(side)
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            o = step(x, r)
        graphs.append((gr, x, r, o))
    for i in (1, 2, 3, 0):
        for gr, x, r, o in graphs:
            x.copy_(xs[i])
            r.copy_(rs[i])
            gr.replay()
        again = step(xs[i], rs[i])
        torch.cuda.synchronize()
        for _, _, _, o in graphs:
            assert torch.equal(o[0], want[i][0]) and torch.equal(o[1], want[i][1])
        assert torch.equal(again[0], want[i][0])


def test_backward_in_a_graph(moe):
    g = gen(2)
    T, H, I = 130, 136, 264
    dout, x, gu = cuda(rnd(g, T, H)), cuda(rnd(g, T, H)), cuda(rnd(g, T, 2 * I))
    w13, w2 = cuda(weight(g, 2 * I, H)), cuda(weight(g, H, I))
    ws = torch.empty(moe.moe_ffn_backward_workspace_size(T, H, I), dtype=torch.uint8, device="cuda")
    moe.moe_ffn_backward(dout, x, gu, w13, w2, workspace=ws)
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        o = moe.moe_ffn_backward(dout, x, gu, w13, w2, workspace=ws)
    for k in range(3):
        dout.copy_(cuda(rnd(g, T, H)))
        ws.fill_(k * 85)
        gr.replay()
        torch.cuda.synchronize()
        want = moe.moe_ffn_backward(dout, x, gu, w13, w2)
        assert all(torch.equal(a, b) for a, b in zip(o, want))


def test_gradients_in_a_graph(moe):
    """Forward and gradients of the differentiable form captured together."""
    g = gen(4)
    T, H, I = 130, 136, 264
    x, probe = cuda(rnd(g, T, H)).requires_grad_(), cuda(rnd(g, T, H))
    w13, w2 = cuda(weight(g, 2 * I, H)).requires_grad_(), cuda(weight(g, H, I)).requires_grad_()

    def step():
        out = moe.moe_ffn(x, w13, w2)
        return (out.detach(), *torch.autograd.grad(out, (x, w13, w2), probe))

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
            probe.copy_(cuda(rnd(g, T, H)))
        gr.replay()
        torch.cuda.synchronize()
        want = step()
        assert all(torch.equal(a, b) for a, b in zip(o, want))


def test_two_streams_at_once(moe):
    g = gen(5)
    T, H, I = 300, 264, 392
    x = [cuda(rnd(g, T, H)) for _ in range(2)]
    w13, w2 = cuda(weight(g, 2 * I, H)), cuda(weight(g, H, I))
    lo = [cuda(adapters(g, T, H, 2 * I, 4, 16)) for _ in range(2)]
    want = [moe.moe_ffn_forward(x[i], w13, w2, lora13=lo[i]) for i in range(2)]
    torch.cuda.synchronize()
    st = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(8):
        for i in range(2):
            got[i].append(moe.moe_ffn_forward(x[i], w13, w2, lora13=lo[i], stream=st[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(t, want[i]) for t in got[i])
