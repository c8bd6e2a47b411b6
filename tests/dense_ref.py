"""Plain fp64 forms of the dense operators (CPU), and how far a kernel may be
from them.

Tolerances, from the arithmetic:
  * one rounding to a type is off by at most eps / 2 of the value (bf16 2^-8,
    fp32 2^-24, e4m3 2^-4 or half of its smallest step, 2^-10 of the scale);
  * an fp32 sum of n products in any order of depth d is off by at most
    d 2^-24 sum |a b|; the kernels add at most K / 8 + 64 terms in a row;
  * a value that is rounded to bf16 on the way (h, dgate, dup) is rounded in
    the reference too. Where the fp32 sum before it differs from the exact one
    by about 1e-6 of it, about 1e-6 / 2^-8 = 3e-4 of the values fall to the
    other side of a tie, by one step, 2^-7 of the value. A result sums them
    with a factor: in the 2-norm sqrt(3e-4) * 2^-7 = 1.3e-4 (FLIPS leaves a
    factor of 15 for small sizes); one result's largest single step is at most
    2^-7 max|values| max|factors| over its row and column (step_tol), and a
    row of a few hundred to 2,000 values has less than one on average;
  * the matrix core adds eight e4m3 products with about 2^-14 of the largest
    lost (measured: 1.3e-5 of a sum): about 1.3e-5 / 2^-4 = 2e-4 of h fall to
    the other side of an e4m3 tie, by one step of at most 2^-3: in the 2-norm
    1.8e-3, singly at most 2^-3 max|h| max|w2| (step_tol).
"""
import torch

FLIPS = 2e-3
MXFLIPS = 1.2e-2


def step_tol(values, factors, step=2.0 ** -7):
    """One rounding step of the largest value of each row, times the largest
    factor of each column: values [m, k], factors [n, k] -> [m, n]."""
    return step * values.abs().amax(1, keepdim=True) * factors.abs().amax(1)


def bf16(v):
    return v.float().bfloat16().double()


def silu(g):
    return g / (1 + torch.exp(-g))


def mx_scale(v):
    """fp64 [..., n] -> the power-of-two scale of each 32."""
    b = v.unflatten(-1, (-1, 32)).abs()
    amax = torch.where(torch.isfinite(b), b, torch.zeros_like(b)).amax(-1)
    m, e = torch.frexp(amax)
    e = (e - 9 + (m > 0.875).to(e.dtype)).clamp(-127, 127)
    e = torch.where(amax == 0, torch.full_like(e, -127), e)
    return torch.ldexp(torch.ones_like(amax), e)


def mx_round(z):
    """fp64 within [-448, 448] -> the nearest e4m3 value, ties to even."""
    k = torch.frexp(z.abs().clamp_min(2.0 ** -6))[1] - 1
    step = torch.ldexp(torch.ones_like(z), k - 3)
    return torch.round(z / step) * step


def mx_quant(v):
    s = mx_scale(v)
    return mx_round(v.unflatten(-1, (-1, 32)) / s.unsqueeze(-1)).flatten(-2), s


def mx_wide(q, s):
    return (q.double().unflatten(-1, (-1, 32)) * s.double().unsqueeze(-1)).flatten(-2)


def lora(x, lo):
    """fp64 x [T, K] -> the adapters' term [T, N], token by token's adapter."""
    a, b, index, ranks, scale = (None if t is None else t.cpu() for t in tuple(lo))
    out = torch.zeros(x.shape[0], b.shape[1], dtype=torch.float64)
    for i in range(a.shape[0]):
        rows = (index == i).nonzero().squeeze(1)
        r = a.shape[1] if ranks is None else min(max(int(ranks[i]), 0), a.shape[1])
        if len(rows) and r:
            s = 1.0 if scale is None else float(scale[i])
            out[rows] = s * ((x[rows] @ a[i, :r].double().t()) @ b[i, :, :r].double().t())
    return out


def norm(x, residual, weight, eps, offset):
    s = x if residual is None else x + residual
    return s, s / torch.sqrt((s * s).mean(-1, keepdim=True) + eps) * (offset + weight)


def ffn(x, w13, w2, addend=None, lora13=None, lora2=None):
    """-> (out, gate_up, h), fp64, with h rounded to bf16."""
    gu = x @ w13.t()
    if lora13 is not None:
        gu = gu + lora(x, lora13)
    I = w2.shape[1]
    h = bf16(silu(gu[:, :I]) * gu[:, I:])
    out = h @ w2.t()
    if lora2 is not None:
        out = out + lora(h, lora2)
    return (out if addend is None else out + addend), gu, h


def ffn_backward(dout, x, gate_up, w13, w2):
    """-> (dx, dw13, dw2), fp64, with h, dgate and dup rounded to bf16, and
    their step tolerances."""
    I = w2.shape[1]
    g, u = gate_up[:, :I], gate_up[:, I:]
    s = torch.sigmoid(g)
    dh = dout @ w2
    d = bf16(torch.cat([dh * u * s * (1 + g * (1 - s)), dh * g * s], 1))
    h = bf16(g * s * u)
    return ((d @ w13, d.t() @ x, dout.t() @ h),
            (step_tol(d, w13.t()), step_tol(d.t(), x.t()), step_tol(h.t(), dout.t()).t()))


def check(got, ref, rel, rms=0.0, absolute=0.0, what="", norm=None):
    """|got - ref| <= rel |ref| + rms RMS(ref) + absolute, element by element,
    and (norm, results of 1,000 values or more) ||got - ref|| <= norm ||ref||."""
    got = got.detach().double().cpu()
    assert got.shape == ref.shape, f"{what}: shape {tuple(got.shape)}, expected {tuple(ref.shape)}"
    if not ref.numel():
        return
    assert bool(torch.isfinite(got).all()), f"{what}: not finite"
    scale = float(ref.square().mean().sqrt())
    over = (got - ref).abs() - (rel * ref.abs() + rms * scale + absolute)
    worst = float(over.max())
    assert worst <= 0, f"{what}: {worst:.3g} over the tolerance (RMS {scale:.3g}) at {int(over.argmax())}"
    if norm is not None and ref.numel() >= 1000:
        far = float((got - ref).norm() / ref.norm())
        assert far <= norm, f"{what}: {far:.3g} of the norm off, {norm:.3g} allowed"


# 2-norms: bf16 rounding is uniform over at most half a step, 2^-8 / sqrt(3) =
# 2.3e-3 where every value sits right above a power of two, and the flips.
NORM = 2.5e-3
MXNORM = 4e-3
