"""Plain fp64 forms of the operators of a trainable expert block (CPU), and how
far a kernel may be from them.

Tolerances, from the arithmetic (F = 2^-24, half a step of fp32):
  * layer norm: the mean and the variance are fp64 sums of s, which is rounded
    to fp32 once (F |s|); what follows is the difference, two products and a
    sum, F each. Normed values are off by 8 F |n w| + 2 F |v| + 2 F |s| r |w|,
    r the row's 1 / deviation;
  * its backward: n is off by 3 F |n| + F |s| r, the row's sums have at most 90
    (rows above 16384 columns: 8 a step of 8192) terms in a row; a column's sum has
    at most T / parts + 70: a workgroup's rows, its four waves, and a join of 128
    runs by halves. Few rows: runs of T / 32 at least, and half as many as the runs
    (128 of more than 8192 columns) behind each other;
  * hardware exp2 and reciprocal are off by about an ulp, 2 F, each; an exponent
    u, itself rounded, by |u| F more (a few of them: 4). So act(z) and act'(z)
    are off by (|u| + 8) 4 F of z p(u) for the sigmoid forms. Phi(-|z|) is off
    by 9e-7 of itself from the fit, by z^2 F from its exponent and 20 F else;
  * a value rounded to bf16 on the way (dz): as in dense_ref.
"""
import math

import torch

F = 2.0 ** -24


def layer_norm(x, residual, weight, bias, eps):
    """fp64 -> (s, y, mean, rstd)."""
    s = x if residual is None else x + residual
    mean = s.mean(1, keepdim=True)
    d = s - mean
    rstd = 1 / torch.sqrt(d.square().mean(1, keepdim=True) + eps)
    y = d * rstd * weight
    return s, y if bias is None else y + bias, mean.squeeze(1), rstd.squeeze(1)


def layer_norm_tol(s, mean, rstd, weight, y):
    r = rstd.unsqueeze(1)
    n = ((s - mean.unsqueeze(1)) * r).abs()
    return 8 * F * n * weight.abs() + 2 * F * y.abs() + 2 * F * (s.abs() + s.abs().mean(1, keepdim=True)) * r * weight.abs()


def layer_norm_backward(dy, s, mean, rstd, weight, dres=None):
    """fp64 -> (ds, dweight, dbias) and their tolerances before the outputs'
    rounding."""
    T, H = s.shape
    r = rstd.unsqueeze(1)
    n = (s - mean.unsqueeze(1)) * r
    g = dy * weight
    mg, mgn = g.mean(1, keepdim=True), (g * n).mean(1, keepdim=True)
    ds = r * (g - mg - n * mgn)
    dn = 3 * F * n.abs() + F * (s.abs() + mean.abs().unsqueeze(1)) * r
    depth = 90 + 8 * (H // 8192) * (H > 16384)
    eg = depth * F * g.abs().mean(1, keepdim=True)
    egn = depth * F * (g * n).abs().mean(1, keepdim=True) + (g.abs() * dn).mean(1, keepdim=True)
    tol = r * (6 * F * (g.abs() + mg.abs() + (n * mgn).abs()) + eg + n.abs() * egn + dn * mgn.abs())
    if dres is not None:
        ds = ds + dres
        tol = tol + 2 * F * (ds.abs() + dres.abs())
    parts = 4096 if H <= 512 else 1024 if H <= 2048 else 512 if H <= 4096 else 256 if H <= 8192 else 64
    terms = T / parts + (132 if H > 8192 else 74)
    tw = terms * F * (dy * n).abs().sum(0) + (dy.abs() * dn).sum(0)
    return (ds, (dy * n).sum(0), dy.sum(0)), (tol, tw, terms * F * dy.abs().sum(0))


def permute(x, ids, E):
    """-> (out, rows, offsets) by loops over the experts."""
    T, k = ids.shape
    flat = ids.flatten().tolist()
    out = torch.zeros(T * k, x.shape[1], dtype=x.dtype)
    rows, offsets, at = [0] * (T * k), [0], 0
    by = [[] for _ in range(E + 1)]
    for p, e in enumerate(flat):
        by[e if 0 <= e < E else E].append(p)
    for e in range(E + 1):
        for p in by[e]:
            if e < E:
                out[at] = x[p // k]
            rows[p] = at if e < E else -1 - at
            at += 1
        if e < E:
            offsets.append(at)
    return out, torch.tensor(rows, dtype=torch.int32).view(T, k), torch.tensor(offsets, dtype=torch.int32)


def unpermute(y, rows, weights, residual):
    """fp64 -> (out, the sum of magnitudes)."""
    T, k = rows.shape
    out = torch.zeros(T, y.shape[1], dtype=torch.float64) if residual is None else residual.clone()
    size = out.abs()
    for j in range(k):
        t = (rows[:, j] >= 0).nonzero().squeeze(1)
        v = y[rows[t, j].long()] * (1.0 if weights is None else weights[t, j, None])
        out[t] += v
        size[t] += v.abs()
    return out, size


def unpermute_backward(dout, rows, y, weights):
    """fp64 -> (dy, dweights, the dot products' sums of magnitudes)."""
    T, k = rows.shape
    dy = torch.zeros(T * k, dout.shape[1], dtype=torch.float64)
    dw = torch.zeros(T, k, dtype=torch.float64)
    size = torch.zeros(T, k, dtype=torch.float64)
    for j in range(k):
        t = (rows[:, j] >= 0).nonzero().squeeze(1)
        r = rows[t, j].long()
        dy[r] = dout[t] * (1.0 if weights is None else weights[t, j, None])
        if y is not None:
            dw[t, j] = (dout[t] * y[r]).sum(1)
            size[t, j] = (dout[t] * y[r]).abs().sum(1)
    return dy, dw, size


NONE, RELU, SILU, GELU, GELU_TANH = range(5)
C = math.sqrt(2 / math.pi)


def _u(act, z):
    """The sigmoid forms' exponent and its slope."""
    if act == SILU:
        return z, torch.ones_like(z)
    return 2 * C * (z + 0.044715 * z ** 3), 2 * C * (1 + 3 * 0.044715 * z ** 2)


def act(a, z):
    """fp64 z -> (act(z), tolerance)."""
    if a == NONE:
        return z, torch.zeros_like(z)
    if a == RELU:
        return z.clamp_min(0), torch.zeros_like(z)
    if a == GELU:
        tail = torch.special.ndtr(-z.abs())
        return z * torch.special.ndtr(z), z.abs() * tail * (9e-7 + (z * z + 20) * F) + 2 * F * z.abs()
    u, _ = _u(a, z)
    v = z * torch.sigmoid(u)
    return v, v.abs() * (u.abs().clamp_max(200) + 8) * 4 * F


def slope(a, z):
    """fp64 z -> (act'(z), tolerance)."""
    one = torch.ones_like(z)
    if a == NONE:
        return one, 0 * z
    if a == RELU:
        return (z > 0).double(), 0 * z
    if a == GELU:
        tail, phi = torch.special.ndtr(-z.abs()), z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
        v = torch.special.ndtr(z) + phi
        return v, tail * (9e-7 + (z * z + 20) * F) + phi.abs() * (z * z + 20) * F + 4 * F * v.abs()
    u, du = _u(a, z)
    p = torch.sigmoid(u)
    q = z * p * (1 - p) * du
    return p + q, (p + 2 * q.abs()) * (u.abs().clamp_max(200) + 8) * 4 * F


def slope_of_act(a, z):
    """Largest slope on the way (a tolerance of z becomes one of act(z))."""
    return 1.2 if a not in (NONE, RELU) else 1.0
