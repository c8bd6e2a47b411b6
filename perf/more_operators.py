"""Cases that measure the operators of a trainable expert block: layer norm
with its backward pass, tokens sorted by expert and back with their gradients,
and the product with bias, activation and addend with its backward pass.

`own` selects between the plain torch form of each operator and the calls a
user makes of this package.
"""
import math

import torch

own = False

# Kinds of a case:
#   norm       residual addition + layer norm; res: the residual's type ("" none);
#              save: mean and 1 / deviation of each row are outputs (training)
#   norm_bwd   its backward; res: type of the stream that was normed ("" bf16
#              without a gradient from the stream)
#   permute    rows sorted by expert; type: bf16, f32 or u8 (codes of an 8-bit
#              dispatch); absent: share of pairs whose expert is elsewhere
#   combine    rows back to tokens with router weights and a residual of `out` type
#   combine_bwd  gradients of the rows and of the router weights
#   linear     act(x W^T + bias) + addend; save: the activation's argument is an
#              output; f32: fp32 output and addend
#   linear_bwd gradients of x, W and bias
EPS = 1e-5
ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")


def listed():
    return [
        # one token of one request: latency of a block's first step
        dict(name="norm_token", kind="norm", T=1, H=3584, res="bf16", save=False),
        # an odd chunk of training sequences in a model with an fp32 residual stream and an odd width
        dict(name="norm_odd_save", kind="norm", T=1531, H=2793, res="f32", save=True),
        # backward over a short odd batch of a small model, fp32 stream
        dict(name="norm_bwd_odd", kind="norm_bwd", T=777, H=1001, res="f32"),
        # backward over a full batch of sequences
        dict(name="norm_bwd_train", kind="norm_bwd", T=16384, H=3584, res="bf16"),
        # a decode batch dispatched to many experts
        dict(name="permute_decode", kind="permute", T=16, H=3584, topk=15, E=112, type="bf16", absent=0.0),
        # a prefill batch dispatched to very many experts, part of which live on other ranks
        dict(name="permute_prompt", kind="permute", T=8192, H=3584, topk=8, E=896, type="bf16", absent=0.125),
        # a prefill batch's rows back into an fp32 residual stream
        dict(name="combine_prompt", kind="combine", T=8192, H=3584, topk=15, E=112, type="bf16", out="f32"),
        # backward of the way back, ragged batch
        dict(name="combine_bwd_ragged", kind="combine_bwd", T=4099, H=2784, topk=4, E=64, type="bf16", out="bf16"),
        # one token through a biased projection with GELU
        dict(name="linear_token", kind="linear", T=1, K=3584, N=4096, act="gelu", bias32=False, addend=False, save=False, f32=False),
        # the training forward of an ungated feed-forward's first product
        dict(name="linear_train", kind="linear", T=8192, K=3584, N=8192, act="gelu", bias32=False, addend=False, save=True, f32=False),
        # backward over a short odd batch of a small block
        dict(name="linear_bwd_odd", kind="linear_bwd", T=777, K=1000, N=520, act="silu", bias32=True, f32=False),
        # backward over a full batch of sequences
        dict(name="linear_bwd_train", kind="linear_bwd", T=8192, K=3584, N=4096, act="gelu", bias32=False, f32=False),
    ]


def _log_int(rng, lo, hi, step=1):
    return max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step)


def draw(rng):
    kind = rng.choice(["norm", "norm_bwd", "permute", "combine", "combine_bwd", "linear", "linear_bwd"])
    if kind.startswith("norm"):
        H = _log_int(rng, 33, 8192)
        T = min(_log_int(rng, 1, 32768), 16384 * 3584 // H)
        c = dict(kind=kind, T=T, H=H, res=rng.choice(["", "bf16", "f32"]))
        if kind == "norm":
            c["save"] = rng.random() < 0.5
        return c
    if kind.startswith("linear"):
        K, N = _log_int(rng, 64, 8192, 8), _log_int(rng, 16, 8192, 8)
        T = min(_log_int(rng, 1, 8192), int(4.8e11 / ((4 if kind == "linear_bwd" else 2) * K * N)))
        f32 = rng.random() < 0.25
        c = dict(kind=kind, T=T, K=K, N=N, act=rng.choice(ACTS), bias32=rng.random() < 0.3, f32=f32)
        if kind == "linear":
            c.update(addend=rng.random() < 0.5, save=rng.random() < 0.3)
        return c
    E = _log_int(rng, 4, 1024)
    topk = rng.randint(1, min(15, E))
    step = 1 if rng.random() < 0.3 else 32
    H = _log_int(rng, 64, 8192, step)
    T = min(_log_int(rng, 1, 32768), 8192 * 8 * 3584 // (H * topk))
    if kind == "permute":
        return dict(kind=kind, T=T, H=H, topk=topk, E=E, type=rng.choice(["bf16", "bf16", "f32", "u8"]),
                    absent=rng.choice([0.0, 0.5]))
    return dict(kind=kind, T=T, H=H, topk=topk, E=E, type=rng.choice(["bf16", "bf16", "f32"]), out=rng.choice(["bf16", "f32"]))


_TYPES = dict(bf16=torch.bfloat16, f32=torch.float32, u8=torch.float8_e4m3fn)


# ---------------------------------------------------------------- inputs
def _routing(g, T, topk, E, absent):
    """A router's choices: distinct experts of uneven popularity and their
    renormalised weights; an absent pair's expert is -1."""
    logits = torch.randn(T, E, generator=g, device="cuda") + 0.7 * torch.randn(E, generator=g, device="cuda")
    top = logits.topk(topk, dim=1)
    ids = top.indices.to(torch.int32)
    if absent:
        ids = ids.masked_fill(torch.rand(T, topk, generator=g, device="cuda") < absent, -1)
    return ids, torch.softmax(top.values, 1)


def _rows_of(ids, E):
    """-> (rows int32 [T, topk]: each pair's place after the stable sort by
    expert, -1 - place for pairs without one, which come last; offsets int32
    [E + 1])."""
    T, topk = ids.shape
    key = ids.flatten().long()
    key = torch.where((key >= 0) & (key < E), key, torch.full_like(key, E))
    order = torch.sort(key, stable=True).indices
    place = torch.empty_like(order)
    place[order] = torch.arange(T * topk, device=ids.device)
    count = torch.zeros(E + 1, dtype=torch.long, device=ids.device).index_add_(0, key, torch.ones_like(key))
    offsets = torch.cat([torch.zeros(1, dtype=torch.long, device=ids.device), count[:E].cumsum(0)])
    rows = torch.where(key < E, place, -1 - place).view(T, topk)
    return rows.to(torch.int32), offsets.to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    dev = "cuda"
    kind, T = case["kind"], case["T"]

    def rnd(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    s = dict(case=case)
    if kind.startswith("norm"):
        H, res = case["H"], case["res"]
        s["weight"] = (1 + 0.1 * rnd(H)).bfloat16()
        s["bias"] = (0.1 * rnd(H)).bfloat16()
        # a residual stream has rows of very different size, and a mean
        stream = (rnd(T, H) + 0.3 * rnd(T, 1)) * torch.exp(rnd(T, 1))
        if kind == "norm":
            s["x"] = rnd(T, H).bfloat16()
            s["residual"] = stream.to(_TYPES[res]) if res else None
            return s
        s["s"] = stream.to(_TYPES[res or "bf16"])
        d = s["s"].double()
        mean = d.mean(1, keepdim=True)
        s["mean"] = mean.squeeze(1).float()
        s["rstd"] = torch.rsqrt((d - mean).square().mean(1) + EPS).float()
        s["dy"] = rnd(T, H).bfloat16()
        s["dres"] = rnd(T, H).to(_TYPES[res]) if res else None
        return s
    if kind.startswith("linear"):
        K, N = case["K"], case["N"]
        s["x"] = rnd(T, K).bfloat16()
        s["w"] = (rnd(N, K) / math.sqrt(K)).bfloat16()
        s["bias"] = (0.5 * rnd(N)).to(torch.float32 if case["bias32"] else torch.bfloat16)
        out = torch.float32 if case["f32"] else torch.bfloat16
        if kind == "linear":
            s["addend"] = rnd(T, N).to(out) if case["addend"] else None
        else:
            s["dout"] = rnd(T, N).to(out)
            s["pre"] = (rnd(T, N) * 1.1).bfloat16()
        return s
    H, topk, E = case["H"], case["topk"], case["E"]
    ids, weights = _routing(g, T, topk, E, case.get("absent", 0.0))
    if kind == "permute":
        s["x"] = rnd(T, H).to(_TYPES[case["type"]])
        s["ids"] = ids
        return s
    s["rows"], _ = _rows_of(ids, E)
    s["weights"] = weights
    s["y"] = rnd(T * topk, H).to(_TYPES[case["type"]])
    s["residual" if kind == "combine" else "dout"] = rnd(T, H).to(_TYPES[case["out"]])
    return s


# ---------------------------------------------------------------- plain forms
def _plain_norm(s):
    t = s["x"].float()
    if s["residual"] is not None:
        t = t + s["residual"].float()
    # rows far from zero: centred before they are squared
    mean = t.mean(1, keepdim=True)
    d = t - mean
    rstd = torch.rsqrt(d.square().mean(1, keepdim=True) + EPS)
    out = dict(y=(d * rstd * s["weight"].float() + s["bias"].float()).bfloat16())
    if s["residual"] is not None:
        out["residual"] = t.to(s["residual"].dtype)
    if s["case"]["save"]:
        out.update(mean=mean.squeeze(1), rstd=rstd.squeeze(1))
    return out


def _plain_norm_bwd(s):
    dy, t, w = s["dy"].float(), s["s"].float(), s["weight"].float()
    rstd = s["rstd"].unsqueeze(1)
    n = (t - s["mean"].unsqueeze(1)) * rstd
    g = dy * w
    ds = rstd * (g - g.mean(1, keepdim=True) - n * (g * n).mean(1, keepdim=True))
    if s["dres"] is not None:
        ds = ds + s["dres"].float()
    out = dict(dx=ds.bfloat16(), dweight=(dy * n).sum(0).bfloat16(), dbias=dy.sum(0).bfloat16())
    if s["case"]["res"] == "f32":
        out["dresidual"] = ds
    return out


def _plain_permute(s):
    c = s["case"]
    rows, offsets = _rows_of(s["ids"], c["E"])
    flat = rows.flatten().long()
    place = torch.where(flat < 0, -1 - flat, flat)
    x = s["x"].float().repeat_interleave(c["topk"], 0)
    x = torch.where((flat >= 0).unsqueeze(1), x, torch.zeros_like(x))
    out = torch.empty_like(x)
    out[place] = x
    return dict(out=out.to(s["x"].dtype), rows=rows, offsets=offsets)


def _plain_combine(s):
    rows = s["rows"].long()
    v = s["y"].float()[rows.clamp_min(0)]
    v = torch.where((rows >= 0).unsqueeze(2), v * s["weights"].unsqueeze(2), torch.zeros_like(v))
    return (v.sum(1) + s["residual"].float()).to(s["residual"].dtype)


def _plain_combine_bwd(s):
    rows, dout = s["rows"].long(), s["dout"].float()
    here = rows >= 0
    flat = torch.where(here, rows, -1 - rows).flatten()
    d = (s["weights"] * here).unsqueeze(2) * dout.unsqueeze(1)
    dy = torch.empty(flat.numel(), dout.shape[1], device=dout.device)
    dy[flat] = d.flatten(0, 1)
    dw = (s["y"].float()[rows.clamp_min(0)] * dout.unsqueeze(1)).sum(2)
    return dict(dy=dy.to(s["y"].dtype), dweights=torch.where(here, dw, torch.zeros_like(dw)))


def _act(name, z):
    if name == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if name == "silu":
        return z / (1 + torch.exp(-z))
    if name == "gelu":
        return z * 0.5 * (1 + torch.erf(z * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return z / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _slope(name, z):
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "silu":
        p = 1 / (1 + torch.exp(-z))
        return p * (1 + z * (1 - p))
    if name == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        c = 2 * math.sqrt(2 / math.pi)
        p = 1 / (1 + torch.exp(-c * (z + 0.044715 * z * z * z)))
        return p + z * p * (1 - p) * c * (1 + 3 * 0.044715 * z * z)
    return torch.ones_like(z)


def _plain_linear(s):
    c = s["case"]
    z = s["x"].float() @ s["w"].float().t() + s["bias"].float()
    out = _act(c["act"], z)
    if s["addend"] is not None:
        out = out + s["addend"].float()
    out = dict(out=out if c["f32"] else out.bfloat16())
    if c["save"]:
        out["pre"] = z.bfloat16()
    return out


def _plain_linear_bwd(s):
    dz = s["dout"].float() * _slope(s["case"]["act"], s["pre"].float())
    return dict(dx=(dz @ s["w"].float()).bfloat16(), dw=(dz.t() @ s["x"].float()).bfloat16(),
                dbias=dz.sum(0).to(s["bias"].dtype))


_PLAIN = dict(norm=_plain_norm, norm_bwd=_plain_norm_bwd, permute=_plain_permute, combine=_plain_combine,
              combine_bwd=_plain_combine_bwd, linear=_plain_linear, linear_bwd=_plain_linear_bwd)


# ---------------------------------------------------------------- one pass
def _own_run(s):
    import mxfp4_grouped_gemm_amd as moe

    c = s["case"]
    kind = c["kind"]
    if kind == "norm":
        y, res, mean, rstd = moe.moe_layer_norm_forward(s["x"], s["weight"], s["bias"], residual=s["residual"], eps=EPS,
                                                        save_stats=c["save"])
        out = dict(y=y)
        if res is not None:
            out["residual"] = res
        if c["save"]:
            out.update(mean=mean, rstd=rstd)
        return out
    if kind == "norm_bwd":
        dx, dres, dweight, dbias = moe.moe_layer_norm_backward(s["dy"], s["s"], s["mean"], s["rstd"], s["weight"],
                                                               dresidual_out=s["dres"], need_dresidual=c["res"] == "f32")
        out = dict(dx=dx, dweight=dweight, dbias=dbias)
        if dres is not None:
            out["dresidual"] = dres
        return out
    if kind == "permute":
        out, rows, offsets = moe.moe_permute(s["x"], s["ids"], c["E"])
        return dict(out=out, rows=rows, offsets=offsets)
    if kind == "combine":
        return moe.moe_unpermute(s["y"], s["rows"], weights=s["weights"], residual=s["residual"])
    if kind == "combine_bwd":
        dy, dweights = moe.moe_unpermute_backward(s["dout"], s["rows"], y=s["y"], weights=s["weights"])
        return dict(dy=dy, dweights=dweights)
    act = (moe.MOE_LINEAR_NONE, moe.MOE_LINEAR_RELU, moe.MOE_LINEAR_SILU, moe.MOE_LINEAR_GELU,
           moe.MOE_LINEAR_GELU_TANH)[ACTS.index(c["act"])]
    if kind == "linear":
        out = moe.moe_linear_forward(s["x"], s["w"], bias=s["bias"], act=act, addend=s["addend"], save_pre=c["save"],
                                     out_dtype=torch.float32 if c["f32"] else torch.bfloat16)
        return dict(out=out[0], pre=out[1]) if c["save"] else dict(out=out)
    dx, dw, dbias = moe.moe_linear_backward(s["dout"], s["x"], s["w"], pre=s["pre"], act=act, bias_dtype=s["bias"].dtype)
    return dict(dx=dx, dw=dw, dbias=dbias)


def run(state):
    if own:
        return _own_run(state)
    return _PLAIN[state["case"]["kind"]](state)


# ---------------------------------------------------------------- work
_SIZE = dict(bf16=2, f32=4, u8=1)


def work(case):
    kind, T = case["kind"], case["T"]
    if kind == "norm":
        H, r = case["H"], _SIZE.get(case["res"], 0)
        return dict(bytes=T * H * (4 + 2 * r) + 4 * H + (8 * T if case["save"] else 0), flops=8 * T * H)
    if kind == "norm_bwd":
        H, r = case["H"], _SIZE.get(case["res"], 0)
        # dy, the stream, its gradient, dx (and the gradient in the stream's type where that is fp32)
        return dict(bytes=T * H * (4 + (r or 2) + r + (4 if r == 4 else 0)) + 6 * H + 8 * T, flops=14 * T * H)
    if kind.startswith("linear"):
        K, N = case["K"], case["N"]
        o, b = 4 if case["f32"] else 2, 4 if case["bias32"] else 2
        if kind == "linear":
            return dict(bytes=2 * (T * K + N * K) + T * N * (o * (2 if case["addend"] else 1) + (2 if case["save"] else 0)) + b * N,
                        flops=2 * T * K * N)
        # without an activation nothing is read of its argument
        return dict(bytes=4 * (T * K + N * K) + T * N * (o + (0 if case["act"] == "none" else 2)) + b * N, flops=4 * T * K * N)
    H, k = case["H"], case["topk"]
    e = _SIZE[case["type"]]
    if kind == "permute":
        return dict(bytes=T * H * e * (1 + k) + 8 * T * k + 4 * case["E"], flops=T * k)
    o = _SIZE[case["out"]]
    if kind == "combine":
        return dict(bytes=T * H * (k * e + 2 * o) + 8 * T * k, flops=2 * T * k * H)
    return dict(bytes=T * H * (2 * k * e + o) + 12 * T * k, flops=3 * T * k * H)


# ---------------------------------------------------------------- 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    d = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor) and k not in ("ids", "rows")}
    kind = case["kind"]
    if kind == "norm":
        t = d["x"] + d["residual"] if "residual" in d else d["x"]
        H = t.shape[1]
        mean = t.sum(1) / H
        var = ((t - mean[:, None]) ** 2).sum(1) / H
        rstd = 1 / torch.sqrt(var + EPS)
        out = dict(y=torch.addcmul(d["bias"], (t - mean[:, None]) * rstd[:, None], d["weight"]))
        if "residual" in d:
            out["residual"] = t
        if case["save"]:
            out.update(mean=mean, rstd=rstd)
        return out
    if kind == "norm_bwd":
        H = case["H"]
        n = (d["s"] - d["mean"][:, None]) * d["rstd"][:, None]
        g = d["dy"] * d["weight"]
        a, b = g.sum(1) / H, torch.linalg.vecdot(g, n) / H
        ds = (g - a[:, None] - b[:, None] * n) * d["rstd"][:, None]
        if "dres" in d:
            ds += d["dres"]
        out = dict(dx=ds, dweight=torch.linalg.vecdot(d["dy"], n, dim=0), dbias=d["dy"].sum(0))
        if case["res"] == "f32":
            out["dresidual"] = ds
        return out
    if kind == "permute":
        E, topk = case["E"], case["topk"]
        ids = s["ids"].cpu().flatten()
        out = torch.zeros(ids.numel(), case["H"], dtype=torch.float64, device="cuda")
        rows, offsets, at = torch.empty(ids.numel(), dtype=torch.int32), [0], 0
        for e in range(E):
            pairs = (ids == e).nonzero().squeeze(1)
            out[at:at + len(pairs)] = d["x"][(pairs // topk).cuda()]
            rows[pairs] = torch.arange(at, at + len(pairs), dtype=torch.int32)
            at += len(pairs)
            offsets.append(at)
        left = ((ids < 0) | (ids >= E)).nonzero().squeeze(1)
        rows[left] = -1 - torch.arange(at, at + len(left), dtype=torch.int32)
        return dict(out=out, rows=rows.view(-1, topk).cuda(), offsets=torch.tensor(offsets, dtype=torch.int32, device="cuda"))
    if kind == "combine":
        out = d["residual"].clone()
        for j in range(case["topk"]):
            r = s["rows"][:, j].long()
            t = (r >= 0).nonzero().squeeze(1)
            out[t] += d["weights"][t, j, None] * d["y"][r[t]]
        return out
    if kind == "combine_bwd":
        dy, dw = torch.zeros_like(d["y"]), torch.zeros_like(d["weights"])
        for j in range(case["topk"]):
            r = s["rows"][:, j].long()
            t = (r >= 0).nonzero().squeeze(1)
            dy[r[t]] = d["weights"][t, j, None] * d["dout"][t]
            dw[t, j] = torch.linalg.vecdot(d["dout"][t], d["y"][r[t]])
        return dict(dy=dy, dweights=dw)
    act = case["act"]
    if kind == "linear":
        z = torch.addmm(d["bias"], d["x"], d["w"].t())
        out = {"none": lambda: z, "relu": lambda: z.clamp_min(0), "silu": lambda: z * torch.sigmoid(z),
               "gelu": lambda: z * torch.special.ndtr(z),
               "gelu_tanh": lambda: 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))}[act]()
        out = dict(out=out + d["addend"] if "addend" in d else out)
        return dict(out, pre=z) if case["save"] else out
    z = d["pre"]
    if act == "none":
        dz = d["dout"]
    elif act == "relu":
        dz = torch.where(z > 0, d["dout"], torch.zeros_like(z))
    elif act == "silu":
        p = torch.sigmoid(z)
        dz = d["dout"] * (p + z * p * (1 - p))
    elif act == "gelu":
        dz = d["dout"] * (torch.special.ndtr(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi))
    else:
        t = torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
        dz = d["dout"] * (0.5 * (1 + t) + 0.5 * z * (1 - t * t) * math.sqrt(2 / math.pi) * (1 + 0.134145 * z * z))
    return dict(dx=torch.mm(dz, d["w"]), dw=torch.mm(dz.t(), d["x"]), dbias=dz.sum(0))
