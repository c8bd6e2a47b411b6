"""Cases that measure the dense operators around the routed experts.

A mixture-of-experts block needs, next to the routed experts: the residual
addition and RMS norm that makes the layer's input (in bf16, and in MXFP8 for
an 8-bit shared expert), the shared expert itself (a gated feed-forward block,
with its backward pass), and the dense projections that may carry one low-rank
adapter per request (without adapters and in fp32: the router's logits).

`own` selects between the plain torch form of each operator and the calls a
user makes of this package.
"""
import math

import torch

own = False

# Kinds of a case:
#   norm    residual addition + RMS norm; mx: also the MXFP8 output; res32:
#           the residual stream is kept in fp32 (else bf16)
#   ffn     gated feed-forward block in bf16; save: gate_up is an output (the
#           training forward); adapters > 0: low-rank adapters on both
#           projections
#   ffn_mx  the same block with MXFP8 activations and weights
#   bwd     backward of the bf16 block
#   linear  projection with low-rank adapters (adapters = 0: none); f32: fp32
#           output
EPS = 1e-6


def listed():
    return [
        # one token of one request: latency of the layer's first step
        dict(name="norm_token", kind="norm", T=1, H=3584, res32=False, mx=False),
        # an odd chunk of prompts in a model with an fp32 residual stream, feeding an 8-bit shared expert
        dict(name="norm_odd_mx", kind="norm", T=1531, H=2784, res32=True, mx=True),
        # a full prefill batch: bf16 for the routed experts, MXFP8 for the shared one
        dict(name="norm_prompt_mx", kind="norm", T=16384, H=3584, res32=False, mx=True),
        # one token through the shared expert
        dict(name="ffn_token", kind="ffn", T=1, H=3584, I=2048, save=False, adapters=0, rank=0),
        # a ragged decode batch whose requests use different adapters, on one rank's share of the block
        dict(name="ffn_adapters_batch", kind="ffn", T=37, H=3584, I=384, save=False, adapters=12, rank=16),
        # the training forward over a full batch of sequences
        dict(name="ffn_train", kind="ffn", T=8192, H=3584, I=4096, save=True, adapters=0, rank=0),
        # a decode batch through an 8-bit shared expert
        dict(name="ffn_mx_batch", kind="ffn_mx", T=16, H=3584, I=2048),
        # a prefill chunk through an 8-bit shared expert
        dict(name="ffn_mx_prompt", kind="ffn_mx", T=4096, H=3584, I=2048),
        # backward over a short odd batch of a small block
        dict(name="bwd_odd", kind="bwd", T=777, H=1000, I=520),
        # backward over a full batch of sequences
        dict(name="bwd_train", kind="bwd", T=8192, H=3584, I=2048),
        # a decode batch of many requests with an adapter each beside one projection
        dict(name="linear_adapters_batch", kind="linear", T=48, K=3584, N=4096, adapters=16, rank=16, f32=False, runs=False),
        # a prefill batch of a few long requests with larger adapters
        dict(name="linear_adapters_prompt", kind="linear", T=4099, K=3584, N=3584, adapters=8, rank=64, f32=False, runs=True),
    ]


def _log_int(rng, lo, hi, step=1):
    return max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step)


def draw(rng):
    most = 7.2e11  # flops of the largest listed cases
    kind = rng.choice(["norm", "ffn", "ffn_mx", "bwd", "linear"])
    if kind == "norm":
        mx = rng.random() < 0.5
        H = _log_int(rng, 64, 8192, 32) if mx else _log_int(rng, 33, 8192)
        T = min(_log_int(rng, 1, 32768), 16384 * 3584 // H)
        return dict(kind=kind, T=T, H=H, res32=rng.random() < 0.5, mx=mx)
    if kind == "linear":
        K, N = _log_int(rng, 64, 8192, 8), _log_int(rng, 16, 8192, 8)
        f32 = rng.random() < 0.25
        T = min(_log_int(rng, 1, 8192), int(most / (2 * K * N)))
        n = 0 if f32 or rng.random() < 0.2 else rng.randint(1, 32)
        return dict(kind=kind, T=T, K=K, N=N, adapters=n, rank=8 * rng.randint(1, 8) if n else 0, f32=f32, runs=rng.random() < 0.5)
    step = 32 if kind == "ffn_mx" else 8
    H, I = _log_int(rng, 128, 8192, step), _log_int(rng, 128, 8192, step)
    T = min(_log_int(rng, 1, 8192), int(most / ((12 if kind == "bwd" else 6) * H * I)))
    c = dict(kind=kind, T=T, H=H, I=I)
    if kind == "ffn":
        save = rng.random() < 0.3
        n = 0 if save or rng.random() < 0.5 else rng.randint(1, 16)
        c.update(save=save, adapters=n, rank=8 * rng.randint(1, 4) if n else 0)
    return c


# ---------------------------------------------------------------- inputs
def _adapters(g, T, K, N, n, rank, runs):
    """A stack of n adapters of at most `rank`, and each token's adapter (-1:
    none): by runs of tokens (prompts) or token by token (decode)."""
    dev = "cuda"
    a = (torch.randn(n, rank, K, generator=g, device=dev) / math.sqrt(K)).bfloat16()
    b = (torch.randn(n, N, rank, generator=g, device=dev) * (0.5 / math.sqrt(rank))).bfloat16()
    ranks = torch.randint(1, rank // 8 + 1, (n,), generator=g, device=dev, dtype=torch.int32) * 8
    scale = torch.rand(n, generator=g, device=dev) + 0.5
    if runs:
        cuts = torch.randint(0, T + 1, (n,), generator=g, device=dev).sort().values
        index = torch.searchsorted(cuts, torch.arange(T, device=dev), right=True).to(torch.int32) - 1
    else:
        index = torch.randint(-1, n, (T,), generator=g, device=dev, dtype=torch.int32)
    return a, b, index, ranks, scale


def _weight(g, n, k):
    return (torch.randn(n, k, generator=g, device="cuda") / math.sqrt(k)).bfloat16()


def _to_mx(v):
    """fp32 [..., n] -> e4m3 values and e8m0 scales, one scale per 32: the
    smallest power of two that brings the largest magnitude to at most 448."""
    blocks = v.unflatten(-1, (-1, 32))
    m, e = torch.frexp(blocks.abs().amax(-1))  # m in [0.5, 1)
    e = (e - 9 + (m > 0.875).to(e.dtype)).clamp(-127, 127)
    e = torch.where(m == 0, torch.full_like(e, -127), e)
    q = torch.ldexp(torch.ldexp(blocks, -(e // 2).unsqueeze(-1)), -(e - e // 2).unsqueeze(-1))
    q = q.clamp(-448, 448).to(torch.float8_e4m3fn).flatten(-2)
    return q, (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _from_mx(q, s):
    return (q.float().unflatten(-1, (-1, 32)) * s.float().unsqueeze(-1)).flatten(-2)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    dev = "cuda"
    kind, T = case["kind"], case["T"]
    if kind == "norm":
        H = case["H"]
        x = (torch.randn(T, H, generator=g, device=dev)).bfloat16()
        # a residual stream has rows of very different size
        r = torch.randn(T, H, generator=g, device=dev) * torch.exp(torch.randn(T, 1, generator=g, device=dev))
        w = (1 + 0.1 * torch.randn(H, generator=g, device=dev)).bfloat16()
        return dict(case=case, x=x, residual=r if case["res32"] else r.bfloat16(), weight=w)
    if kind == "linear":
        K, N = case["K"], case["N"]
        s = dict(case=case, x=torch.randn(T, K, generator=g, device=dev).bfloat16(), w=_weight(g, N, K))
        n = case["adapters"]
        s["lora"] = _adapters(g, T, K, N, n, case["rank"], case["runs"]) if n else None
        return s
    H, I = case["H"], case["I"]
    x = torch.randn(T, H, generator=g, device=dev).bfloat16()
    w13, w2 = _weight(g, 2 * I, H), _weight(g, H, I)
    # what the routed experts gave for these tokens
    addend = torch.randn(T, H, generator=g, device=dev).bfloat16()
    if kind == "ffn":
        s = dict(case=case, x=x, w13=w13, w2=w2, addend=addend)
        n = case["adapters"]
        s["lora13"] = _adapters(g, T, H, 2 * I, n, case["rank"], False) if n else None
        if n:
            a, b, _, ranks, scale = _adapters(g, T, I, H, n, case["rank"], False)
            s["lora2"] = (a, b, s["lora13"][2], ranks, scale)
        else:
            s["lora2"] = None
        return s
    if kind == "ffn_mx":
        xq, xs = _to_mx(x.float())
        w13q, w13s = _to_mx(w13.float())
        w2q, w2s = _to_mx(w2.float())
        return dict(case=case, xq=xq, xs=xs, w13q=w13q, w13s=w13s, w2q=w2q, w2s=w2s, addend=addend)
    gate_up = x @ w13.t()
    return dict(case=case, x=x, w13=w13, w2=w2, gate_up=gate_up, dout=addend)


# ---------------------------------------------------------------- plain forms
def _plain_norm(s):
    c = s["case"]
    v = s["x"].float() + s["residual"].float()
    n = v * torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS) * s["weight"].float()
    out = dict(y=n.bfloat16(), residual=v.to(s["residual"].dtype))
    if c["mx"]:
        out["q"], out["scale"] = _to_mx(n)
    return out


def _plain_lora(x, lora):
    """x fp32 [T, K] -> fp32 [T, N]: every adapter's narrow product, masked to
    the token's own adapter and its rank."""
    a, b, index, ranks, scale = lora
    n, rank, _ = a.shape
    v = (x @ a.float().flatten(0, 1).t()).unflatten(1, (n, rank))
    ids = torch.arange(n, device=x.device)
    keep = (index.unsqueeze(1) == ids).unsqueeze(2) & (torch.arange(rank, device=x.device) < ranks.unsqueeze(1))
    v = torch.where(keep, v * scale.view(1, n, 1), torch.zeros_like(v)).flatten(1)
    return v @ b.float().transpose(1, 2).flatten(0, 1)


def _plain_linear(s):
    x = s["x"].float()
    y = x @ s["w"].float().t()
    if s["lora"] is not None:
        y = y + _plain_lora(x, s["lora"])
    return y if s["case"]["f32"] else y.bfloat16()


def _plain_ffn(s):
    x = s["x"].float()
    I = s["case"]["I"]
    gu = x @ s["w13"].float().t()
    if s["lora13"] is not None:
        gu = gu + _plain_lora(x, s["lora13"])
    g, u = gu[:, :I], gu[:, I:]
    h = g / (1 + torch.exp(-g)) * u
    y = h @ s["w2"].float().t() + s["addend"].float()
    if s["lora2"] is not None:
        y = y + _plain_lora(h, s["lora2"])
    return dict(out=y.bfloat16(), gate_up=gu.bfloat16()) if s["case"]["save"] else dict(out=y.bfloat16())


def _plain_ffn_mx(s):
    I = s["case"]["I"]
    gu = _from_mx(s["xq"], s["xs"]) @ _from_mx(s["w13q"], s["w13s"]).t()
    g, u = gu[:, :I], gu[:, I:]
    h = _from_mx(*_to_mx(g / (1 + torch.exp(-g)) * u))
    return dict(out=(h @ _from_mx(s["w2q"], s["w2s"]).t() + s["addend"].float()).bfloat16())


def _plain_bwd(s):
    I = s["case"]["I"]
    dout, x = s["dout"].float(), s["x"].float()
    g, u = s["gate_up"][:, :I].float(), s["gate_up"][:, I:].float()
    sig = 1 / (1 + torch.exp(-g))
    silu = g * sig
    dh = dout @ s["w2"].float()
    dgu = torch.cat([dh * u * sig * (1 + g * (1 - sig)), dh * silu], 1)
    return dict(dx=(dgu @ s["w13"].float()).bfloat16(), dw13=(dgu.t() @ x).bfloat16(),
                dw2=(dout.t() @ (silu * u)).bfloat16())


_PLAIN = dict(norm=_plain_norm, linear=_plain_linear, ffn=_plain_ffn, ffn_mx=_plain_ffn_mx, bwd=_plain_bwd)


# ---------------------------------------------------------------- one pass
def _own_run(s):
    import mxfp4_grouped_gemm_amd as moe

    c = s["case"]
    kind = c["kind"]
    if kind == "norm":
        y, res, q, scale = moe.moe_rms_norm(s["x"], s["weight"], residual=s["residual"], eps=EPS, mxfp8=c["mx"])
        return dict(y=y, residual=res, q=q, scale=scale) if c["mx"] else dict(y=y, residual=res)
    if kind == "linear":
        return moe.moe_lora_linear(s["x"], s["w"], lora=s["lora"],
                                   out_dtype=torch.float32 if c["f32"] else torch.bfloat16)
    if kind == "ffn":
        if c["save"]:
            out, gate_up = moe.moe_ffn_forward(s["x"], s["w13"], s["w2"], addend=s["addend"], save_gate_up=True)
            return dict(out=out, gate_up=gate_up)
        return dict(out=moe.moe_ffn_forward(s["x"], s["w13"], s["w2"], addend=s["addend"], lora13=s["lora13"],
                                            lora2=s["lora2"]))
    if kind == "ffn_mx":
        return dict(out=moe.moe_ffn_forward_mxfp8(s["xq"], s["xs"], s["w13q"], s["w13s"], s["w2q"], s["w2s"],
                                                  addend=s["addend"]))
    dx, dw13, dw2 = moe.moe_ffn_backward(s["dout"], s["x"], s["gate_up"], s["w13"], s["w2"])
    return dict(dx=dx, dw13=dw13, dw2=dw2)


def run(state):
    if own:
        return _own_run(state)
    return _PLAIN[state["case"]["kind"]](state)


# ---------------------------------------------------------------- work
def work(case):
    kind, T = case["kind"], case["T"]
    if kind == "norm":
        H = case["H"]
        r = 4 if case["res32"] else 2
        return dict(bytes=T * H * (2 + r + r + 2 + (33 / 32 if case["mx"] else 0)) + 2 * H, flops=4 * T * H)
    if kind == "linear":
        K, N, n, r = case["K"], case["N"], case["adapters"], case["rank"]
        used = min(n, T)  # adapters that a batch can touch; their mean rank is about half the largest
        mean = (r + 8) / 2
        return dict(bytes=2 * (T * K + N * K) + (4 if case["f32"] else 2) * T * N + used * mean * 2 * (K + N),
                    flops=2 * T * K * N + (2 * T * mean * (K + N) if n else 0))
    H, I = case["H"], case["I"]
    if kind == "ffn":
        n, r = case["adapters"], case["rank"]
        mean = (r + 8) / 2
        extra = min(n, T) * mean * 2 * (H + 2 * I + I + H)
        return dict(bytes=6 * H * I + 6 * T * H + (4 * T * I if case["save"] else 0) + extra,
                    flops=6 * T * H * I + (2 * T * mean * (2 * H + 3 * I) if n else 0))
    if kind == "ffn_mx":
        return dict(bytes=3 * H * I * 33 / 32 + T * H * (33 / 32 + 4), flops=6 * T * H * I)
    return dict(bytes=2 * (3 * H * I * 2 + 3 * T * H + 2 * T * I), flops=12 * T * H * I)


# ---------------------------------------------------------------- 64 bits
def _mx64(v):
    """fp64 -> the (values, scales) that MXFP8 holds, by arithmetic on the
    exponent: three mantissa bits down to 2^-6, steps of 2^-9 below."""
    T, n = v.shape
    b = v.reshape(T, n // 32, 32)
    amax = b.abs().max(-1, keepdim=True).values
    safe = torch.where(amax > 0, amax, torch.ones_like(amax))
    e = torch.ceil(torch.log2(safe / 448))
    two = torch.full_like(e, 2.0)
    # log2 may be off by an ulp next to a power of two: settle it by products
    e = torch.where(safe > 448 * torch.pow(two, e), e + 1, e)
    e = torch.where(safe <= 448 * torch.pow(two, e - 1), e - 1, e)
    e = torch.where(amax > 0, e, torch.full_like(e, -127)).clamp(-127, 127)
    scale = torch.pow(two, e)
    z = b / scale
    k = torch.floor(torch.log2(z.abs().clamp_min(2.0 ** -6)))
    step = torch.pow(torch.full_like(k, 2.0), k - 3)
    z = (torch.round(z / step) * step).clamp(-448, 448)  # torch.round: ties to even
    return z.reshape(T, n), scale.squeeze(-1)


def _lora64(x, lora):
    a, b, index, ranks, scale = lora
    out = torch.zeros(x.shape[0], b.shape[1], dtype=torch.float64, device=x.device)
    for i in range(a.shape[0]):
        rows = (index == i).nonzero().squeeze(1)
        r = int(ranks[i])
        out[rows] = float(scale[i]) * ((x[rows] @ a[i, :r].double().t()) @ b[i, :, :r].double().t())
    return out


def exact(case, seed):
    s = prepare(case, seed)
    d = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor)}
    kind = case["kind"]
    if kind == "norm":
        t = d["x"] + d["residual"]
        n = t / torch.sqrt((t * t).sum(1, keepdim=True) / t.shape[1] + EPS) * d["weight"]
        out = dict(y=n, residual=t)
        if case["mx"]:
            out["q"], out["scale"] = _mx64(n)
        return out
    if kind == "linear":
        y = torch.mm(d["x"], d["w"].t())
        return y + _lora64(d["x"], s["lora"]) if s["lora"] is not None else y
    I = case["I"]
    if kind == "bwd":
        g, u = d["gate_up"].split(I, dim=1)
        p = torch.sigmoid(g)
        dh = torch.mm(d["dout"], d["w2"])
        dgate, dup = dh * u * (p + g * p * (1 - p)), dh * g * p
        return dict(dx=torch.mm(dgate, d["w13"][:I]) + torch.mm(dup, d["w13"][I:]),
                    dw13=torch.cat([torch.mm(dgate.t(), d["x"]), torch.mm(dup.t(), d["x"])]),
                    dw2=torch.mm(d["dout"].t(), g * p * u))
    if kind == "ffn_mx":
        def wide(q, e):
            return q * e.repeat_interleave(32, dim=1)
        x, w13, w2 = wide(d["xq"], d["xs"]), wide(d["w13q"], d["w13s"]), wide(d["w2q"], d["w2s"])
        g, u = torch.mm(x, w13[:I].t()), torch.mm(x, w13[I:].t())
        return dict(out=torch.mm(wide(*_mx64(g * torch.sigmoid(g) * u)), w2.t()) + d["addend"])
    gu = torch.mm(d["x"], d["w13"].t())
    if s["lora13"] is not None:
        gu = gu + _lora64(d["x"], s["lora13"])
    h = gu[:, :I] * torch.sigmoid(gu[:, :I]) * gu[:, I:]
    y = torch.mm(h, d["w2"].t()) + d["addend"]
    if s["lora2"] is not None:
        y = y + _lora64(h, s["lora2"])
    return dict(out=y, gate_up=gu) if case["save"] else dict(out=y)
