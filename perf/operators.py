"""The pre-norm feed-forward operators around the MoE layer, as cases to measure.

Three operators, each with its backward pass:

``norm``    s = x + residual, y = s / sqrt(mean(s^2) + eps) * weight, with y in
            bf16 and, where asked for, in e4m3 codes with one power-of-two
            scale a row (the form the e4m3 experts read);
``gated``   h = silu(x W1^T) * (x W3^T), the up half of a dense expert (a shared
            expert that every token visits), keeping both projections where a
            backward pass follows;
``linear``  y = residual + act(x W^T + bias), the down half and any projection
            beside the layer.

``run`` computes one of them on the inputs that ``prepare`` made: with ``own``
false in plain 32-bit torch operations, with ``own`` true through the package's
entry points.  ``exact`` is the definition in 64 bits.
"""
import math

import torch

own = False

EPS = 1e-6
GAIN = math.sqrt(2.0 / math.pi)


def listed():
    return [
        # One token of decode at the width of the DeepSeek-shaped layer: the residual's addition and the
        # norm, for the router (bf16) and for e4m3 experts (codes and scale).  Latency.
        dict(name="norm_1x7168", op="norm", n=1, d=7168, residual=True, codes=True),
        # A prefill batch of the same layer.
        dict(name="norm_4096x7168", op="norm", n=4096, d=7168, residual=True, codes=True),
        # The norm's gradient in a training step whose batch is ragged (packed sequences).
        dict(name="norm_bwd_4093x4096", op="norm_bwd", n=4093, d=4096, residual=True),
        # The shared expert's up half on one token: two weight streams.
        dict(name="gated_1x7168x2048", op="gated", n=1, d=7168, f=2048, save=False),
        # A ragged decode batch at the widths of the Qwen3-shaped layer.
        dict(name="gated_100x2048x768", op="gated", n=100, d=2048, f=768, save=False),
        # Prefill or a training forward at the widths of the Mixtral-shaped layer, keeping both projections.
        dict(name="gated_4096x4096x14336", op="gated", n=4096, d=4096, f=14336, save=True),
        # The up half's gradients for a ragged batch at the DeepSeek-shaped shared expert.
        dict(name="gated_bwd_2050x7168x2048", op="gated_bwd", n=2050, d=7168, f=2048),
        # The down half on eight tokens, added to the residual stream.
        dict(name="linear_8x2048x7168", op="linear", n=8, d=2048, f=7168, act="none", bias=False, residual=True, save=False),
        # A biased projection with its activation in a training forward, odd sizes, pre-activation kept.
        dict(name="linear_1001x4096x2056", op="linear", n=1001, d=4096, f=2056, act="gelu", bias=True, residual=False, save=True),
        # The down half of a Mixtral-shaped dense block on a prefill batch, added to the residual stream.
        dict(name="linear_4096x14336x4096", op="linear", n=4096, d=14336, f=4096, act="none", bias=False, residual=True, save=False),
        # A small biased projection's gradients through its activation.
        dict(name="linear_bwd_777x1024x4096", op="linear_bwd", n=777, d=1024, f=4096, act="gelu", bias=True),
        # The down half's gradients at the DeepSeek-shaped shared expert.
        dict(name="linear_bwd_4096x2048x7168", op="linear_bwd", n=4096, d=2048, f=7168, act="none", bias=False),
    ]


def _spread(rng, lo, hi, step):
    """A multiple of ``step`` in lo..hi, spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return min(hi, max(lo, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_bwd", "gated", "gated", "gated_bwd", "linear", "linear", "linear_bwd"])
    while True:
        if op in ("norm", "norm_bwd"):
            c = dict(op=op, n=_spread(rng, 1, 8192, 1), d=_spread(rng, 256, 16384, 8), residual=rng.random() < 0.7)
            if op == "norm":
                c["codes"] = rng.random() < 0.6
            if c["n"] * c["d"] <= 4096 * 7168:
                return c
            continue
        c = dict(op=op, n=_spread(rng, 1, 8192, 1), d=_spread(rng, 256, 14336, 8), f=_spread(rng, 256, 14336, 8))
        if op.startswith("linear"):
            c["act"] = rng.choice(["none", "none", "relu", "silu", "gelu", "gelu_tanh"])
            c["bias"] = rng.random() < 0.5
        if op == "linear":
            c["residual"] = rng.random() < 0.6
        if op in ("gated", "linear"):
            c["save"] = rng.random() < 0.4
        if work(c)["flops"] <= 4.0e11 and c["d"] * c["f"] <= 4096 * 14336:
            return c


def work(case):
    n, d, op = case["n"], case["d"], case["op"]
    if op == "norm":
        streams = 2 + (2 if case["residual"] else 0)  # x, y; the residual in and out
        b = n * d * 2 * streams + d * 2 + ((n * d + 4 * n) if case["codes"] else 0)
        return {"bytes": b, "flops": 6 * n * d}
    if op == "norm_bwd":
        return {"bytes": n * d * 2 * (3 + (1 if case["residual"] else 0)) + d * 2 + d * 4, "flops": 12 * n * d}
    f = case["f"]
    if op == "gated":
        return {"bytes": 2 * (n * d + 2 * d * f + n * f * (3 if case["save"] else 1)), "flops": 4 * n * d * f}
    if op == "gated_bwd":
        return {"bytes": 2 * (3 * n * f + 2 * n * d + 4 * d * f), "flops": 8 * n * d * f}
    if op == "linear":
        b = 2 * (n * d + d * f + n * f * (1 + int(case["residual"]) + int(case["save"]))) + (4 * f if case["bias"] else 0)
        return {"bytes": b, "flops": 2 * n * d * f}
    b = 2 * (n * f * (1 + int(case["act"] != "none")) + 2 * n * d + 2 * d * f) + (4 * f if case["bias"] else 0)
    return {"bytes": b, "flops": 4 * n * d * f}


# ------------------------------------------------------------------ inputs
def _inputs(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed) * 1_000_003 + 17)

    def normal(*shape, scale=1.0):
        return torch.randn(shape, generator=gen, device=dev).mul_(scale).to(torch.bfloat16)

    n, d, op = case["n"], case["d"], case["op"]
    t = {}
    if op in ("norm", "norm_bwd"):
        # a residual stream: tokens of different size, a few channels much larger than the rest
        size = torch.exp(torch.randn((n, 1), generator=gen, device=dev))
        channel = torch.ones(d, device=dev)
        channel[torch.randint(0, d, (max(1, d // 512),), generator=gen, device=dev)] = 20.0
        stream = (torch.randn((n, d), generator=gen, device=dev) * size * channel).to(torch.bfloat16)
        t["weight"] = (1.0 + 0.2 * torch.randn(d, generator=gen, device=dev)).to(torch.bfloat16)
        if op == "norm":
            t["x"] = normal(n, d) if case["residual"] else stream
            t["residual"] = stream if case["residual"] else None
        else:
            t["s"] = stream
            t["dy"] = normal(n, d, scale=0.05)
            t["dresidual"] = normal(n, d, scale=0.05) if case["residual"] else None
        return t
    f = case["f"]
    if op in ("gated", "gated_bwd"):
        t["x"] = normal(n, d)
        t["w1"] = normal(f, d, scale=d ** -0.5)
        t["w3"] = normal(f, d, scale=d ** -0.5)
        if op == "gated_bwd":  # what the forward pass kept, and the gradient that comes in
            t["g"] = normal(n, f)
            t["u"] = normal(n, f)
            t["dh"] = normal(n, f, scale=0.05)
        return t
    t["x"] = normal(n, d)
    t["w"] = normal(f, d, scale=d ** -0.5)
    if op == "linear":
        t["bias"] = torch.randn(f, generator=gen, device=dev) * 0.5 if case["bias"] else None
        t["residual"] = normal(n, f, scale=2.0) if case["residual"] else None
    else:
        t["dy"] = normal(n, f, scale=0.05)
        t["z"] = normal(n, f) if case["act"] != "none" else None
    return t


def prepare(case, seed):
    """The inputs, and the output buffers that a program keeps from step to step."""
    t = _inputs(case, seed)
    op, n, d, f = case["op"], case["n"], case["d"], case.get("f", 0)
    dev = torch.device("cuda")

    def buf(*shape, dtype=torch.bfloat16):
        return torch.empty(shape, dtype=dtype, device=dev)

    if op == "norm":
        t["y"] = buf(n, d)
        t["residual_out"] = buf(n, d) if case["residual"] else None
        t["yq"] = buf(n, d, dtype=torch.uint8) if case["codes"] else None
        t["y_scale"] = buf(n, dtype=torch.float32) if case["codes"] else None
    elif op == "norm_bwd":
        t["dx"], t["dweight"] = buf(n, d), buf(d, dtype=torch.float32)
    elif op == "gated":
        t["h"] = buf(n, f)
        t["g"], t["u"] = (buf(n, f), buf(n, f)) if case["save"] else (None, None)
    elif op == "gated_bwd":
        t["dx"], t["dw1"], t["dw3"] = buf(n, d), buf(f, d), buf(f, d)
    elif op == "linear":
        t["y"] = buf(n, f)
        t["z"] = buf(n, f) if case["save"] else None
    else:
        t["dx"], t["dw"] = buf(n, d), buf(f, d)
        t["dbias"] = buf(f, dtype=torch.float32) if case["bias"] else None
    t["op"], t["act"], t["case"] = op, case.get("act", "silu"), case
    return t


# ------------------------------------------------------------------ the package's calls
def _handle(t):
    """The package, the activation's code and the workspace: made at a state's first call and kept with its buffers."""
    if "handle" not in t:
        from mixture_experts_layer_02_gb300 import moe
        fn = {"none": moe.FN_NONE, "relu": moe.FN_RELU, "silu": moe.FN_SILU, "gelu": moe.FN_GELU,
              "gelu_tanh": moe.FN_GELU_TANH}[t["act"]]
        name = {"norm_bwd": "rmsnorm_backward", "gated": "gated_linear", "gated_bwd": "gated_linear_backward",
                "linear": "linear", "linear_bwd": "linear_backward"}.get(t["op"])
        c = t["case"]
        t["handle"] = moe, fn, name and moe.workspace(name, N=c["n"], D=c["d"], Dff=c.get("f", 0))
    return t["handle"]


def _run_own(t):
    (moe, fn, ws), op = _handle(t), t["op"]
    if op == "norm":
        y, yq, scale, s = moe.moe_rmsnorm(t["x"], t["weight"], residual=t["residual"], eps=EPS, y=t["y"], yq=t["yq"],
                                          y_scale=t["y_scale"], residual_out=t["residual_out"])
        return [y, s, None if yq is None else yq.view(torch.float8_e4m3fn), scale]
    if op == "norm_bwd":
        return list(moe.moe_rmsnorm_backward(t["dy"], t["s"], t["weight"], dresidual=t["dresidual"], eps=EPS, dx=t["dx"],
                                             dweight=t["dweight"], ws=ws))
    if op == "gated":
        return list(moe.moe_gated_linear(t["x"], t["w1"], t["w3"], fn, h=t["h"], g=t["g"], u=t["u"], ws=ws))
    if op == "gated_bwd":
        return list(moe.moe_gated_linear_backward(t["dh"], t["x"], t["w1"], t["w3"], t["g"], t["u"], fn, dx=t["dx"],
                                                  dw1=t["dw1"], dw3=t["dw3"], ws=ws))
    if op == "linear":
        return list(moe.moe_linear(t["x"], t["w"], bias=t["bias"], residual=t["residual"], fn=fn, y=t["y"], z=t["z"],
                                   ws=ws))
    return list(moe.moe_linear_backward(t["dy"], t["x"], t["w"], z=t["z"], fn=fn, dx=t["dx"], dw=t["dw"],
                                        dbias=t["dbias"], ws=ws))


# ------------------------------------------------------------------ plain form, 32 bits
def _act(z, name):
    if name == "none":
        return z
    if name == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if name == "silu":
        return z / (1 + torch.exp(-z))
    if name == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    return 0.5 * z * (1 + torch.tanh(GAIN * (z + 0.044715 * z * z * z)))


def _act_slope(z, name):
    if name == "none":
        return torch.ones_like(z)
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "silu":
        p = 1 / (1 + torch.exp(-z))
        return p * (1 + z * (1 - p))
    if name == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    t = torch.tanh(GAIN * (z + 0.044715 * z * z * z))
    return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * GAIN * (1 + 3 * 0.044715 * z * z)


def _run_plain(t):
    bf16, op = torch.bfloat16, t["op"]
    if op == "norm":
        s = t["x"].float()
        if t["residual"] is not None:
            s = s + t["residual"].float()
        y = s * torch.rsqrt((s * s).mean(1, keepdim=True) + EPS) * t["weight"].float()
        codes = scale = None
        if t["yq"] is not None:
            top = y.abs().amax(1)
            m, e = torch.frexp(top)  # top = m 2^e, m in [0.5, 1): the smallest k with top <= 448 2^k
            k = torch.where(top > 0, e - 9 + (m > 0.875).int(), torch.full_like(e, -126)).clamp(min=-126)
            scale = torch.ldexp(torch.ones_like(top), k)
            codes = (y / scale[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
        return [y.to(bf16), s.to(bf16) if t["residual"] is not None else None, codes, scale]
    if op == "norm_bwd":
        s, dy, w = t["s"].float(), t["dy"].float(), t["weight"].float()
        r = torch.rsqrt((s * s).mean(1, keepdim=True) + EPS)
        xhat, v = s * r, dy * w
        dx = r * (v - xhat * (v * xhat).mean(1, keepdim=True))
        if t["dresidual"] is not None:
            dx = dx + t["dresidual"].float()
        return [dx.to(bf16), (dy * xhat).sum(0)]
    if op == "gated":
        x = t["x"].float()
        g, u = x @ t["w1"].float().T, x @ t["w3"].float().T
        keep = [g.to(bf16), u.to(bf16)] if t["g"] is not None else [None, None]
        return [(_act(g, "silu") * u).to(bf16)] + keep
    if op == "gated_bwd":
        x, g, u, dh = t["x"].float(), t["g"].float(), t["u"].float(), t["dh"].float()
        dg, du = dh * u * _act_slope(g, "silu"), dh * _act(g, "silu")
        dx = dg @ t["w1"].float() + du @ t["w3"].float()
        return [dx.to(bf16), (dg.T @ x).to(bf16), (du.T @ x).to(bf16)]
    if op == "linear":
        z = t["x"].float() @ t["w"].float().T
        if t["bias"] is not None:
            z = z + t["bias"]
        y = _act(z, t["act"])
        if t["residual"] is not None:
            y = y + t["residual"].float()
        return [y.to(bf16), z.to(bf16) if t["z"] is not None else None]
    dz = t["dy"].float()
    if t["act"] != "none":
        dz = dz * _act_slope(t["z"].float(), t["act"])
    return [(dz @ t["w"].float()).to(bf16), (dz.T @ t["x"].float()).to(bf16), dz.sum(0) if t["dbias"] is not None else None]


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------ the definition, 64 bits
def _sigmoid64(z):
    e = torch.exp(-z.abs())
    return torch.where(z >= 0, 1 / (1 + e), e / (1 + e))


def _phi64(z):  # the normal distribution function and its density
    return 0.5 * torch.erfc(-z / math.sqrt(2.0)), torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)


def _act64(z, name):
    """(value, slope) of an activation."""
    if name == "none":
        return z, torch.ones_like(z)
    if name == "relu":
        return z.clamp(min=0), torch.heaviside(z, torch.zeros((), dtype=z.dtype, device=z.device))
    if name == "silu":
        p = _sigmoid64(z)
        return z * p, p + z * p * (1 - p)
    if name == "gelu":
        c, pdf = _phi64(z)
        return z * c, c + z * pdf
    q = 2 * GAIN * (z + 0.044715 * z ** 3)  # (1 + tanh(q / 2)) / 2 is the sigmoid of q
    p = _sigmoid64(q)
    return z * p, p + z * p * (1 - p) * 2 * GAIN * (1 + 0.134145 * z ** 2)


def exact(case, seed):
    t = {k: (v.double() if isinstance(v, torch.Tensor) else v) for k, v in _inputs(case, seed).items()}
    op = case["op"]
    if op == "norm":
        s = t["x"] if t["residual"] is None else t["x"].add(t["residual"])
        y = torch.einsum("nd,n,d->nd", s, s.square().sum(1).div(case["d"]).add(EPS).pow(-0.5), t["weight"])
        codes = scale = None
        if case["codes"]:
            scale = torch.exp2(torch.ceil(torch.log2(y.abs().amax(1).clamp(min=448 * 2.0 ** -126) / 448)))
            codes = y / scale.unsqueeze(1)
        return [y, s if t["residual"] is not None else None, codes, scale]
    if op == "norm_bwd":
        s, dy = t["s"], t["dy"]
        inv = s.square().sum(1).div(case["d"]).add(EPS).pow(-0.5)
        dweight = torch.einsum("nd,nd,n->d", dy, s, inv)
        along = torch.einsum("nd,d,nd,n->n", dy, t["weight"], s, inv ** 3) / case["d"]
        dx = torch.einsum("nd,d,n->nd", dy, t["weight"], inv) - s * along.unsqueeze(1)
        return [dx if t["dresidual"] is None else dx + t["dresidual"], dweight]
    if op == "gated":
        g, u = torch.einsum("nd,fd->nf", t["x"], t["w1"]), torch.einsum("nd,fd->nf", t["x"], t["w3"])
        return [_act64(g, "silu")[0] * u] + ([g, u] if case["save"] else [None, None])
    if op == "gated_bwd":
        value, slope = _act64(t["g"], "silu")
        both = torch.cat([t["dh"] * t["u"] * slope, t["dh"] * value], 1)
        dw = torch.einsum("nf,nd->fd", both, t["x"])
        return [torch.einsum("nf,fd->nd", both, torch.cat([t["w1"], t["w3"]]))] + list(dw.split(case["f"]))
    if op == "linear":
        z = torch.einsum("nd,fd->nf", t["x"], t["w"])
        if t["bias"] is not None:
            z = z + t["bias"].unsqueeze(0)
        y = _act64(z, case["act"])[0]
        return [y if t["residual"] is None else y + t["residual"], z if case["save"] else None]
    dz = t["dy"] if t["z"] is None else t["dy"] * _act64(t["z"], case["act"])[1]
    return [torch.einsum("nf,fd->nd", dz, t["w"]), torch.einsum("nf,nd->fd", dz, t["x"]), dz.sum(0) if case["bias"] else None]
