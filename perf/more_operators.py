"""The routed layer's training operators, as cases to measure.

``combine_bwd``  gradient of the weighted sum back to token order: for assignment (t, k) with
                 row r = inv_perm[t,k], dy[r] = w[t,k] dout[t] and dw[t,k] = <dout[t], y[r]>;
``permute_bwd``  gradient of the sort by expert: dx[t] = dresidual[t] + sum_k dx_perm[inv_perm[t,k]];
``route_bwd``    gradient of the routing weights down to the router's logits, and of those to the
                 tokens, the gate and its bias;
``quant``        e4m3 codes with one power-of-two scale for each block of 128: 1 x 128 of an
                 activation ("rows"), 128 x 128 of a weight ("blocks"), and 1 x 128 together with
                 128 x 1 inside each expert's rows ("segments", what the weight gradient reads);
``block``        the experts' product in e4m3 with a scale for each block of 128 of both operands:
                 y[r,f] = sum_b sx[r,b] sw[e,f/128,b] sum_{d in block b} xq[r,d] wq[e,f,d];
``block_bwd``    its gradients: dx over blocks of f, dw over blocks of each expert's rows.

``run`` computes one of them on the inputs that ``prepare`` made: with ``own``
false in plain 32-bit torch operations, with ``own`` true through the package's
entry points.  ``exact`` is the definition in 64 bits.
"""
import math

import torch

own = False

B = 128  # length of a block that shares a scale


def listed():
    return [
        # The weighted sum's gradient in a training step at the DeepSeek-shaped layer.
        dict(name="combine_bwd_4096x7168", op="combine_bwd", n=4096, d=7168, e=256, k=8, skew=0.0),
        # The sort's gradient for a ragged batch of the Mixtral-shaped layer, added to the residual stream's.
        dict(name="permute_bwd_4093x4096", op="permute_bwd", n=4093, d=4096, e=8, k=2, skew=0.0, residual=True),
        # The router's gradient on a small batch (softmax over the chosen experts, with a bias).
        dict(name="route_bwd_100x2048x128", op="route_bwd", n=100, d=2048, e=128, k=8, skew=0.0, score="softmax",
             residual=False, bias=True),
        # The same in a large step with normalised sigmoid scores, added to what reached x otherwise.
        dict(name="route_bwd_4096x7168x256", op="route_bwd", n=4096, d=7168, e=256, k=8, skew=0.0, score="sigmoid",
             residual=True, bias=False),
        # The tokens of a ragged prefill batch before the experts.
        dict(name="quant_rows_1001x7168", op="quant", form="rows", rows=1001, d=7168),
        # Activations of a training step in both forms at once: for the product and for the weight gradient.
        dict(name="quant_segments_4093x4096", op="quant", form="segments", n=4093, d=4096, e=8, k=2, skew=0.0),
        # One token through a dense (shared) expert's projection: the weight stream and the launch.
        dict(name="block_1x7168x2048", op="block", n=1, d=7168, f=2048, e=1, k=1, skew=0.0),
        # A decode batch at the Qwen3-shaped layer: about one row an expert.
        dict(name="block_8x2048x768", op="block", n=8, d=2048, f=768, e=128, k=8, skew=0.0),
        # Prefill of the DeepSeek-shaped layer with favoured experts: ragged segments, all weights read.
        dict(name="block_4096x7168x2048", op="block", n=4096, d=7168, f=2048, e=256, k=8, skew=0.6),
        # Prefill of the Mixtral-shaped layer: few experts with many rows.
        dict(name="block_4096x4096x14336", op="block", n=4096, d=4096, f=14336, e=8, k=2, skew=0.0),
        # Both gradients on a small training batch of the Qwen3-shaped layer.
        dict(name="block_bwd_256x2048x768", op="block_bwd", n=256, d=2048, f=768, e=128, k=8, skew=0.0),
        # Both gradients on a ragged training batch of the Mixtral-shaped layer.
        dict(name="block_bwd_4093x4096x14336", op="block_bwd", n=4093, d=4096, f=14336, e=8, k=2, skew=0.0),
    ]


def _spread(rng, lo, hi, step):
    """A multiple of ``step`` in lo..hi, spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return min(hi, max(lo, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["combine_bwd", "permute_bwd", "route_bwd", "quant", "quant", "block", "block", "block", "block_bwd",
                     "block_bwd"])
    while True:
        e = rng.choice([1, 4, 8, 16, 60, 64, 128, 160, 256])
        c = dict(op=op, n=_spread(rng, 1, 8192, 1), d=_spread(rng, 256, 8192, 16), e=e,
                 k=min(e, rng.choice([1, 2, 4, 6, 8])), skew=rng.choice([0.0, 0.0, 0.6, 1.2]))
        n, d, k = c["n"], c["d"], c["k"]
        if op == "combine_bwd":
            if n * d * k <= 4096 * 7168 * 8:
                return c
        elif op == "permute_bwd":
            c["residual"] = rng.random() < 0.5
            if n * d * k <= 4096 * 7168 * 8:
                return c
        elif op == "route_bwd":
            c["e"], c["k"] = max(e, 4), max(k, 2)  # one choice has the weight 1 and no gradient
            c["score"], c["residual"], c["bias"] = rng.choice(["softmax", "sigmoid"]), rng.random() < 0.5, rng.random() < 0.5
            if n * d <= 4096 * 7168:
                return c
        elif op == "quant":
            c["form"] = rng.choice(["rows", "blocks", "segments"])
            if c["form"] == "rows":
                c = dict(op=op, form="rows", rows=n * k, d=d)
            elif c["form"] == "blocks":
                c = dict(op=op, form="blocks", e=rng.choice([1, 3, 8]), rows=_spread(rng, 64, 8192, 16), d=d)
            if c.get("rows", n * k) * c["d"] * (c["e"] if c["form"] == "blocks" else 1) <= 4096 * 7168 * 2:
                return c
        else:
            c["f"] = _spread(rng, 256, 14336, 16)
            limit = (2 * 32768 * 7168 * 2048, 256 * 7168 * 2048) if op == "block" else (4 * 8192 * 4096 * 14336, 8 * 4096 * 14336)
            if work(c)["flops"] <= limit[0] and e * d * c["f"] <= limit[1]:
                return c


def _blocks(v):
    return (v + B - 1) // B


def _segment_rows(rows, e):
    """Rows of the buffer whose segments start at multiples of 128: an upper bound for any routing."""
    return (rows + (B - 1) * min(e, rows)) // B * B


def work(case):
    op, d = case["op"], case["d"]
    if op == "quant":
        mats = case["e"] if case["form"] == "blocks" else 1
        rows = case.get("rows", case.get("n", 0) * case.get("k", 0)) * mats
        if case["form"] == "blocks":
            b = rows * d * 3 + 4 * rows * d // (B * B)
        elif case["form"] == "rows":
            b = rows * d * 3 + 4 * rows * _blocks(d)
        else:
            b = rows * d * 4 + 8 * rows * _blocks(d)
        return {"bytes": b, "flops": 2 * rows * d}
    n, k, e = case["n"], case["k"], case["e"]
    rows = n * k
    if op == "combine_bwd":
        return {"bytes": 2 * n * d + 4 * rows * d + 12 * rows, "flops": 3 * rows * d}
    if op == "permute_bwd":
        return {"bytes": 2 * rows * d + 2 * n * d * (1 + case["residual"]) + 4 * rows, "flops": rows * d}
    if op == "route_bwd":
        b = 2 * n * d * (2 + case["residual"]) + 4 * e * d + rows * 12 + (4 * rows if case["score"] == "sigmoid" else 0)
        return {"bytes": b, "flops": 4 * rows * d}
    f = case["f"]
    used = e * (1 - (1 - 1 / e) ** rows) if e > 1 else 1  # experts with rows
    codes = d + 4 * _blocks(d), f + 4 * _blocks(f)
    if op == "block":
        return {"bytes": int(rows * (codes[0] + 2 * f) + used * f * d), "flops": 2 * rows * d * f}
    return {"bytes": int(rows * (2 * codes[1] + codes[0] + 2 * d) + used * f * d + 2 * e * f * d), "flops": 4 * rows * d * f}


# ------------------------------------------------------------------ inputs
def _routing(case, gen, t):
    """Distinct experts for every token, best first; the sort's indices."""
    n, e, k = case["n"], case["e"], case["k"]
    dev = gen.device
    score = -torch.log(-torch.log(torch.rand((n, e), generator=gen, device=dev).clamp(1e-30, 1 - 1e-7)))
    score -= case["skew"] * torch.log(torch.arange(1, e + 1, device=dev, dtype=torch.float32))
    t["logits"], ids = score, torch.topk(score, k, dim=1).indices
    order = torch.sort(ids.flatten(), stable=True).indices
    inv = torch.empty_like(order)
    inv[order] = torch.arange(n * k, device=dev)
    counts = torch.bincount(ids.flatten(), minlength=e)
    t["ids"], t["inv"] = ids.to(torch.int32), inv.view(n, k).to(torch.int32)
    t["src"] = (order // k).to(torch.int32)
    t["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
    t["counts"] = counts.tolist()


def _codes(gen, *shape):
    """e4m3 codes as quantised normal values have them: the largest of a block is near the format's 448."""
    out = torch.empty(shape, dtype=torch.uint8, device=gen.device)
    for part in (out if len(shape) == 3 else out.unsqueeze(0)):
        v = torch.randn(part.shape, generator=gen, device=gen.device).mul_(140.0).clamp_(-448, 448)
        part.copy_(v.to(torch.float8_e4m3fn).view(torch.uint8))
    return out


def _scales(gen, size, *shape):
    """Scales of any value, as trained checkpoints carry them."""
    return torch.exp(0.4 * torch.randn(shape, generator=gen, device=gen.device)) * (size / 140.0)


def _inputs(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed) * 1_000_003 + 29)

    def normal(*shape, scale=1.0):
        return torch.randn(shape, generator=gen, device=dev).mul_(scale).to(torch.bfloat16)

    op, d, t = case["op"], case["d"], {}
    if "n" in case:
        _routing(case, gen, t)
    n, e, k = case.get("n"), case.get("e"), case.get("k")
    if op == "combine_bwd":
        t["dout"], t["y"] = normal(n, d, scale=0.05), normal(n * k, d)
        t["w"] = torch.softmax(torch.randn((n, k), generator=gen, device=dev), 1)
    elif op == "permute_bwd":
        t["dx_perm"] = normal(n * k, d, scale=0.05)
        t["dresidual"] = normal(n, d, scale=0.05) if case["residual"] else None
    elif op == "route_bwd":
        t["x"], t["w_gate"] = normal(n, d), normal(e, d, scale=d ** -0.5)
        chosen = torch.gather(t["logits"], 1, t["ids"].long())
        if case["score"] == "softmax":
            t["w"] = torch.softmax(chosen, 1)
        else:
            s = torch.sigmoid(chosen)
            t["w"] = s / s.sum(1, keepdim=True)
        t["dw"] = torch.randn((n, k), generator=gen, device=dev)
        t["dresidual"] = normal(n, d, scale=0.05) if case["residual"] else None
    elif op == "quant":
        rows = (case["e"], case["rows"]) if case["form"] == "blocks" else (case.get("rows") or n * k,)
        # channels and tokens of different size, as activations have them
        size = torch.exp(torch.randn((*rows, 1), generator=gen, device=dev))
        channel = torch.exp(0.7 * torch.randn(d, generator=gen, device=dev))
        t["src"] = (torch.randn((*rows, d), generator=gen, device=dev) * size * channel).to(torch.bfloat16)
    else:
        f, rows = case["f"], n * k
        t["wq"], t["w_scale"] = _codes(gen, e, f, d), _scales(gen, d ** -0.5, e, _blocks(f), _blocks(d))
        if op == "block":  # the sorted tokens' codes; their scales stay in token order
            t["xq"], t["x_scale"] = _codes(gen, rows, d), _scales(gen, 1.0, n, _blocks(d))
        else:
            t["dyq"], t["dy_scale"] = _codes(gen, rows, f), _scales(gen, 0.05, rows, _blocks(f))
            m = _segment_rows(rows, e)
            t["dyq_seg"], t["dy_scale_seg"] = _codes(gen, m, f), _scales(gen, 0.05, m // B, f)
            t["xq_seg"], t["x_scale_seg"] = _codes(gen, m, d), _scales(gen, 1.0, m // B, d)
            at = 0
            for c in t["counts"]:  # rows behind a segment are zero up to the next multiple of 128
                end = at + _blocks(c) * B
                t["dyq_seg"][at + c:end] = 0
                t["xq_seg"][at + c:end] = 0
                at = end
    return t


def prepare(case, seed):
    """The inputs, and the output buffers that a program keeps from step to step."""
    t = _inputs(case, seed)
    op, d = case["op"], case["d"]
    n, e, k, f = case.get("n", 0), case.get("e", 1), case.get("k", 1), case.get("f", 0)
    dev = torch.device("cuda")

    def buf(*shape, dtype=torch.bfloat16):
        return torch.zeros(shape, dtype=dtype, device=dev)

    if op == "combine_bwd":
        t["dy"], t["dw"] = buf(n * k, d), buf(n, k, dtype=torch.float32)
    elif op == "permute_bwd":
        t["dx"] = buf(n, d)
    elif op == "route_bwd":
        t["dx"], t["dw_gate"] = buf(n, d), buf(e, d)
        t["dbias"] = buf(e, dtype=torch.float32) if case["bias"] else None
    elif op == "quant":
        src, u8, f32 = t["src"], torch.uint8, torch.float32
        t["q"] = torch.zeros(src.shape, dtype=u8, device=dev)
        if case["form"] == "blocks":
            t["scale"] = buf(e, _blocks(case["rows"]), _blocks(d), dtype=f32)
        else:
            t["scale"] = buf(src.shape[0], _blocks(d), dtype=f32)
        if case["form"] == "segments":
            m = _segment_rows(n * k, e)
            t["q_seg"], t["scale_seg"] = buf(m, d, dtype=u8), buf(m // B, d, dtype=f32)
    elif op == "block":
        t["y_out"] = buf(n * k, f)
    else:
        t["dx"], t["dw"] = buf(n * k, d), buf(e, f, d)
    t["op"], t["case"] = op, case
    return t


# ------------------------------------------------------------------ the package's calls
def _handle(t):
    """The package and the workspace: made at a state's first call and kept with its buffers."""
    if "handle" not in t:
        from mixture_experts_layer_02_gb300 import moe
        name = {"combine_bwd": "combine", "permute_bwd": "combine", "route_bwd": "route_backward",
                "quant": "combine", "block": "grouped_linear_e4m3_block",
                "block_bwd": "grouped_linear_e4m3_block_backward"}[t["op"]]
        c = t["case"]
        rows = c.get("n", 0) * (1 if t["op"] == "route_bwd" else c.get("k", 1))
        t["handle"] = moe, moe.workspace(name, N=rows, D=c["d"], E=c.get("e", 1), K=c.get("k", 1), Dff=c.get("f", 0))
    return t["handle"]


def _run_own(t):
    (moe, ws), op, c = _handle(t), t["op"], t["case"]
    if op == "combine_bwd":
        return list(moe.moe_combine_backward(t["dout"], t["y"], t["inv"], t["w"], dy_perm=t["dy"], dtopk_w=t["dw"], ws=ws))
    if op == "permute_bwd":
        return [moe.moe_permute_backward(t["dx_perm"], t["inv"], dresidual=t["dresidual"], dx=t["dx"], ws=ws)]
    if op == "route_bwd":
        mode = moe.SOFTMAX_TOPK if c["score"] == "softmax" else moe.SIGMOID_NORM
        return list(moe.moe_route_backward(t["dw"], t["ids"], t["w"], t["logits"], t["x"], t["w_gate"], mode,
                                           dresidual=t["dresidual"], dx=t["dx"], dw_gate=t["dw_gate"], dbias=t["dbias"],
                                           ws=ws))
    if op == "quant":
        e4m3 = torch.float8_e4m3fn
        if c["form"] != "segments":
            q, scale = moe.moe_quantize_e4m3_block(t["src"], block_rows=B if c["form"] == "blocks" else 1, q=t["q"],
                                                   scale=t["scale"])
            return [q.view(e4m3), scale]
        q, scale, q_seg, scale_seg = moe.moe_quantize_e4m3_segments(t["src"], t["offsets"], q=t["q"], scale=t["scale"],
                                                                    q_seg=t["q_seg"], scale_seg=t["scale_seg"], ws=ws)
        return [q.view(e4m3), scale, q_seg.view(e4m3), scale_seg]
    if op == "block":
        one = c["e"] == 1  # a dense expert: no segments, scales in the rows' own order
        return [moe.moe_grouped_linear_e4m3_block(t["xq"], t["x_scale"], t["wq"], t["w_scale"],
                                                  expert_offsets=None if one else t["offsets"],
                                                  x_scale_index=None if one else t["src"], y=t["y_out"], ws=ws)]
    return list(moe.moe_grouped_linear_e4m3_block_backward(
        t["wq"], t["w_scale"], dyq=t["dyq"], dy_scale=t["dy_scale"], dyq_seg=t["dyq_seg"], dy_scale_seg=t["dy_scale_seg"],
        xq_seg=t["xq_seg"], x_scale_seg=t["x_scale_seg"], expert_offsets=t["offsets"], dx=t["dx"], dw=t["dw"], ws=ws))


# ------------------------------------------------------------------ plain form, 32 bits
def _values(q, scale, dim):
    """codes * scale, one scale for every 128 along ``dim`` (both, for the weights' blocks)."""
    s = scale
    for i in ((0, 1) if dim is None else (dim,)):
        s = s.repeat_interleave(B, i).narrow(i, 0, q.shape[i])
    return q.view(torch.float8_e4m3fn).float() * s


def _spans(counts, padded=False):
    """(expert, first row, last row + 1) of every segment, or with segments that start at multiples of 128."""
    at = 0
    for e, c in enumerate(counts):
        yield e, at, at + c
        at += _blocks(c) * B if padded else c


def _scale_of(top):
    """The smallest 2^k, k >= -126, with top <= 448 2^k: top = m 2^x, m in [0.5, 1)."""
    m, x = torch.frexp(top)
    k = torch.where(top > 0, x - 9 + (m > 0.875).int(), torch.full_like(x, -126)).clamp(min=-126)
    return torch.ldexp(torch.ones_like(top), k)


def _pad(v, dim):
    """Zeros up to a multiple of 128 along ``dim``."""
    short = -v.shape[dim] % B
    if not short:
        return v
    shape = list(v.shape)
    shape[dim] = short
    return torch.cat([v, v.new_zeros(shape)], dim)


def _quant_plain(v, rows, cols):
    """(codes, scales) of a matrix in blocks of rows x cols."""
    p = v
    if rows == B:
        p = _pad(p, 0)
    if cols == B:
        p = _pad(p, 1)
    tiles = p.view(p.shape[0] // rows, rows, p.shape[1] // cols, cols)
    scale = _scale_of(tiles.abs().amax((1, 3)))
    q = (tiles / scale[:, None, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    return q.view(torch.uint8).reshape(p.shape)[:v.shape[0], :v.shape[1]], scale


def _run_plain(t):
    bf16, op, c = torch.bfloat16, t["op"], t["case"]
    if op == "combine_bwd":
        n, k = c["n"], c["k"]
        dout, rows = t["dout"].float(), t["inv"].long().flatten()
        dy = torch.empty_like(t["y"])
        dw = torch.empty((n, k), device=dout.device)
        for j in range(k):
            r = t["inv"][:, j].long()
            dy[r] = (t["w"][:, j, None] * dout).to(bf16)
            dw[:, j] = (dout * t["y"][r].float()).sum(1)
        return [dy, dw]
    if op == "permute_bwd":
        dx = t["dx_perm"][t["inv"][:, 0].long()].float()
        for j in range(1, c["k"]):
            dx = dx + t["dx_perm"][t["inv"][:, j].long()].float()
        if t["dresidual"] is not None:
            dx = dx + t["dresidual"].float()
        return [dx.to(bf16)]
    if op == "route_bwd":
        w, dw, ids = t["w"], t["dw"], t["ids"].long()
        dl = w * (dw - (w * dw).sum(1, keepdim=True))
        if c["score"] == "sigmoid":
            dl = dl / (1 + torch.exp(torch.gather(t["logits"], 1, ids)))  # 1 - sigmoid
        full = torch.zeros_like(t["logits"]).scatter(1, ids, dl)
        dx = full @ t["w_gate"].float()
        if t["dresidual"] is not None:
            dx = dx + t["dresidual"].float()
        return [dx.to(bf16), (full.T @ t["x"].float()).to(bf16), full.sum(0) if t["dbias"] is not None else None]
    if op == "quant":
        e4m3, v = torch.float8_e4m3fn, t["src"].float()
        if c["form"] == "blocks":
            parts = [_quant_plain(m, B, B) for m in v]
            return [torch.stack([q for q, _ in parts]).view(e4m3), torch.stack([s for _, s in parts])]
        q, scale = _quant_plain(v, 1, B)
        if c["form"] == "rows":
            return [q.view(e4m3), scale]
        q_seg, scale_seg = torch.zeros_like(t["q_seg"]), torch.zeros_like(t["scale_seg"])
        for (_, a, b), (_, pa, _) in zip(_spans(t["counts"]), _spans(t["counts"], True)):
            if b > a:
                qs, s = _quant_plain(v[a:b], B, 1)
                q_seg[pa:pa + b - a] = qs
                scale_seg[pa // B:pa // B + s.shape[0]] = s
        return [q.view(e4m3), scale, q_seg.view(e4m3), scale_seg]
    if op == "block":
        scale = t["x_scale"] if c["e"] == 1 else t["x_scale"][t["src"].long()]
        x = _values(t["xq"], scale, 1)
        y = torch.empty((x.shape[0], c["f"]), dtype=bf16, device=x.device)
        for e, a, b in _spans(t["counts"]):
            if b > a:
                y[a:b] = (x[a:b] @ _values(t["wq"][e], t["w_scale"][e], None).T).to(bf16)
        return [y]
    dy = _values(t["dyq"], t["dy_scale"], 1)
    dx = torch.empty((dy.shape[0], c["d"]), dtype=bf16, device=dy.device)
    dw = torch.zeros((c["e"], c["f"], c["d"]), dtype=bf16, device=dy.device)
    for (e, a, b), (_, pa, _) in zip(_spans(t["counts"]), _spans(t["counts"], True)):
        if b > a:
            dx[a:b] = (dy[a:b] @ _values(t["wq"][e], t["w_scale"][e], None)).to(bf16)
            pb = pa + _blocks(b - a) * B
            left = _values(t["dyq_seg"][pa:pb], t["dy_scale_seg"][pa // B:pb // B], 0)
            dw[e] = (left.T @ _values(t["xq_seg"][pa:pb], t["x_scale_seg"][pa // B:pb // B], 0)).to(bf16)
    return [dx, dw]


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------ the definition, 64 bits
def _grid(scale, rows, cols, by_rows, by_cols):
    """scale[i // by_rows, j // by_cols] for every element of a rows x cols matrix."""
    i = torch.arange(rows, device=scale.device) // by_rows
    j = torch.arange(cols, device=scale.device) // by_cols
    return scale.double()[i][:, j]


def _real(q, scale, by_rows, by_cols):
    return q.view(torch.float8_e4m3fn).double() * _grid(scale, q.shape[0], q.shape[1], by_rows, by_cols)


def _scale64(v, by_rows, by_cols):
    """Scales of the blocks of a matrix: 2^ceil(log2(top / 448)), at least 2^-126; powers of two stay as they are."""
    i = torch.arange(v.shape[0], device=v.device) // by_rows
    j = torch.arange(v.shape[1], device=v.device) // by_cols
    top = v.new_zeros((int(i[-1]) + 1, v.shape[1])).index_reduce_(0, i, v.abs(), "amax")
    top = v.new_zeros((top.shape[0], int(j[-1]) + 1)).index_reduce_(1, j, top, "amax")
    half, power = torch.frexp(top.clamp(min=448 * 2.0 ** -126) / 448)  # half in [0.5, 1)
    return torch.ldexp(torch.where(half == 0.5, 0.5, 1.0).to(top), power)


def exact(case, seed):
    t = _inputs(case, seed)
    op = case["op"]
    if op == "combine_bwd":
        dout, y, w, rows = t["dout"].double(), t["y"].double(), t["w"].double(), t["inv"].long().flatten()
        token = torch.arange(case["n"], device=rows.device).repeat_interleave(case["k"])
        dy = torch.empty_like(y).index_copy_(0, rows, w.reshape(-1, 1) * dout[token])
        return [dy, torch.einsum("ad,ad->a", dout[token], y[rows]).view(case["n"], case["k"])]
    if op == "permute_bwd":
        token = torch.empty(case["n"] * case["k"], dtype=torch.long, device=t["inv"].device)
        token[t["inv"].long().flatten()] = torch.arange(case["n"], device=token.device).repeat_interleave(case["k"])
        dx = torch.zeros((case["n"], case["d"]), dtype=torch.float64, device=token.device)
        dx.index_add_(0, token, t["dx_perm"].double())
        return [dx if t["dresidual"] is None else dx + t["dresidual"].double()]
    if op == "route_bwd":
        w, dw, ids = t["w"].double(), t["dw"].double(), t["ids"].long()
        jac = torch.diag_embed(w) - w.unsqueeze(2) * w.unsqueeze(1)
        dl = torch.einsum("nk,nkj->nj", dw, jac)
        if case["score"] == "sigmoid":
            dl = dl * torch.sigmoid(-torch.gather(t["logits"].double(), 1, ids))
        one = torch.nn.functional.one_hot(ids, case["e"]).double()
        full = torch.einsum("nk,nke->ne", dl, one)
        dx = torch.einsum("ne,ed->nd", full, t["w_gate"].double())
        if t["dresidual"] is not None:
            dx = dx + t["dresidual"].double()
        return [dx, torch.einsum("ne,nd->ed", full, t["x"].double()), full.sum(0) if case["bias"] else None]
    if op == "quant":
        v, form = t["src"].double(), case["form"]
        if form == "blocks":
            scale = torch.stack([_scale64(m, B, B) for m in v])
            return [torch.stack([m / _grid(s, *m.shape, B, B) for m, s in zip(v, scale)]), scale]
        scale = _scale64(v, 1, B)
        out = [v / _grid(scale, *v.shape, 1, B), scale]
        if form == "segments":
            m = _segment_rows(v.shape[0], case["e"])
            q, s = v.new_zeros((m, v.shape[1])), v.new_zeros((m // B, v.shape[1]))
            row = at = 0
            for c in t["counts"]:
                if c:
                    part = v[row:row + c]
                    own_scale = _scale64(part, B, 1)
                    q[at:at + c] = part / _grid(own_scale, *part.shape, B, 1)
                    s[at // B:at // B + own_scale.shape[0]] = own_scale
                row, at = row + c, at + _blocks(c) * B
            out += [q, s]
        return out
    d, f = case["d"], case["f"]
    first = [0]
    for c in t["counts"]:
        first.append(first[-1] + c)
    if op == "block":
        y = torch.empty((first[-1], f), dtype=torch.float64, device=t["xq"].device)
        token = t["src"].long()
        for e, (a, b) in enumerate(zip(first, first[1:])):
            if b > a:
                x = _real(t["xq"][a:b], t["x_scale"][token[a:b]], 1, B)
                y[a:b] = torch.einsum("rd,fd->rf", x, _real(t["wq"][e], t["w_scale"][e], B, B))
        return [y]
    dx = torch.empty((first[-1], d), dtype=torch.float64, device=t["dyq"].device)
    dw = torch.zeros((case["e"], f, d), dtype=torch.float64, device=dx.device)
    at = 0
    for e, (a, b) in enumerate(zip(first, first[1:])):
        if b > a:
            dx[a:b] = torch.einsum("rf,fd->rd", _real(t["dyq"][a:b], t["dy_scale"][a:b], 1, B),
                                   _real(t["wq"][e], t["w_scale"][e], B, B))
            end = at + _blocks(b - a) * B
            dw[e] = torch.einsum("rf,rd->fd", _real(t["dyq_seg"][at:end], t["dy_scale_seg"][at // B:end // B], B, 1),
                                 _real(t["xq_seg"][at:end], t["x_scale_seg"][at // B:end // B], B, 1))
            at = end
    return [dx, dw]
