"""64-bit definitions of the routed layer's training operators and the error bounds of their tests.

Bounds count roundings, as in dense_reference: U = 2^-24 is half a step of fp32, H = 2^-8 of bf16 (both relative).
  sums      of n fp32 terms in any order: n U sum|terms|
  blocks    a block's 128 products of e4m3 values are exact and are added by the tensor core, which may truncate (one
            whole step, 2U, an addition); the scale of both sides is one fp32 product, and each block's multiply-add
            rounds once: (2 * 130 + blocks + 4) U sum|x w| for a sum over `blocks` blocks
  route     c = sum_k w_k d_k has K products and additions, d - c, its product with w and the sigmoid's slope
            (exponential within 2 steps, quotient within half a step) a few more: (K + 12) U |w| (|d| + sum|w d|)
"""
import torch

from dense_reference import H, U

B = 128


def blocks(n):
    return -(-n // B)


def segment_rows(rows, E):
    return (rows + (B - 1) * min(rows, E)) // B * B


# ------------------------------------------------------------------ sort, weighted sum, router
def combine_backward(dout, y, inv, w):
    """((dy by row, bound), (dw, bound), rows that are named)."""
    dout, y, w = dout.double(), y.double(), w.double()
    dy, named = torch.zeros_like(y), torch.zeros(y.shape[0], dtype=torch.bool, device=y.device)
    dw, ew = torch.zeros_like(w), torch.zeros_like(w)
    for t in range(inv.shape[0]):
        for k in range(inv.shape[1]):
            r = int(inv[t, k])
            if 0 <= r < y.shape[0]:
                dy[r], named[r] = w[t, k] * dout[t], True
                dw[t, k] = dout[t] @ y[r]
                ew[t, k] = (y.shape[1] + 2) * U * (dout[t].abs() @ y[r].abs())
    return (dy, (H + 2 * U) * dy.abs()), (dw, ew), named


def permute_backward(dx_perm, inv, dresidual):
    """(dx, bound)."""
    src = dx_perm.double()
    dx = torch.zeros((inv.shape[0], src.shape[1]), dtype=torch.float64, device=src.device)
    size = torch.zeros_like(dx)
    if dresidual is not None:
        dx, size = dx + dresidual.double(), size + dresidual.double().abs()
    for t in range(inv.shape[0]):
        for r in inv[t].tolist():
            if 0 <= r < src.shape[0]:
                dx[t] += src[r]
                size[t] += src[r].abs()
    return dx, H * dx.abs() + 2 * (inv.shape[1] + 1) * U * size


def route_backward(dw, ids, w, logits, x, w_gate, sigmoid, dresidual):
    """((dx, bound), (dw_gate, bound), (dbias, bound))."""
    E, K = w_gate.shape[0], ids.shape[1]
    d, w, i = dw.double(), w.double(), ids.long()
    on = (i >= 0) & (i < E)
    i = i.clamp(0, E - 1)
    c = (w * d * on).sum(1, keepdim=True)
    dl = w * (d - c) * on
    err = (K + 12) * U * w.abs() * (d.abs() + (w * d * on).abs().sum(1, keepdim=True)) * on
    if sigmoid:
        q = torch.sigmoid(-torch.gather(logits.double(), 1, i))
        dl, err = dl * q, err * q
    full = torch.zeros((x.shape[0], E), dtype=torch.float64, device=x.device).scatter_add(1, i, dl)
    e_full = torch.zeros_like(full).scatter_add(1, i, err + K * U * dl.abs())
    e_bf = e_full + H * full.abs() + H * e_full
    xd, g = x.double(), w_gate.double()
    dx = full @ g
    e_dx = e_bf @ g.abs() + 2 * (E + 2) * U * (full.abs() @ g.abs())
    if dresidual is not None:
        dx = dx + dresidual.double()
        e_dx = e_dx + 2 * U * dx.abs()
    dg = full.T @ xd
    e_dg = e_bf.T @ xd.abs() + 2 * (x.shape[0] + 2) * U * (full.abs().T @ xd.abs())
    return ((dx, 2 * H * dx.abs() + e_dx * 2), (dg, 2 * H * dg.abs() + e_dg * 2),
            (full.sum(0), e_full.sum(0) + (x.shape[0] + 2) * U * full.abs().sum(0)))


# ------------------------------------------------------------------ e4m3 with a scale for each block of 128
def scale_of(top):
    """The smallest 2^k, k >= -126, with top <= 448 2^k (float64)."""
    half, power = torch.frexp(top.clamp(min=448 * 2.0 ** -126) / 448)
    return torch.ldexp(torch.where(half == 0.5, 0.5, 1.0).to(top), power)


def spread(scale, shape, by_rows, by_cols):
    s = scale.repeat_interleave(by_rows, 0)[:shape[0]].repeat_interleave(by_cols, 1)[:, :shape[1]]
    return s.double()


def quantize(v, by_rows, by_cols):
    """(codes uint8, scale fp32) of a matrix, as the rule says; x 2^-k is exact, so the one rounding is the cast's."""
    rows, cols = v.shape
    v = v.float()
    pad = torch.zeros((-(-rows // by_rows) * by_rows, -(-cols // by_cols) * by_cols), device=v.device)
    pad[:rows, :cols] = v.abs()
    top = pad.view(pad.shape[0] // by_rows, by_rows, pad.shape[1] // by_cols, by_cols).amax((1, 3)).double()
    scale = scale_of(top)
    q = (v.double() / spread(scale, v.shape, by_rows, by_cols)).clamp(-448, 448).float().to(torch.float8_e4m3fn)
    return q.view(torch.uint8), scale.float()


def values(q, scale, by_rows, by_cols):
    return q.view(torch.float8_e4m3fn).double() * spread(scale, q.shape, by_rows, by_cols)


def spans(counts):
    """(expert, first row, last + 1, first padded row, last padded + 1)."""
    at = pad = 0
    for e, c in enumerate(counts):
        yield e, at, at + c, pad, pad + blocks(c) * B
        at, pad = at + c, pad + blocks(c) * B


def bound(ref, size, nb):
    return H * ref.abs() + 2 * (2 * 130 + nb + 4) * U * size


def product(xq, xs, wq, ws, counts):
    """(y, bound) of the rows that belong to an expert; xs has one row a row."""
    x = values(xq, xs, 1, B)
    y = torch.zeros((sum(counts), wq.shape[1]), dtype=torch.float64, device=x.device)
    size = torch.zeros_like(y)
    for e, a, b, _, _ in spans(counts):
        w = values(wq[e], ws[e], B, B)
        y[a:b], size[a:b] = x[a:b] @ w.T, x[a:b].abs() @ w.abs().T
    return y, bound(y, size, blocks(x.shape[1]))


def product_backward(dyq, dys, dyq_seg, dys_seg, xq_seg, xs_seg, wq, ws, counts):
    """((dx, bound), (dw, bound))."""
    dy = values(dyq, dys, 1, B)
    E, F, D = wq.shape
    dx = torch.zeros((sum(counts), D), dtype=torch.float64, device=dy.device)
    sx = torch.zeros_like(dx)
    dw = torch.zeros((E, F, D), dtype=torch.float64, device=dy.device)
    sw = torch.zeros_like(dw)
    for e, a, b, pa, pb in spans(counts):
        w = values(wq[e], ws[e], B, B)
        dx[a:b], sx[a:b] = dy[a:b] @ w, dy[a:b].abs() @ w.abs()
        left = values(dyq_seg[pa:pb], dys_seg[pa // B:pb // B], B, 1)
        right = values(xq_seg[pa:pb], xs_seg[pa // B:pb // B], B, 1)
        dw[e], sw[e] = left.T @ right, left.abs().T @ right.abs()
    return (dx, bound(dx, sx, blocks(F))), (dw, bound(dw, sw, blocks(max(counts + [1]))))
