"""64-bit definitions of the dense operators and the error bounds of their tests.

Bounds count roundings.  u = 2^-24 is half a step of fp32, h = 2^-8 half a step
of bf16 (torch.finfo(bfloat16).eps / 2), both relative to the rounded value.
  sums      a product of K terms accumulated in fp32 (the tensor core may
            truncate: one whole step, 2u, an addition) is off by at most
            2 K u sum|a b|
  act       the fast exponential is off by 2 + 1.173 |z| steps and the fast
            division by 2: below 2^-18 relative for |z| < 20; the slope, a sum of
            terms of size up to 1 + |z|, by 2^-18 (1 + |z|)
  slope     |act'| <= 1.2 for every activation here
"""
import math

import torch

U = 2.0 ** -24
H = 2.0 ** -8
ACT_EPS = 2.0 ** -18
LIP = 1.2

FNS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}
GAIN = math.sqrt(2 / math.pi)


def act(z, fn):
    if fn == "none":
        return z
    if fn == "relu":
        return z.clamp(min=0)
    if fn == "silu":
        return z * torch.sigmoid(z)
    if fn == "gelu":
        return 0.5 * z * torch.erfc(-z / math.sqrt(2))
    return z * torch.sigmoid(2 * GAIN * (z + 0.044715 * z ** 3))


def slope(z, fn):
    if fn == "none":
        return torch.ones_like(z)
    if fn == "relu":
        return (z > 0).to(z.dtype)
    if fn == "silu":
        p = torch.sigmoid(z)
        return p + z * p * (1 - p)
    if fn == "gelu":
        return 0.5 * torch.erfc(-z / math.sqrt(2)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    p = torch.sigmoid(2 * GAIN * (z + 0.044715 * z ** 3))
    return p + z * p * (1 - p) * 2 * GAIN * (1 + 3 * 0.044715 * z ** 2)


def f64(t):
    return None if t is None else t.double()


# ------------------------------------------------------------------ norm
def norm(x, weight, residual=None, eps=1e-6):
    s = f64(x) if residual is None else f64(x) + f64(residual)
    return s, s * f64(weight) * (s.square().mean(1, keepdim=True) + eps).rsqrt()


def norm_scale(y):
    """2^k of each row: the smallest k >= -126 with max|y| <= 448 2^k."""
    top = y.abs().amax(1)
    k = torch.full_like(top, -126.0)
    on = top > 448 * 2.0 ** -126
    k[on] = torch.ceil(torch.log2(top[on] / 448))
    return torch.exp2(k)


def norm_backward(dy, s, weight, dresidual=None, eps=1e-6):
    """(dx, dweight, bound of dx, bound of dweight)."""
    dy, s, w = f64(dy), f64(s), f64(weight)
    D = s.shape[1]
    r = (s.square().mean(1, keepdim=True) + eps).rsqrt()
    v = dy * w
    along = s * r ** 3 * (v * s).mean(1, keepdim=True)
    dx = r * v - along
    size = (r * v).abs() + s.abs() * r ** 3 * (v * s).abs().mean(1, keepdim=True)
    if dresidual is not None:
        dx = dx + f64(dresidual)
        size = size + f64(dresidual).abs()
    dweight = (dy * s * r).sum(0)
    return dx, dweight, H * dx.abs() + (D + 16) * 2 * U * size, (s.shape[0] + D + 16) * U * (dy * s * r).abs().sum(0)


# ------------------------------------------------------------------ products
def product(x, w):
    """(x w^T, its fp32 accumulation bound)."""
    x, w = f64(x), f64(w)
    return x @ w.T, 2 * (x.shape[1] + 2) * U * (x.abs() @ w.abs().T)


def gated(x, w1, w3, fn):
    """((h, bound), (g, bound), (u, bound))."""
    g, eg = product(x, w1)
    u, eu = product(x, w3)
    a = act(g, fn)
    ea = LIP * eg + ACT_EPS * g.abs()
    h = a * u
    return (h, H * h.abs() + ea * u.abs() + a.abs() * eu + ea * eu + 2 * U * h.abs()), (g, H * g.abs() + 2 * eg), (u, H * u.abs() + 2 * eu)


def gated_backward(dh, x, w1, w3, g, u, fn):
    """((dx, bound), (dw1, bound), (dw3, bound)): dg and du are rounded to bf16 before the products."""
    dh, x, w1, w3, g, u = map(f64, (dh, x, w1, w3, g, u))
    dg, du = dh * u * slope(g, fn), dh * act(g, fn)
    eg = 2 * H * dg.abs() + (dh * u).abs() * ACT_EPS * (1 + g.abs())
    eu = 2 * H * du.abs() + dh.abs() * ACT_EPS * g.abs()
    dx = dg @ w1 + du @ w3
    ex = eg @ w1.abs() + eu @ w3.abs() + 2 * (2 * g.shape[1] + 2) * U * (dg.abs() @ w1.abs() + du.abs() @ w3.abs())
    out = [(dx, 2 * H * dx.abs() + ex)]
    for d, e in ((dg, eg), (du, eu)):
        dw = d.T @ x
        out.append((dw, 2 * H * dw.abs() + e.T @ x.abs() + 2 * (x.shape[0] + 2) * U * (d.abs().T @ x.abs())))
    return out


def linear(x, w, bias, residual, fn):
    """((y, bound), (z, bound))."""
    z, ez = product(x, w)
    if bias is not None:
        z = z + f64(bias)
        ez = ez + 2 * U * z.abs()
    y = act(z, fn)
    e = LIP * ez + ACT_EPS * z.abs()
    if residual is not None:
        y = y + f64(residual)
        e = e + 2 * U * y.abs()
    return (y, H * y.abs() + 2 * e), (z, H * z.abs() + 2 * ez)


def linear_backward(dy, x, w, z, fn):
    """((dx, bound), (dw, bound), (dbias, bound))."""
    dy, x, w = map(f64, (dy, x, w))
    dz, e, eb = dy, 0 * dy, 0 * dy
    if fn != "none":
        z = f64(z)
        dz = dy * slope(z, fn)
        eb = dy.abs() * ACT_EPS * (1 + z.abs())
        e = 2 * H * dz.abs() + eb
    dx, dw, db = dz @ w, dz.T @ x, dz.sum(0)
    return ((dx, 2 * H * dx.abs() + e @ w.abs() + 2 * (w.shape[0] + 2) * U * (dz.abs() @ w.abs())),
            (dw, 2 * H * dw.abs() + e.T @ x.abs() + 2 * (x.shape[0] + 2) * U * (dz.abs().T @ x.abs())),
            (db, eb.sum(0) + 2 * (x.shape[0] + 2) * U * dz.abs().sum(0)))


def assert_within(got, ref, bound, name):
    got = got.double()
    assert got.shape == ref.shape, name
    off = (got - ref).abs()
    bad = ~(off <= bound + 1e-30)
    assert not bad.any(), (f"{name}: {int(bad.sum())} of {bad.numel()} outside, first at "
                           f"{tuple(bad.nonzero()[0].tolist())}: got {got[bad][0].item()}, want {ref[bad][0].item()}, "
                           f"bound {(bound + 0 * ref)[bad][0].item()}")
