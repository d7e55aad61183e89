"""The dense operators on the GPU against their 64-bit definitions."""
import pytest
import torch

import dense_reference as R
from dense_reference import assert_within

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def moe(cuda_device):
    from mixture_experts_layer_02_gb300 import moe
    moe.load()
    return moe


def randn(*shape, seed=0, scale=1.0, dtype=BF16):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + sum((i + 1) * n for i, n in enumerate(shape)))
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


class Guarded:
    """Buffers between two guard zones; check() fails if a zone was written."""

    def __init__(self):
        self.all = []

    def __call__(self, *shape, dtype=BF16):
        n = 1
        for s in shape:
            n *= s
        size = torch.empty((), dtype=dtype).element_size()
        raw = torch.full((n * size + 2048,), 0xA5, dtype=torch.uint8, device="cuda")
        self.all.append((raw, n * size))
        return raw[1024:1024 + n * size].view(dtype).view(shape)

    def check(self):
        for raw, n in self.all:
            assert (raw[:1024] == 0xA5).all() and (raw[1024 + n:] == 0xA5).all(), "a guard zone was written"


# ------------------------------------------------------------------ norm
NORM_SHAPES = [(1, 8), (3, 64), (1, 7168), (7, 7168), (33, 264), (9, 1000), (130, 2048), (5, 4096), (3, 8200), (2, 16384),
               (2, 16392), (3, 32768), (700, 512)]


@pytest.mark.parametrize("n,d", NORM_SHAPES)
@pytest.mark.parametrize("residual", [False, True])
def test_norm(moe, n, d, residual):
    x, w = randn(n, d, seed=1), randn(d, seed=2) + 1
    res = randn(n, d, seed=3, scale=3.0) if residual else None
    if n > 1:
        x[1] = 0  # a padding row
        if residual:
            res[1] = 0
    b = Guarded()
    y, yq, scale, out = moe.moe_rmsnorm(x, w, residual=res, y=b(n, d), yq=b(n, d, dtype=torch.uint8),
                                        y_scale=b(n, dtype=torch.float32), residual_out=b(n, d) if residual else None)
    b.check()
    s, ref = R.norm(x, w, res)
    slack = (d + 16) * R.U
    assert_within(y, ref, (R.H + slack) * ref.abs(), "y")
    if residual:
        assert torch.equal(out, s.float().to(BF16)), "residual_out"
    else:
        assert out is None
    # the scale: exact wherever the row's maximum is not within fp32 rounding of a border
    want = R.norm_scale(ref)
    top = ref.abs().amax(1)
    near = (top / (448 * want) - 1).abs().minimum((top / (224 * want) - 1).abs()) <= slack
    assert torch.equal(scale.double()[~near], want[~near]), "y_scale"
    on = ref / scale.double()[:, None]
    codes = yq.view(torch.float8_e4m3fn).float()
    assert_within(codes, on.clamp(-448, 448), 2.0 ** -4 * on.abs() + 2.0 ** -10 + slack * on.abs(), "yq")


def test_norm_codes_alone_and_in_place(moe):
    x, w, res = randn(5, 1024, seed=1), randn(1024, seed=2), randn(5, 1024, seed=3)
    y, yq, scale, s = moe.moe_rmsnorm(x, w, residual=res, quantize=True)
    keep = res.clone()
    y2, yq2, scale2, s2 = moe.moe_rmsnorm(x, w, residual=keep, quantize=True, residual_out=keep)
    assert s2 is keep
    for a, b in ((y, y2), (yq, yq2), (scale, scale2), (s, s2)):
        assert torch.equal(a, b)
    L = moe.load()
    q3, sc3 = torch.zeros_like(yq), torch.zeros_like(scale)
    assert L.moe_rmsnorm(x.data_ptr(), res.data_ptr(), w.data_ptr(), 5, 1024, 1e-6, None, q3.data_ptr(), sc3.data_ptr(),
                         None, torch.cuda.current_stream().cuda_stream) == 0
    assert torch.equal(q3, yq) and torch.equal(sc3, scale)


def test_norm_codes_feed_the_e4m3_permutation(moe):
    """The codes and scales are what the e4m3 path takes: near the quantised bf16 rows, and permuted as bytes."""
    x, w = randn(40, 256, seed=1), randn(256, seed=2) + 1
    y, yq, scale, _ = moe.moe_rmsnorm(x, w, quantize=True)
    q2, s2 = moe.moe_quantize_e4m3(y)
    same = (scale == s2)
    assert same.float().mean() > 0.9  # a row whose maximum sits on a border may take the next scale
    a, b = yq.view(torch.float8_e4m3fn).float()[same], q2.view(torch.float8_e4m3fn).float()[same]
    # each is within half an e4m3 step of y / scale, the second after a bf16 rounding
    assert ((a - b).abs() <= 2 * (2.0 ** -4 + R.H) * torch.maximum(a.abs(), b.abs()) + 2.0 ** -9).all()
    ids = torch.randint(0, 4, (40, 1), device="cuda", dtype=torch.int32)
    off, src, inv, rows = moe.moe_permute_e4m3(yq, ids, 4)
    assert torch.equal(rows, yq[src.long()])


def test_norm_nonfinite_rows_stay_alone(moe):
    x, w = randn(6, 520, seed=1), randn(520, seed=2)
    x[2, 5] = float("nan")
    x[4, 100] = float("inf")
    clean = randn(6, 520, seed=1)
    y, yq, scale, _ = moe.moe_rmsnorm(x, w, quantize=True)
    y0, yq0, scale0, _ = moe.moe_rmsnorm(clean, w, quantize=True)
    for r in (0, 1, 3, 5):
        assert torch.equal(y[r], y0[r]) and torch.equal(yq[r], yq0[r]) and scale[r] == scale0[r]
    assert y[2].isnan().all() and y[4, 100].isnan() and (yq[2] & 0x7F == 0x7F).all()


@pytest.mark.parametrize("n,d", NORM_SHAPES + [(1500, 7168)])
@pytest.mark.parametrize("down", [False, True])
def test_norm_backward(moe, n, d, down):
    dy, s, w = randn(n, d, seed=1, scale=0.1), randn(n, d, seed=2, scale=2.0), randn(d, seed=3) + 1
    dres = randn(n, d, seed=4, scale=0.1) if down else None
    if n > 1:
        s[1] = 0
    b = Guarded()
    dx, dw = moe.moe_rmsnorm_backward(dy, s, w, dresidual=dres, dx=b(n, d), dweight=b(d, dtype=torch.float32))
    b.check()
    rx, rw, ex, ew = R.norm_backward(dy, s, w, dres)
    assert_within(dx, rx, ex, "dx")
    assert_within(dw, rw, ew, "dweight")


# ------------------------------------------------------------------ products
#: rows, in, out: one row, tails of every dimension, widths below a tile, several tiles
SHAPES = [(1, 8, 8), (1, 2048, 768), (3, 72, 200), (8, 1000, 264), (9, 1024, 40), (17, 264, 1032), (33, 520, 72), (64, 512, 512),
          (127, 64, 136), (128, 1024, 256), (129, 2056, 328), (300, 776, 520), (513, 136, 1288), (700, 4104, 400)]


#: the plan's choice; one-CTA tiles and pair tiles (bn * 10) with parts of K; persistent pairs; two pairs that share an operand
KERNELS = {"plan": {}} | {f"split{c}": dict(KERNEL="1", SPLIT=c) for c in ("1", "2", "8", "1281", "1282", "1284", "2561", "2562", "2564")} | {
           "pair": dict(KERNEL="2", CLUSTER="2"), "pairs4": dict(KERNEL="2", CLUSTER="4")}


@pytest.fixture(params=list(KERNELS))
def splits(request, monkeypatch):
    for k, v in KERNELS[request.param].items():
        monkeypatch.setenv("MOE_DENSE_" + k, v)
    return request.param


@pytest.mark.parametrize("n,d,f", SHAPES)
def test_gated(moe, splits, n, d, f):
    x, w1, w3 = randn(n, d, seed=1), randn(f, d, seed=2, scale=d ** -0.5), randn(f, d, seed=3, scale=d ** -0.5)
    b = Guarded()
    ws = moe.workspace("gated_linear", N=n, D=d, Dff=f)
    h, g, u = moe.moe_gated_linear(x, w1, w3, h=b(n, f), g=b(n, f), u=b(n, f), ws=ws)
    b.check()
    assert moe.read_device_error(ws) == moe.MOE_OK
    for got, (ref, bound), name in zip((h, g, u), R.gated(x, w1, w3, "silu"), "hgu"):
        assert_within(got, ref, bound, name)
    h2, g2, u2 = moe.moe_gated_linear(x, w1, w3, ws=ws)
    assert g2 is None and u2 is None and torch.equal(h, h2)


@pytest.mark.parametrize("fn", ["none", "relu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("n", [2, 50, 300])
def test_gated_activations(moe, fn, n):
    x, w1, w3 = randn(n, 136, seed=1), randn(72, 136, seed=2, scale=0.3), randn(72, 136, seed=3, scale=0.1)
    h, _, _ = moe.moe_gated_linear(x, w1, w3, R.FNS[fn])
    ref, bound = R.gated(x, w1, w3, fn)[0]
    assert_within(h, ref, bound, fn)


@pytest.mark.parametrize("n,d,f", SHAPES)
@pytest.mark.parametrize("extra", [False, True])
def test_linear(moe, splits, n, d, f, extra):
    x, w = randn(n, d, seed=1), randn(f, d, seed=2, scale=d ** -0.5)
    bias = randn(f, seed=3, dtype=torch.float32) if extra else None
    res = randn(n, f, seed=4) if extra else None
    fn = "gelu" if extra else "none"
    b = Guarded()
    y, z = moe.moe_linear(x, w, bias=bias, residual=res, fn=R.FNS[fn], y=b(n, f), z=b(n, f))
    b.check()
    (ry, ey), (rz, ez) = R.linear(x, w, bias, res, fn)
    assert_within(y, ry, ey, "y")
    assert_within(z, rz, ez, "z")


@pytest.mark.parametrize("fn", sorted(R.FNS))
@pytest.mark.parametrize("n", [1, 40, 300])
@pytest.mark.parametrize("bias,residual", [(False, False), (True, False), (False, True), (True, True)])
def test_linear_epilogues(moe, fn, n, bias, residual):
    x, w = randn(n, 200, seed=1), randn(136, 200, seed=2, scale=0.2)
    bias = randn(136, seed=3, dtype=torch.float32) if bias else None
    res = randn(n, 136, seed=4) if residual else None
    y, z = moe.moe_linear(x, w, bias=bias, residual=res, fn=R.FNS[fn])
    assert z is None
    (ry, ey), _ = R.linear(x, w, bias, res, fn)
    assert_within(y, ry, ey, "y")
    if residual:  # in place
        keep = res.clone()
        y2, _ = moe.moe_linear(x, w, bias=bias, residual=keep, fn=R.FNS[fn], y=keep)
        assert y2 is keep and torch.equal(y, y2)


@pytest.mark.parametrize("n,d,f", SHAPES)
def test_gated_backward(moe, splits, n, d, f):
    x, w1, w3 = randn(n, d, seed=1), randn(f, d, seed=2, scale=d ** -0.5), randn(f, d, seed=3, scale=d ** -0.5)
    g, u, dh = randn(n, f, seed=4), randn(n, f, seed=5), randn(n, f, seed=6, scale=0.1)
    b = Guarded()
    ws = moe.workspace("gated_linear_backward", N=n, D=d, Dff=f)
    got = moe.moe_gated_linear_backward(dh, x, w1, w3, g, u, dx=b(n, d), dw1=b(f, d), dw3=b(f, d), ws=ws)
    b.check()
    assert moe.read_device_error(ws) == moe.MOE_OK
    for t, (ref, bound), name in zip(got, R.gated_backward(dh, x, w1, w3, g, u, "silu"), ("dx", "dw1", "dw3")):
        assert_within(t, ref, bound, name)


@pytest.mark.parametrize("n,d,f", SHAPES)
@pytest.mark.parametrize("fn", ["none", "gelu"])
def test_linear_backward(moe, splits, n, d, f, fn):
    x, w, dy = randn(n, d, seed=1), randn(f, d, seed=2, scale=d ** -0.5), randn(n, f, seed=3, scale=0.1)
    z = randn(n, f, seed=4) if fn != "none" else None
    b = Guarded()
    got = moe.moe_linear_backward(dy, x, w, z=z, fn=R.FNS[fn], dx=b(n, d), dw=b(f, d), dbias=b(f, dtype=torch.float32))
    b.check()
    for t, (ref, bound), name in zip(got, R.linear_backward(dy, x, w, z, fn), ("dx", "dw", "dbias")):
        assert_within(t, ref, bound, name)


@pytest.mark.parametrize("fn", sorted(R.FNS))
def test_activation_slopes(moe, fn):
    n, d, f = 40, 64, 136
    x, w, dy = randn(n, d, seed=1), randn(f, d, seed=2, scale=0.2), randn(n, f, seed=3, scale=0.1)
    z = randn(n, f, seed=4, scale=3.0)
    got = moe.moe_linear_backward(dy, x, w, z=z, fn=R.FNS[fn], need_dbias=True)
    for t, (ref, bound), name in zip(got, R.linear_backward(dy, x, w, z, fn), ("dx", "dw", "dbias")):
        assert_within(t, ref, bound, name)
    u = randn(n, f, seed=5)
    w3 = randn(f, d, seed=6, scale=0.2)
    got = moe.moe_gated_linear_backward(dy, x, w, w3, z, u, fn=R.FNS[fn])
    for t, (ref, bound), name in zip(got, R.gated_backward(dy, x, w, w3, z, u, fn), ("dx", "dw1", "dw3")):
        assert_within(t, ref, bound, name)


@pytest.mark.parametrize("fn", sorted(R.FNS))
def test_slopes_in_fp32(moe, fn):
    """One row: dbias is the fp32 slope itself, over the whole range of z."""
    z = torch.linspace(-18, 18, 16384, device="cuda").to(BF16)[None]
    f = z.shape[1]
    x, w, dy = torch.ones(1, 8, device="cuda", dtype=BF16), torch.zeros(f, 8, device="cuda", dtype=BF16), torch.ones_like(z)
    _, _, db = moe.moe_linear_backward(dy, x, w, z=z, fn=R.FNS[fn], need_dbias=True)
    assert_within(db, R.slope(z.double(), fn)[0], R.ACT_EPS * (1 + z.double().abs())[0], fn)
    # the value, through the gated product's gradient du = dh fn(g), whose sums over one row are the values in bf16
    got = moe.moe_gated_linear_backward(dy, x, w, w, z, torch.zeros_like(z), R.FNS[fn])[2]
    ref = R.act(z.double(), fn)[0][:, None].expand(f, 8)
    assert_within(got, ref, 4 * R.H * ref.abs() + R.ACT_EPS * z.double().abs()[0][:, None], fn)


def test_extreme_pre_activations(moe):
    """Slopes far out: 0 or 1, never NaN, for every activation."""
    z = torch.tensor([[-3e38, -1e30, -200.0, -90.0, 90.0, 200.0, 1e30, 3e38]], device="cuda").to(BF16)
    x, w, dy = torch.ones(1, 8, device="cuda", dtype=BF16), torch.eye(8, device="cuda", dtype=BF16), torch.ones_like(z)
    for fn in sorted(R.FNS):
        dx, dw, db = moe.moe_linear_backward(dy, x, w, z=z, fn=R.FNS[fn], need_dbias=True)
        want = R.slope(z.double(), fn)  # at -90 the slope is -89 e^-90, not 0
        assert_within(dx, want, (2 * R.H + R.ACT_EPS) * want.abs(), fn)
        want = R.act(z.double(), fn)
        assert_within(moe.moe_linear(z, w, fn=R.FNS[fn])[0], want, (R.H + R.ACT_EPS) * want.abs(), fn)


@pytest.mark.parametrize("n", [4, 40, 300])
def test_nonfinite_rows_stay_alone(moe, n):
    """NaN in one token reaches that token's outputs only, also through the tails of K and M."""
    x, w1, w3 = randn(n, 200, seed=1), randn(136, 200, seed=2, scale=0.1), randn(136, 200, seed=3, scale=0.1)
    clean = moe.moe_gated_linear(x, w1, w3)[0]
    lin = moe.moe_linear(x, w1)[0]
    bad = x.clone()
    bad[n // 2] = float("nan")
    h, y = moe.moe_gated_linear(bad, w1, w3)[0], moe.moe_linear(bad, w1)[0]
    keep = torch.arange(n, device="cuda") != n // 2
    assert torch.equal(h[keep], clean[keep]) and torch.equal(y[keep], lin[keep])
    assert h[n // 2].isnan().all() and y[n // 2].isnan().all()


# ------------------------------------------------------------------ streams, graphs, repeats, empty calls
def _step(moe, t, stream=None):
    y, yq, scale, s = moe.moe_rmsnorm(t["x"], t["weight"], residual=t["res"], quantize=True, stream=stream)
    h, g, u = moe.moe_gated_linear(y, t["w1"], t["w3"], save=True, stream=stream)
    out, _ = moe.moe_linear(h, t["w2"], residual=s, stream=stream)
    dh, dw2, _ = moe.moe_linear_backward(t["dout"], h, t["w2"], stream=stream)
    dy, dw1, dw3 = moe.moe_gated_linear_backward(dh, y, t["w1"], t["w3"], g, u, stream=stream)
    dx, dweight = moe.moe_rmsnorm_backward(dy, s, t["weight"], dresidual=t["dout"], stream=stream)
    return [y, yq, scale, s, h, out, dx, dweight, dw1, dw3, dw2]


def _tensors(n=70, d=264, f=520):
    return dict(x=randn(n, d, seed=1), res=randn(n, d, seed=2), weight=randn(d, seed=3) + 1, dout=randn(n, d, seed=4, scale=0.1),
                w1=randn(f, d, seed=5, scale=d ** -0.5), w3=randn(f, d, seed=6, scale=d ** -0.5),
                w2=randn(d, f, seed=7, scale=f ** -0.5))


@pytest.mark.parametrize("n", [1, 70, 600])
def test_repeats_are_bitwise_equal(moe, n):
    t = _tensors(n)
    first = _step(moe, t)
    for _ in range(3):
        for a, b in zip(first, _step(moe, t)):
            assert torch.equal(a, b)


def test_another_stream(moe):
    t = _tensors()
    want = _step(moe, t)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = _step(moe, t, stream=side)
    side.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)


def test_graph_capture(moe):
    t = _tensors()
    want = _step(moe, t)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = _step(moe, t)
    for o in got:
        o.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    t["x"].copy_(randn(70, 264, seed=9))  # replays read the new inputs
    graph.replay()
    torch.cuda.synchronize()
    again = [o.clone() for o in got]
    for a, b in zip(_step(moe, t), again):
        assert torch.equal(a, b)


def test_binding_refuses_shapes_and_strides(moe):
    x, w, wf = randn(4, 64, seed=1), randn(64, seed=2), randn(40, 64, seed=3)
    with pytest.raises(ValueError, match="shape"):
        moe.moe_rmsnorm(x, w[:32].contiguous())
    with pytest.raises(ValueError, match="contiguous"):
        moe.moe_linear(randn(64, 4).T, wf)
    with pytest.raises(ValueError, match="shape"):
        moe.moe_gated_linear(x, wf, wf[:32])
    with pytest.raises(ValueError, match="contiguous"):
        moe.moe_rmsnorm(randn(4, 128)[:, :64], w)
    with pytest.raises(moe.MoEError, match="multiple of 8"):
        moe.moe_linear(randn(4, 12), randn(8, 12))
    with pytest.raises(moe.MoEError, match="16-byte aligned"):
        moe.moe_linear(randn(257)[1:].view(4, 64), wf)


def test_no_rows(moe):
    d, f = 64, 128
    e = torch.empty(0, d, device="cuda", dtype=BF16)
    ef = torch.empty(0, f, device="cuda", dtype=BF16)
    w, wf = randn(d, seed=1), randn(f, d, seed=2)
    assert moe.moe_rmsnorm(e, w)[0].shape == (0, d)
    assert moe.moe_gated_linear(e, wf, wf)[0].shape == (0, f)
    assert moe.moe_linear(e, wf)[0].shape == (0, f)
    dx, dweight = moe.moe_rmsnorm_backward(e, e, w)
    assert dx.shape == (0, d) and (dweight == 0).all()
    for g in moe.moe_gated_linear_backward(ef, e, wf, wf, ef, ef)[1:]:
        assert (g == 0).all()
    dx, dw, db = moe.moe_linear_backward(ef, e, wf, need_dbias=True)
    assert (dw == 0).all() and (db == 0).all()


def test_more_than_two_to_the_31_elements(moe):
    """Offsets past 32 bits: the last rows of tensors of 2.2e9 elements."""
    n, wide, narrow = 270_001, 8192, 64
    tail = slice(n - 3, n)
    x, w = randn(n, narrow, seed=1), randn(wide, narrow, seed=2, scale=narrow ** -0.5)
    y, _ = moe.moe_linear(x, w)
    (ry, ey), _ = R.linear(x[tail], w, None, None, "none")
    assert_within(y[tail], ry, ey, "y")
    weight = randn(wide, seed=3) + 1
    z, _, _, s = moe.moe_rmsnorm(y, weight, residual=y)
    s64, z64 = R.norm(y[tail], weight, y[tail])
    assert torch.equal(s[tail], s64.float().to(BF16))
    assert_within(z[tail], z64, (R.H + (wide + 16) * R.U) * z64.abs(), "norm")
    del z
    dx, dw, db = moe.moe_linear_backward(y, x, w, z=s, fn=R.FNS["silu"], need_dbias=True)
    (rx, ex), _, _ = R.linear_backward(y[tail], x[tail], w, s[tail], "silu")
    assert_within(dx[tail], rx, ex, "dx")
    assert dw.isfinite().all() and db.isfinite().all()
    dn, _ = moe.moe_rmsnorm_backward(y, s, weight)
    rn, _, en, _ = R.norm_backward(y[tail], s[tail], weight)
    assert_within(dn[tail], rn, en, "norm dx")


@pytest.mark.parametrize("fn", ["silu", "gelu"])
def test_gradients_against_differences(moe, fn):
    """The kernels' gradients along a direction against differences of the 64-bit forward."""
    n, d, f = 48, 128, 192
    x, w1, w3 = randn(n, d, seed=1), randn(f, d, seed=2, scale=d ** -0.5), randn(f, d, seed=3, scale=d ** -0.5)
    up = randn(n, f, seed=4, scale=0.1)
    _, g, u = moe.moe_gated_linear(x, w1, w3, R.FNS[fn], save=True)
    grads = moe.moe_gated_linear_backward(up, x, w1, w3, g, u, R.FNS[fn])

    def loss(x, w1, w3):
        return (R.act(x @ w1.T, fn) * (x @ w3.T) * up.double()).sum()

    at = [t.double() for t in (x, w1, w3)]
    for i, grad in enumerate(grads):
        v = randn(*grad.shape, seed=20 + i).double()
        step = 1e-4
        lo, hi = list(at), list(at)
        lo[i], hi[i] = at[i] - step * v, at[i] + step * v
        want = (loss(*hi) - loss(*lo)) / (2 * step)
        # every element of the gradient carries a few bf16 roundings (the kept g and u, dg and du, itself),
        # independent of the direction: 8 half steps of the norms' product is far above their random sum
        assert abs((grad.double() * v).sum() - want) <= 8 * R.H * grad.double().norm() * v.norm() / grad.numel() ** 0.5 * 4


@pytest.mark.parametrize("n,d,f", [(5000, 512, 2600), (2050, 1544, 4400), (257, 2048, 8200)])
def test_more_tiles_than_pairs(moe, n, d, f):
    """Several rounds of tiles, ragged in every dimension."""
    x, w = randn(n, d, seed=1), randn(f, d, seed=2, scale=d ** -0.5)
    res, dy = randn(n, f, seed=3), randn(n, f, seed=4, scale=0.1)
    ws = moe.workspace("linear_backward", N=n, D=d, Dff=f)
    y, _ = moe.moe_linear(x, w, residual=res, ws=ws)
    (ry, ey), _ = R.linear(x, w, None, res, "none")
    assert_within(y, ry, ey, "y")
    got = moe.moe_linear_backward(dy, x, w, ws=ws)
    for t, (ref, bound), name in zip(got, R.linear_backward(dy, x, w, None, "none"), ("dx", "dw")):
        assert_within(t, ref, bound, name)
    again = moe.moe_linear_backward(dy, x, w, ws=ws)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])
    assert moe.read_device_error(ws) == moe.MOE_OK


@pytest.mark.parametrize("kernel,split", [("1", "1"), ("1", "4"), ("1", "1282"), ("1", "2561"), ("2", "0")])
def test_withheld_load_times_out_and_recovers(moe, kernel, split, monkeypatch):
    """A load that never lands: the call ends, says so, and the next one is right."""
    monkeypatch.setenv("MOE_DENSE_KERNEL", kernel)
    monkeypatch.setenv("MOE_DENSE_SPLIT", split)
    x, w = randn(70, 264, seed=1), randn(136, 264, seed=2, scale=0.1)
    ws = moe.workspace("linear", N=70, D=264, Dff=136)
    want = moe.moe_linear(x, w, ws=ws)[0].clone()
    moe.set_debug_flags(ws, 1)
    moe.moe_linear(x, w, ws=ws)
    assert moe.read_device_error(ws) == moe.MOE_ERR_DEVICE_TIMEOUT
    moe.clear_device_error(ws)
    assert torch.equal(moe.moe_linear(x, w, ws=ws)[0], want)
    assert moe.read_device_error(ws) == moe.MOE_OK
