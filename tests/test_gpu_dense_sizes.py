"""The dense products at the ends of their sizes, on forced kernels over several rounds, and with only some outputs."""
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


def randn(*shape, seed=0, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + sum((i + 1) * n for i, n in enumerate(shape)))
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(BF16)


def test_as_many_rows_as_are_taken(moe):
    """2^31 - 4096 rows of width 8, zero but for a few: products, gradients and the bias gradient of those are exact."""
    n, d, f = 2 ** 31 - 4096, 8, 8
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 160e9:
        pytest.skip("four tensors of 34 GB")
    at = [0, 1, 2 ** 28 + 5, 2 ** 30 - 1, 2 ** 30 + 77, n - 130, n - 1]
    rows = torch.tensor(at, device="cuda")
    x = torch.zeros(n, d, device="cuda", dtype=BF16)
    x[rows] = torch.randint(-8, 9, (len(at), d), device="cuda").to(BF16)
    w = torch.randint(-4, 5, (f, d), device="cuda").to(BF16)  # sums of integers below 2^8: exact in bf16
    w[:, 4:] = 0
    y, _ = moe.moe_linear(x, w)
    want = x[rows].double() @ w.double().T
    assert torch.equal(y[rows].double(), want.to(BF16).double())
    assert torch.equal((y != 0).any(1).nonzero()[:, 0], rows[(want != 0).any(1)])
    del y
    dy = torch.zeros(n, f, device="cuda", dtype=BF16)
    dy[rows] = torch.randint(-3, 4, (len(at), f), device="cuda").to(BF16)
    dx, dw, db = moe.moe_linear_backward(dy, x, w, need_dbias=True)
    assert torch.equal(dx[rows].double(), (dy[rows].double() @ w.double()).to(BF16).double())
    assert torch.equal(dw.double(), (dy[rows].double().T @ x[rows].double()).to(BF16).double())
    assert torch.equal(db.double(), dy[rows].double().sum(0))
    del x, dy, dx
    torch.cuda.empty_cache()


# ------------------------------------------------------------------ persistent pairs over several rounds
@pytest.fixture
def pairs(monkeypatch):
    monkeypatch.setenv("MOE_DENSE_KERNEL", "2")


@pytest.mark.parametrize("n,d,f", [(2050, 200, 3400), (5000, 72, 1800)])
def test_gated_rounds_of_pairs(moe, pairs, n, d, f):
    """More than three tiles for each of the 76 pairs: both accumulators in use again, g and u kept."""
    x, w1, w3 = randn(n, d, seed=1), randn(f, d, seed=2, scale=d ** -0.5), randn(f, d, seed=3, scale=d ** -0.5)
    ws = moe.workspace("gated_linear", N=n, D=d, Dff=f)
    got = moe.moe_gated_linear(x, w1, w3, save=True, ws=ws)
    assert moe.read_device_error(ws) == moe.MOE_OK
    for t, (ref, bound), name in zip(got, R.gated(x, w1, w3, "silu"), "hgu"):
        assert_within(t, ref, bound, name)


def test_linear_rounds_of_pairs(moe, pairs):
    n, d, f = 2050, 200, 6600
    x, w, bias, res = randn(n, d, seed=1), randn(f, d, seed=2, scale=d ** -0.5), randn(f, seed=3).float(), randn(n, f, seed=4)
    (ry, ey), (rz, ez) = R.linear(x, w, bias, res, "gelu")
    y, z = moe.moe_linear(x, w, bias=bias, residual=res, fn=moe.FN_GELU, save=True)
    assert_within(y, ry, ey, "y")
    assert_within(z, rz, ez, "z")


@pytest.mark.parametrize("n,d,f", [(2050, 6600, 264), (264, 3400, 3400)])
def test_gated_gradient_rounds_of_pairs(moe, pairs, n, d, f):
    """The two summed products of dx over several rounds, then the two outputs dw1 and dw3."""
    x, w1, w3 = randn(n, d, seed=1), randn(f, d, seed=2, scale=d ** -0.5), randn(f, d, seed=3, scale=d ** -0.5)
    g, u, dh = randn(n, f, seed=4), randn(n, f, seed=5), randn(n, f, seed=6, scale=0.1)
    ws = moe.workspace("gated_linear_backward", N=n, D=d, Dff=f)
    got = moe.moe_gated_linear_backward(dh, x, w1, w3, g, u, ws=ws)
    assert moe.read_device_error(ws) == moe.MOE_OK
    for t, (ref, bound), name in zip(got, R.gated_backward(dh, x, w1, w3, g, u, "silu"), ("dx", "dw1", "dw3")):
        assert_within(t, ref, bound, name)


# ------------------------------------------------------------------ one-CTA tiles, four parts of K
@pytest.mark.parametrize("n,d,f", [(100, 2048, 768), (129, 2056, 328), (300, 776, 520), (700, 4104, 400)])
def test_four_parts(moe, n, d, f, monkeypatch):
    monkeypatch.setenv("MOE_DENSE_KERNEL", "1")
    monkeypatch.setenv("MOE_DENSE_SPLIT", "4")
    x, w1, w3 = randn(n, d, seed=1), randn(f, d, seed=2, scale=d ** -0.5), randn(f, d, seed=3, scale=d ** -0.5)
    g, u, dh = randn(n, f, seed=4), randn(n, f, seed=5), randn(n, f, seed=6, scale=0.1)
    for t, (ref, bound), name in zip(moe.moe_gated_linear(x, w1, w3, save=True), R.gated(x, w1, w3, "silu"), "hgu"):
        assert_within(t, ref, bound, name)
    res = randn(n, f, seed=7)
    y, _ = moe.moe_linear(x, w1, residual=res)
    (ry, ey), _ = R.linear(x, w1, None, res, "none")
    assert_within(y, ry, ey, "y")
    got = moe.moe_gated_linear_backward(dh, x, w1, w3, g, u)
    for t, (ref, bound), name in zip(got, R.gated_backward(dh, x, w1, w3, g, u, "silu"), ("dx", "dw1", "dw3")):
        assert_within(t, ref, bound, name)
    got = moe.moe_linear_backward(dh, x, w1)
    for t, (ref, bound), name in zip(got, R.linear_backward(dh, x, w1, None, "none"), ("dx", "dw")):
        assert_within(t, ref, bound, name)


# ------------------------------------------------------------------ only some of the gradients
@pytest.mark.parametrize("n", [3, 200])
def test_gradients_whose_pointer_is_null_are_left_out(moe, n):
    """Each output alone has the bits it has among all of them."""
    d, f = 264, 328
    x, w1, w3 = randn(n, d, seed=1), randn(f, d, seed=2, scale=0.1), randn(f, d, seed=3, scale=0.1)
    g, u, dy = randn(n, f, seed=4), randn(n, f, seed=5), randn(n, f, seed=6, scale=0.1)
    L, st = moe.load(), torch.cuda.current_stream().cuda_stream

    def check(op, full, call, groups):
        ws = moe.workspace(op, N=n, D=d, Dff=f)
        for keep in groups:
            outs = [torch.zeros_like(t) if i in keep else None for i, t in enumerate(full)]
            status = call([None if t is None else t.data_ptr() for t in outs], ws)
            assert status == moe.MOE_OK and moe.read_device_error(ws) == moe.MOE_OK
            for t, want in zip(outs, full):
                assert t is None or torch.equal(t, want)

    full = moe.moe_gated_linear_backward(dy, x, w1, w3, g, u)
    check("gated_linear_backward", full, lambda o, ws: L.moe_gated_linear_backward(
        dy.data_ptr(), x.data_ptr(), w1.data_ptr(), w3.data_ptr(), g.data_ptr(), u.data_ptr(), n, d, f, moe.FN_SILU, *o,
        ws.data_ptr(), ws.numel(), st), [(0,), (1, 2), ()])
    for fn, z in ((moe.FN_NONE, None), (moe.FN_GELU, g)):
        full = moe.moe_linear_backward(dy, x, w1, z=z, fn=fn, need_dbias=True)
        check("linear_backward", full, lambda o, ws: L.moe_linear_backward(
            dy.data_ptr(), x.data_ptr(), w1.data_ptr(), None if z is None else z.data_ptr(), n, d, f, fn, *o, ws.data_ptr(),
            ws.numel(), st), [(0,), (1,), (2,), (0, 1), (0, 2), (1, 2), ()])
    weight = randn(d, seed=8)
    full = moe.moe_rmsnorm_backward(x, x, weight)
    check("rmsnorm_backward", full, lambda o, ws: L.moe_rmsnorm_backward(
        x.data_ptr(), x.data_ptr(), weight.data_ptr(), None, n, d, 1e-6, *o, ws.data_ptr(), ws.numel(), st), [(0,)])


def test_sums_over_more_than_two_to_the_31_elements(moe):
    """dw and dbias of a gradient of 2.2e9 elements, on columns from both ends and the middle."""
    n, wide, narrow = 270_001, 8192, 64
    x, w = randn(n, narrow, seed=1), randn(wide, narrow, seed=2, scale=narrow ** -0.5)
    dy, z = randn(n, wide, seed=3, scale=0.1), randn(n, wide, seed=4)
    _, dw, db = moe.moe_linear_backward(dy, x, w, z=z, fn=moe.FN_SILU, need_dbias=True)
    cols = torch.tensor([0, 1, 63, 64, 4095, 4096, 8128, 8191], device="cuda")
    _, (rw, ew), (rb, eb) = R.linear_backward(dy[:, cols], x, w[cols], z[:, cols], "silu")
    assert_within(dw[cols], rw, ew, "dw")
    assert_within(db[cols], rb, eb, "dbias")
