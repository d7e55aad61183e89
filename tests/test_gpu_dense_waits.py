"""The bounded waits of the dense products: valid products that run longer than a wait may take, and loads withheld
from every kind of product and tile."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def moe(cuda_device):
    from mixture_experts_layer_02_gb300 import moe
    moe.load()
    return moe


@pytest.mark.parametrize("kernel,split", [("2", "0"), ("1", "2561")])
def test_a_tile_of_more_than_a_second(moe, kernel, split, monkeypatch):
    """dW = dy^T x over 3.2e8 rows as one pair's tile: five million k-blocks of at least 512 clocks each, 1.2 s at the
    highest clock, against a wait limit of 1 s.  All rows but four are zero, so the product is exact."""
    monkeypatch.setenv("MOE_DENSE_KERNEL", kernel)
    monkeypatch.setenv("MOE_DENSE_SPLIT", split)
    n, d, f = 320_000_000, 8, 8
    dy, x = torch.zeros(n, f, device="cuda", dtype=BF16), torch.zeros(n, d, device="cuda", dtype=BF16)
    want = torch.zeros(f, d, device="cuda", dtype=torch.float64)
    for i, r in enumerate((0, 131, n // 2 + 7, n - 1)):
        dy[r] = torch.arange(i - 3, i - 3 + f, device="cuda").to(BF16)
        x[r] = torch.arange(1, 1 + d, device="cuda").to(BF16) * 2.0 ** -i
        want += torch.outer(dy[r].double(), x[r].double())
    dw = torch.full((f, d), 7.0, device="cuda", dtype=BF16)
    w = torch.zeros(f, d, device="cuda", dtype=BF16)
    ws = moe.workspace("linear_backward", N=n, D=d, Dff=f)
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    status = moe.load().moe_linear_backward(dy.data_ptr(), x.data_ptr(), w.data_ptr(), None, n, d, f, moe.FN_NONE, None,
                                            dw.data_ptr(), None, ws.data_ptr(), ws.numel(),
                                            torch.cuda.current_stream().cuda_stream)
    end.record()
    assert status == moe.MOE_OK
    assert moe.read_device_error(ws) == moe.MOE_OK
    assert torch.equal(dw, want.to(BF16))
    assert start.elapsed_time(end) > 1000.0, "the product has to outlast the limit"


def randn(*shape, seed=0, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + sum((i + 1) * n for i, n in enumerate(shape)))
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(BF16)


@pytest.mark.parametrize("n,d", [(5000, 256), (3000, 520), (1500, 4096), (700, 16384)])
@pytest.mark.parametrize("down", [False, True])
def test_norm_gradient_gives_up_and_recovers(moe, n, d, down):
    """A row whose copies never start: the call ends, says so, and the next one is right.  One, two and four chunks a
    thread, one and several groups a block."""
    dy, s, w = randn(n, d, seed=1, scale=0.1), randn(n, d, seed=2), randn(d, seed=3) + 1
    dres = randn(n, d, seed=4) if down else None
    ws = moe.workspace("rmsnorm_backward", N=n, D=d)
    want = [t.clone() for t in moe.moe_rmsnorm_backward(dy, s, w, dresidual=dres, ws=ws)]
    assert moe.read_device_error(ws) == moe.MOE_OK
    moe.set_debug_flags(ws, 1)
    moe.moe_rmsnorm_backward(dy, s, w, dresidual=dres, ws=ws)
    assert moe.read_device_error(ws) == moe.MOE_ERR_DEVICE_TIMEOUT
    moe.set_debug_flags(ws, 0)
    moe.clear_device_error(ws)
    for a, b in zip(moe.moe_rmsnorm_backward(dy, s, w, dresidual=dres, ws=ws), want):
        assert torch.equal(a, b)
    assert moe.read_device_error(ws) == moe.MOE_OK


#: one-CTA tiles and pair tiles with K whole and in parts, persistent pairs
TILES = [("1", "1"), ("1", "4"), ("1", "1281"), ("1", "2562"), ("2", "0")]


@pytest.mark.parametrize("kernel,split", TILES)
@pytest.mark.parametrize("kind", ["gated", "linear", "dgrad", "dgrad2", "wgrad", "wgrad2"])
def test_withheld_load_of_every_kind(moe, kind, kernel, split, monkeypatch):
    """A load that never lands in each kind of product on each kind of tile: the call ends, says so, and the next one
    is right.  dgrad2 sums two products, wgrad2 has two outputs.  K is 9 to 18 k-blocks: more than the
    stages of the whole tiles."""
    monkeypatch.setenv("MOE_DENSE_KERNEL", kernel)
    monkeypatch.setenv("MOE_DENSE_SPLIT", split)
    m, wide, k = 300, 264, 568
    n, d, f = {"gated": (m, k, wide), "linear": (m, k, wide), "dgrad": (m, wide, k), "dgrad2": (m, wide, k),
               "wgrad": (k, wide, m - 4), "wgrad2": (k, wide, m - 4)}[kind]
    x, w1, w3 = randn(n, d, seed=1), randn(f, d, seed=2, scale=d ** -0.5), randn(f, d, seed=3, scale=d ** -0.5)
    g, u, dy = randn(n, f, seed=4), randn(n, f, seed=5), randn(n, f, seed=6, scale=0.1)
    op = {"gated": "gated_linear", "linear": "linear", "dgrad": "linear_backward", "wgrad": "linear_backward"}.get(
        kind, "gated_linear_backward")
    ws = moe.workspace(op, N=n, D=d, Dff=f)
    L, size, st = moe.load(), ws.numel(), torch.cuda.current_stream().cuda_stream
    outs = [torch.zeros(n, f, device="cuda", dtype=BF16)] if kind in ("gated", "linear") else \
        [torch.zeros(n, d, device="cuda", dtype=BF16)] if kind.startswith("dgrad") else \
        [torch.zeros(f, d, device="cuda", dtype=BF16) for _ in range(2 if kind == "wgrad2" else 1)]
    a = [t.data_ptr() for t in (x, w1, w3, g, u, dy, ws)]
    o = [t.data_ptr() for t in outs]

    def call():
        xp, p1, p3, gp, up, dp, wp = a
        status = {
            "gated": lambda: L.moe_gated_linear(xp, p1, p3, n, d, f, moe.FN_SILU, o[0], None, None, wp, size, st),
            "linear": lambda: L.moe_linear(xp, p1, None, None, n, d, f, moe.FN_NONE, o[0], None, wp, size, st),
            "dgrad": lambda: L.moe_linear_backward(dp, xp, p1, None, n, d, f, moe.FN_NONE, o[0], None, None, wp, size, st),
            "wgrad": lambda: L.moe_linear_backward(dp, xp, p1, None, n, d, f, moe.FN_NONE, None, o[0], None, wp, size, st),
            "dgrad2": lambda: L.moe_gated_linear_backward(dp, xp, p1, p3, gp, up, n, d, f, moe.FN_SILU, o[0], None, None, wp,
                                                          size, st),
            "wgrad2": lambda: L.moe_gated_linear_backward(dp, xp, p1, p3, gp, up, n, d, f, moe.FN_SILU, None, o[0], o[1], wp,
                                                          size, st)}[kind]()
        assert status == moe.MOE_OK

    call()
    assert moe.read_device_error(ws) == moe.MOE_OK
    want = [t.clone() for t in outs]
    moe.set_debug_flags(ws, 1)
    call()
    assert moe.read_device_error(ws) == moe.MOE_ERR_DEVICE_TIMEOUT
    moe.clear_device_error(ws)
    call()
    assert moe.read_device_error(ws) == moe.MOE_OK
    for t, ref in zip(outs, want):
        assert torch.equal(t, ref) and t.isfinite().all() and (t != 0).any()
