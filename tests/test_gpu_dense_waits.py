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
