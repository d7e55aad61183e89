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
