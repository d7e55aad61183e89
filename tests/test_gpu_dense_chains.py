"""Chains of small products through reused buffers: each call reads what the one before it wrote, into memory that
the calls before that one read."""
import pytest
import torch

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


def both(run, steps):
    """run(k) for k < steps, once waiting for the GPU after each call and then as a stream of calls, five times;
    run(-1) sets the buffers back and returns what to compare."""
    outs = run(-1)
    for k in range(steps):
        run(k)
        torch.cuda.synchronize()
    want = [o.clone() for o in outs]
    assert all(w.isfinite().all() for w in want) and all((w != 0).any() for w in want)
    for _ in range(5):
        outs = run(-1)
        torch.cuda.synchronize()
        for k in range(steps):
            run(k)
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("n", [1, 4, 8, 30])
@pytest.mark.parametrize("d", [264, 1024, 4096])
def test_two_buffers_in_turn(moe, n, d):
    """y = act(x w^T) back and forth between two buffers."""
    ws = moe.workspace("linear", N=n, D=d, Dff=d)
    w = randn(d, d, seed=2, scale=1.5 * d ** -0.5)
    start = randn(n, d, seed=1)
    a, b = torch.empty_like(start), torch.empty_like(start)

    def run(k):
        if k < 0:
            a.copy_(start)
            b.zero_()
            return [a, b]
        moe.moe_linear(b if k & 1 else a, w, residual=a if k & 1 else b, fn=moe.FN_RELU if k % 3 else moe.FN_NONE,
                       y=a if k & 1 else b, ws=ws)
        if k % 16 == 15:  # keep the values of one size
            (a if k & 1 else b).mul_(0.25)

    both(run, 64)


@pytest.mark.parametrize("n", [2, 8])
def test_gated_and_norm_in_turn(moe, n):
    """norm, gated product and residual projection of one block, step after step through the same buffers."""
    d, f = 1024, 768
    ws = moe.workspace("linear", N=n, D=max(d, f), Dff=max(d, f))
    w1, w3, w2 = randn(f, d, seed=2, scale=d ** -0.5), randn(f, d, seed=3, scale=d ** -0.5), randn(d, f, seed=4, scale=f ** -0.5)
    weight = randn(d, seed=5, scale=0.1) + 1
    start = randn(n, d, seed=1)
    s, y, h = torch.empty_like(start), torch.empty_like(start), torch.empty(n, f, dtype=BF16, device="cuda")

    def run(k):
        if k < 0:
            s.copy_(start)
            return [s, y, h]
        moe.moe_rmsnorm(s, weight, y=y)
        moe.moe_gated_linear(y, w1, w3, h=h, ws=ws)
        moe.moe_linear(h, w2, residual=s, y=s, ws=ws)

    both(run, 40)


def test_products_as_the_next_weights(moe):
    """The output of one streamed product is the weight of the next, in two buffers."""
    n, d = 8, 512
    ws = moe.workspace("linear", N=n, D=d, Dff=d)
    w, start = randn(d, d, seed=2, scale=d ** -0.5), randn(n, d, seed=1)
    x = randn(n, d, seed=3, scale=d ** -0.5)
    a, b, out = torch.empty_like(start), torch.empty_like(start), torch.empty(n, 8, dtype=BF16, device="cuda")
    total = torch.empty(48, n, 8, dtype=BF16, device="cuda")

    def run(k):
        if k < 0:
            a.copy_(start)
            b.zero_()
            out.zero_()
            total.zero_()
            return [a, b, total]
        cur, new = (b, a) if k & 1 else (a, b)
        moe.moe_linear(x, cur, y=total[k], ws=ws)          # [n, 8] = x cur^T: cur [8, d] as the weight
        moe.moe_linear(cur, w, y=new, ws=ws)

    both(run, 48)
