"""Gradients of the weighted sum, the sort by expert and the routing weights against their 64-bit definitions."""
import pytest
import torch

import train_reference as T
from dense_reference import assert_within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe(cuda_device):
    from mixture_experts_layer_02_gb300 import moe
    return moe


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(g, *shape, scale=1.0):
    return torch.randn(shape, generator=g, device="cuda").mul_(scale).to(torch.bfloat16)


def rows_of(g, N, K, rows=None, dropped=0.0):
    """[N, K] distinct rows of 0..rows-1, some of them dropped (-1)."""
    rows = N * K if rows is None else rows
    inv = torch.randperm(rows, generator=g, device="cuda")[:N * K].view(N, K).to(torch.int32)
    if dropped:
        inv[torch.rand((N, K), generator=g, device="cuda") < dropped] = -1
    return inv


SIZES = [(1, 8, 1), (1, 7168, 8), (3, 16, 32), (5, 264, 2), (33, 1032, 3), (64, 4104, 8), (700, 512, 6), (40, 16392, 2)]


@pytest.mark.parametrize("N,D,K", SIZES)
@pytest.mark.parametrize("dropped", [0.0, 0.4])
def test_combine_backward(moe, N, D, K, dropped):
    g = gen(N + D)
    rows = N * K + (17 if dropped else 0)
    dout, y, w, inv = normal(g, N, D), normal(g, rows, D), torch.rand((N, K), generator=g, device="cuda"), rows_of(g, N, K, rows, dropped)
    (dy, e_dy), (dw, e_dw), named = T.combine_backward(dout, y, inv.cpu(), w)
    ws = moe.workspace("combine")
    got = torch.full((rows, D), 7.0, dtype=torch.bfloat16, device="cuda")
    _, got_w = moe.moe_combine_backward(dout, y, inv, w, dy_perm=got, ws=ws)
    assert moe.read_device_error(ws) == 0
    assert_within(got[named], dy[named], e_dy[named], "dy")
    assert (got[~named] == 7).all()
    assert_within(got_w, dw, e_dw, "dw")
    own = moe.moe_combine_backward(dout, y, inv, w, dy_perm=y, ws=ws)  # over its own input
    assert torch.equal(own[0][named], got[named]) and torch.equal(own[1], got_w)


@pytest.mark.parametrize("N,D,K", SIZES)
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("dropped", [0.0, 0.4])
def test_permute_backward(moe, N, D, K, residual, dropped):
    g = gen(N + D)
    rows = N * K + (17 if dropped else 0)
    src, inv = normal(g, rows, D), rows_of(g, N, K, rows, dropped)
    res = normal(g, N, D) if residual else None
    ws = moe.workspace("combine")
    got = moe.moe_permute_backward(src, inv, dresidual=res, ws=ws)
    assert moe.read_device_error(ws) == 0
    assert_within(got, *T.permute_backward(src, inv.cpu(), res), "dx")
    if residual:
        assert torch.equal(moe.moe_permute_backward(src, inv, dresidual=res, dx=res, ws=ws), got)


def test_tokens_without_any_row(moe):
    g = gen(3)
    src, res = normal(g, 8, 64), normal(g, 4, 64)
    inv = torch.full((4, 2), -1, dtype=torch.int32, device="cuda")
    w = torch.rand((4, 2), generator=g, device="cuda")
    assert torch.equal(moe.moe_permute_backward(src, inv, dresidual=res), res)
    assert (moe.moe_permute_backward(src, inv) == 0).all()
    dy, dw = moe.moe_combine_backward(res, src, inv, w, dy_perm=torch.ones_like(src))
    assert (dy == 1).all() and (dw == 0).all()
    empty = src[:0]
    assert torch.equal(moe.moe_permute_backward(empty, inv, dresidual=res), res)
    assert (moe.moe_combine_backward(res, empty, inv, w)[1] == 0).all()


def test_rows_outside_are_flagged_and_skipped(moe):
    g = gen(4)
    src, dout, w = normal(g, 8, 64), normal(g, 4, 64), torch.rand((4, 2), generator=g, device="cuda")
    inv = torch.tensor([[0, 8], [-2, 3], [1, 2], [2 ** 31 - 1, 5]], dtype=torch.int32, device="cuda")
    kept = torch.where((inv >= 0) & (inv < 8), inv, -1)
    for call in (lambda i, ws: moe.moe_permute_backward(src, i, ws=ws),
                 lambda i, ws: moe.moe_combine_backward(dout, src, i, w, dy_perm=torch.zeros_like(src), ws=ws)[0]):
        ws = moe.workspace("combine")
        got = call(inv, ws)
        assert moe.read_device_error(ws) == moe.MOE_ERR_DEVICE_BOUNDS
        assert torch.equal(got, call(kept, None))


def test_infinite_and_nan_rows_touch_their_tokens_only(moe):
    g = gen(5)
    src, inv = normal(g, 12, 64), rows_of(gen(6), 6, 2)
    clean = moe.moe_permute_backward(src, inv)
    src[int(inv[2, 1])] = float("nan")
    src[int(inv[4, 0])] = float("inf")
    got = moe.moe_permute_backward(src, inv)
    keep = [0, 1, 3, 5]
    assert torch.equal(got[keep], clean[keep]) and got[2].isnan().all() and got[4].isinf().all()


def test_padded_paradigm(moe):
    """The gradient through moe_permute_padded and moe_combine_padded: slots with dropped assignments."""
    g = gen(7)
    N, D, E, K, cap = 40, 128, 8, 2, 6
    x = normal(g, N, D)
    ids = torch.rand((N, E), generator=g, device="cuda").topk(K, 1).indices.to(torch.int32)
    _, kept, slot, x_pad = moe.moe_permute_padded(x, ids, E, cap)
    assert (slot == -1).any()
    w = torch.rand((N, K), generator=g, device="cuda")
    dout = normal(g, N, D)
    dy, dw = moe.moe_combine_backward(dout, x_pad, slot, w)
    (want, e), (want_w, e_w), named = T.combine_backward(dout, x_pad, slot.cpu(), w)
    assert_within(dy, want, e, "dy")  # rows that no assignment has are zero in a buffer made by the call
    assert_within(dw, want_w, e_w, "dw")
    assert_within(moe.moe_permute_backward(dy, slot), *T.permute_backward(dy, slot.cpu(), None), "dx")


def routed(g, N, D, E, K, sigmoid, duplicate=False):
    x, wg = normal(g, N, D), normal(g, E, D, scale=D ** -0.5)
    logits = 2 * torch.randn((N, E), generator=g, device="cuda")
    top = torch.topk(logits, K, 1)
    if sigmoid:
        s = torch.sigmoid(top.values)
        w = s / s.sum(1, keepdim=True)
    else:
        w = torch.softmax(top.values, 1)
    ids = top.indices.to(torch.int32).contiguous()
    if duplicate and K > 1:
        ids[::3, 1] = ids[::3, 0]
    return x, wg, logits, ids, w.contiguous(), torch.randn((N, K), generator=g, device="cuda")


def test_empty_slots_of_a_buffer_made_here_are_zero(moe):
    """As many slots as assignments, some dropped and some empty: capacity factor one under a lopsided routing."""
    N, D, E, K = 64, 256, 4, 2
    cap = N * K // E
    x = normal(gen(5), N, D)
    ids = torch.tensor([0, 1], dtype=torch.int32, device="cuda").repeat(N, 1)
    w = torch.rand((N, K), generator=gen(6), device="cuda")
    _, kept, slot, x_pad = moe.moe_permute_padded(x, ids, E, cap)
    assert kept.tolist() == [cap, cap, 0, 0] and (slot < 0).sum() == N * K - 2 * cap
    ws = moe.workspace("combine")
    held = [torch.full((E * cap, D), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(64)]
    del held  # every free block of this size holds NaN
    dy, _ = moe.moe_combine_backward(x, x_pad, slot, w, ws=ws)
    assert (dy[2 * cap:] == 0).all() and torch.isfinite(dy).all()


@pytest.mark.parametrize("N,D,E,K", [(1, 64, 8, 2), (3, 8, 4, 4), (100, 2048, 128, 8), (77, 520, 60, 6), (513, 256, 7, 3),
                                     (40, 136, 1024, 32), (300, 1032, 256, 8), (5, 64, 1, 1)])
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("residual", [False, True])
def test_route_backward(moe, N, D, E, K, sigmoid, residual):
    g = gen(N + E)
    x, wg, logits, ids, w, dw = routed(g, N, D, E, K, sigmoid)
    res = normal(g, N, D) if residual else None
    mode = moe.SIGMOID_NORM if sigmoid else moe.SOFTMAX_TOPK
    ws = moe.workspace("route_backward", N=N, D=D, E=E)
    got = moe.moe_route_backward(dw, ids, w, logits if sigmoid else None, x, wg, mode, dresidual=res, need_dbias=True, ws=ws)
    assert moe.read_device_error(ws) == 0
    want = T.route_backward(dw, ids, w, logits, x, wg, sigmoid, res)
    for a, (ref, e), name in zip(got, want, ("dx", "dw_gate", "dbias")):
        assert_within(a, ref, e, name)
    if residual:
        over = moe.moe_route_backward(dw, ids, w, logits, x, wg, mode, dresidual=res, dx=res, ws=ws)
        assert torch.equal(over[0], got[0]) and torch.equal(over[1], got[1]) and over[2] is None


@pytest.mark.parametrize("kernel,split", [("1", "1"), ("1", "2"), ("1", "4"), ("1", "8"), ("1", "1281"), ("1", "1284"), ("1", "2561"),
                                          ("1", "2564"), ("2", "-1")])
def test_route_backward_residual_in_every_tile_kind(moe, monkeypatch, kernel, split):
    """The residual's addition in the epilogue of each form of the dense gradient product."""
    g = gen(9)
    x, wg, logits, ids, w, dw = routed(g, 600, 520, 1024, 8, True)
    res = normal(g, 600, 520)
    monkeypatch.setenv("MOE_DENSE_KERNEL", kernel)
    monkeypatch.setenv("MOE_DENSE_SPLIT", split)
    got = moe.moe_route_backward(dw, ids, w, logits, x, wg, moe.SIGMOID_NORM, dresidual=res)
    want = T.route_backward(dw, ids, w, logits, x, wg, True, res)
    assert_within(got[0], *want[0], "dx")
    assert_within(got[1], *want[1], "dw_gate")


def test_route_backward_same_expert_twice_and_outside(moe):
    g = gen(11)
    x, wg, logits, ids, w, dw = routed(g, 50, 128, 16, 4, False, duplicate=True)
    got = moe.moe_route_backward(dw, ids, w, None, x, wg, moe.SOFTMAX_TOPK, need_dbias=True)
    for a, (ref, e) in zip(got, T.route_backward(dw, ids, w, logits, x, wg, False, None)):
        assert_within(a, ref, e, "twice")
    ids[7, 2], ids[9, 0] = 16, -1
    ws = moe.workspace("route_backward", N=50, D=128, E=16)
    got = moe.moe_route_backward(dw, ids, w, None, x, wg, moe.SOFTMAX_TOPK, need_dbias=True, ws=ws)
    assert moe.read_device_error(ws) == moe.MOE_ERR_DEVICE_BOUNDS
    for a, (ref, e) in zip(got, T.route_backward(dw, ids, w, logits, x, wg, False, None)):
        assert_within(a, ref, e, "outside")


@pytest.mark.parametrize("sigmoid", [False, True])
def test_route_backward_against_differences(moe, sigmoid):
    """The definition itself against central differences of the forward pass in 64 bits."""
    g = gen(12)
    N, D, E, K = 6, 32, 8, 3
    x, wg, logits, ids, w, dw = routed(g, N, D, E, K, sigmoid)
    xd, gd, i = x.double(), wg.double(), ids.long()

    def loss(a, b, bias):
        chosen = torch.gather(a @ b.T + bias, 1, i)
        s = torch.sigmoid(chosen)
        wt = s / s.sum(1, keepdim=True) if sigmoid else torch.softmax(chosen, 1)
        return (wt * dw.double()).sum()

    bias = torch.zeros(E, dtype=torch.float64, device="cuda")
    lg = xd @ gd.T
    chosen = torch.gather(lg, 1, i)
    s = torch.sigmoid(chosen)
    wt = (s / s.sum(1, keepdim=True) if sigmoid else torch.softmax(chosen, 1))
    want = T.route_backward(dw, ids, wt, lg, x, wg, sigmoid, None)
    h = 1e-6
    for leaf, (ref, _) in zip((xd, gd, bias), want):
        flat = leaf.view(-1)
        for j in range(0, flat.numel(), max(1, flat.numel() // 16)):
            keep = flat[j].item()
            flat[j] = keep + h
            up = loss(xd, gd, bias)
            flat[j] = keep - h
            down = loss(xd, gd, bias)
            flat[j] = keep
            # second differences are of order 1, so the quotient is off by h^2 and by rounding over h
            assert abs((up - down).item() / (2 * h) - ref.reshape(-1)[j].item()) < 1e-7
    got = moe.moe_route_backward(dw, ids, wt.float(), lg.float(), x, wg, moe.SIGMOID_NORM if sigmoid else moe.SOFTMAX_TOPK,
                                 need_dbias=True)
    for a, (ref, e), name in zip(got, T.route_backward(dw, ids, wt.float(), lg.float(), x, wg, sigmoid, None), ("dx", "dw", "db")):
        assert_within(a, ref, e, name)


def test_no_tokens(moe):
    dev, bf = "cuda", torch.bfloat16
    x, wg = torch.empty((0, 64), dtype=bf, device=dev), torch.ones((8, 64), dtype=bf, device=dev)
    k = torch.empty((0, 2), device=dev)
    ids = torch.empty((0, 2), dtype=torch.int32, device=dev)
    dx, dg, db = moe.moe_route_backward(k, ids, k, None, x, wg, moe.SOFTMAX_TOPK, need_dbias=True,
                                        dw_gate=torch.ones((8, 64), dtype=bf, device=dev), dbias=torch.ones(8, device=dev))
    assert dx.shape == (0, 64) and (dg == 0).all() and (db == 0).all()
    assert moe.moe_permute_backward(x, ids).shape == (0, 64)
    assert moe.moe_combine_backward(x, x, ids, k)[1].shape == (0, 2)


def test_same_bits_in_a_graph_and_on_another_stream(moe):
    g = gen(13)
    N, D, E, K = 200, 512, 32, 4
    x, wg, logits, ids, w, dw = routed(g, N, D, E, K, True)
    inv = rows_of(g, N, K)
    y, dout = normal(g, N * K, D), normal(g, N, D)
    ws = moe.workspace("route_backward", N=N, D=D, E=E)

    def run(stream=None):
        dy, dwk = moe.moe_combine_backward(dout, y, inv, w, ws=ws, stream=stream)
        dx = moe.moe_permute_backward(dy, inv, dresidual=dout, ws=ws, stream=stream)
        return [dy, dwk, *moe.moe_route_backward(dwk, ids, w, logits, x, wg, moe.SIGMOID_NORM, dresidual=dx, need_dbias=True,
                                                 ws=ws, stream=stream)]

    first = run()
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    second = run(other)
    other.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        third = run()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for a, b, c in zip(first, second, third):
        assert torch.equal(a, b) and torch.equal(a, c)
    assert moe.read_device_error(ws) == 0
