"""The experts' product in e4m3 with a scale for each block of 128, and its gradients, against the 64-bit definition."""
import pytest
import torch

import train_reference as T
from dense_reference import assert_within

pytestmark = pytest.mark.gpu

B = T.B
#: every tile kind: 128 x 128 with K in 1, 2 or 4 parts, 128 x 256, CTA pairs; the stream of weight rows
KERNELS = ["1/1", "1/2", "1/4", "2", "3", "4/1", "4/2", "4/4", "4/8"]


@pytest.fixture(scope="module")
def moe(cuda_device):
    from mixture_experts_layer_02_gb300 import moe
    return moe


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def codes(g, *shape):
    v = torch.randn(shape, generator=g, device="cuda").mul_(140).clamp_(-448, 448)
    return v.to(torch.float8_e4m3fn).view(torch.uint8)


def scales(g, *shape):
    return torch.exp(torch.randn(shape, generator=g, device="cuda"))


def offsets_of(counts):
    return torch.tensor([0] + torch.tensor(counts).cumsum(0).tolist(), dtype=torch.int32, device="cuda")


def forward_inputs(counts, D, F, extra=0, seed=1):
    g, rows, E = gen(seed), sum(counts) + extra, len(counts)
    return codes(g, rows, D), scales(g, rows, T.blocks(D)), codes(g, E, F, D), scales(g, E, T.blocks(F), T.blocks(D))


def backward_inputs(moe, counts, D, F, seed=2, extra=0):
    """The weights, dy in both forms and x along its rows, with zero rows behind each segment and noise behind the last."""
    g, rows, E = gen(seed), sum(counts) + extra, len(counts)
    m = moe.segment_rows(rows, E)
    assert m == T.segment_rows(rows, E)
    w = codes(g, E, F, D), scales(g, E, T.blocks(F), T.blocks(D))
    dy = codes(g, rows, F), scales(g, rows, T.blocks(F))
    seg = codes(g, m, F), scales(g, m // B, F), codes(g, m, D), scales(g, m // B, D)
    for _, a, b, pa, pb in T.spans(counts):
        seg[0][pa + b - a:pb] = 0
        seg[2][pa + b - a:pb] = 0
    return w, dy, seg


def choose(monkeypatch, kernel):
    if kernel:
        k, _, s = kernel.partition("/")
        monkeypatch.setenv("MOE_BLOCK_KERNEL", k)
        monkeypatch.setenv("MOE_BLOCK_SPLIT", s or "1")


COUNTS = [[1], [3, 0, 0, 2], [0, 127, 1, 0, 128, 129, 0], [257, 40, 300], [700]]


@pytest.mark.parametrize("kernel", KERNELS + [""])
@pytest.mark.parametrize("counts", COUNTS, ids=str)
@pytest.mark.parametrize("D,F", [(16, 16), (128, 256), (272, 400), (1040, 144)])
def test_forward(moe, monkeypatch, kernel, counts, D, F):
    choose(monkeypatch, kernel)
    xq, xs, wq, ws = forward_inputs(counts, D, F)
    wsp = moe.workspace("grouped_linear_e4m3_block", N=sum(counts), D=D, E=len(counts), Dff=F)
    y = moe.moe_grouped_linear_e4m3_block(xq, xs, wq, ws, expert_offsets=offsets_of(counts), ws=wsp)
    assert moe.read_device_error(wsp) == 0
    assert_within(y, *T.product(xq, xs, wq, ws, counts), "y")


@pytest.mark.parametrize("kernel", KERNELS + [""])
@pytest.mark.parametrize("counts", COUNTS, ids=str)
@pytest.mark.parametrize("D,F", [(16, 16), (128, 256), (272, 400), (1040, 144)])
def test_backward(moe, monkeypatch, kernel, counts, D, F):
    choose(monkeypatch, kernel)
    (wq, ws), (dyq, dys), seg = backward_inputs(moe, counts, D, F)
    wsp = moe.workspace("grouped_linear_e4m3_block_backward", N=sum(counts), D=D, E=len(counts), Dff=F)
    dx, dw = moe.moe_grouped_linear_e4m3_block_backward(wq, ws, dyq, dys, *seg, expert_offsets=offsets_of(counts), ws=wsp)
    assert moe.read_device_error(wsp) == 0
    want_dx, want_dw = T.product_backward(dyq, dys, *seg, wq, ws, counts)
    assert_within(dx, *want_dx, "dx")
    assert_within(dw, *want_dw, "dw")


@pytest.mark.parametrize("kernel", KERNELS + [""])
def test_rows_behind_the_last_segment_stay(moe, monkeypatch, kernel):
    choose(monkeypatch, kernel)
    counts, D, F = [70, 0, 133], 272, 144
    off = offsets_of(counts)
    xq, xs, wq, ws = forward_inputs(counts, D, F, extra=90)
    y = torch.full((293, F), 7.0, dtype=torch.bfloat16, device="cuda")
    moe.moe_grouped_linear_e4m3_block(xq, xs, wq, ws, expert_offsets=off, y=y)
    assert_within(y[:203], *T.product(xq[:203], xs[:203], wq, ws, counts), "y")
    assert (y[203:] == 7).all()
    (wq, ws), (dyq, dys), seg = backward_inputs(moe, counts, D, F, extra=90)
    dx = torch.full((293, D), 7.0, dtype=torch.bfloat16, device="cuda")
    _, dw = moe.moe_grouped_linear_e4m3_block_backward(wq, ws, dyq, dys, *seg, expert_offsets=off, dx=dx)
    want_dx, want_dw = T.product_backward(dyq[:203], dys[:203], *seg, wq, ws, counts)
    assert_within(dx[:203], *want_dx, "dx")
    assert (dx[203:] == 7).all()
    assert_within(dw, *want_dw, "dw")


@pytest.mark.parametrize("kernel", KERNELS + [""])
def test_no_rows_at_all(moe, monkeypatch, kernel):
    """Rows that belong to no expert, and no rows: outputs stay, weight gradients are zero."""
    choose(monkeypatch, kernel)
    for rows in (5, 0):
        off = torch.zeros(4, dtype=torch.int32, device="cuda")
        xq, xs, wq, ws = forward_inputs([0, 0, 0], 144, 272, extra=rows)
        y = torch.full((rows, 272), 7.0, dtype=torch.bfloat16, device="cuda")
        moe.moe_grouped_linear_e4m3_block(xq, xs, wq, ws, expert_offsets=off, y=y)
        (wq, ws), (dyq, dys), seg = backward_inputs(moe, [0, 0, 0], 144, 272, extra=rows)
        dx = torch.full((rows, 144), 7.0, dtype=torch.bfloat16, device="cuda")
        dw = torch.full((3, 272, 144), 7.0, dtype=torch.bfloat16, device="cuda")
        wsp = moe.workspace("combine")
        moe.moe_grouped_linear_e4m3_block_backward(wq, ws, dyq, dys, *seg, expert_offsets=off, dx=dx, dw=dw, ws=wsp)
        assert moe.read_device_error(wsp) == 0
        assert (y == 7).all() and (dx == 7).all() and (dw == 0).all()
        src = torch.ones((rows, 144), dtype=torch.bfloat16, device="cuda")
        q_seg = torch.full((moe.segment_rows(rows, 3), 144), 99, dtype=torch.uint8, device="cuda")
        assert (moe.moe_quantize_e4m3_segments(src, off, both=False, q_seg=q_seg)[2] == 99).all()


def test_dense_form_needs_no_offsets(moe):
    xq, xs, wq, ws = forward_inputs([37], 528, 272)
    a = moe.moe_grouped_linear_e4m3_block(xq, xs, wq, ws)
    assert_within(a, *T.product(xq, xs, wq, ws, [37]), "y")
    (wq, ws), (dyq, dys), seg = backward_inputs(moe, [37], 528, 272)
    dx, dw = moe.moe_grouped_linear_e4m3_block_backward(wq, ws, dyq, dys, *seg)
    want_dx, want_dw = T.product_backward(dyq, dys, *seg, wq, ws, [37])
    assert_within(dx, *want_dx, "dx")
    assert_within(dw, *want_dw, "dw")


@pytest.mark.parametrize("kernel", KERNELS)
def test_scales_found_through_the_tokens(moe, monkeypatch, kernel):
    choose(monkeypatch, kernel)
    counts, D, F = [150, 3, 90], 400, 272
    xq, _, wq, ws = forward_inputs(counts, D, F)
    by_token = scales(gen(5), 61, T.blocks(D))
    src = torch.randint(0, 61, (243,), generator=gen(6), device="cuda", dtype=torch.int32)
    y = moe.moe_grouped_linear_e4m3_block(xq, by_token, wq, ws, expert_offsets=offsets_of(counts), x_scale_index=src)
    assert_within(y, *T.product(xq, by_token[src.long()], wq, ws, counts), "y")


def test_every_row_has_its_own_place(moe):
    """One-hot rows and weights with their position in them: a row, column or block that is mixed up shows."""
    D, F, rows = 384, 512, 300
    xq = torch.zeros((rows, D), dtype=torch.uint8, device="cuda")
    xq[torch.arange(rows), torch.arange(rows) % D] = 0x38  # 1.0
    xs = (torch.arange(rows, device="cuda")[:, None] * 4 + torch.arange(3, device="cuda")[None] + 1).float()
    wq = torch.full((1, F, D), 0x38, dtype=torch.uint8, device="cuda")
    ws = torch.tensor([[1.0, 2.0, 4.0], [8.0, 16.0, 32.0], [64.0, 128.0, 256.0], [512.0, 1024.0, 2048.0]], device="cuda")[None]
    y = moe.moe_grouped_linear_e4m3_block(xq, xs, wq, ws)
    b = torch.arange(rows, device="cuda") % D // B
    want = xs[torch.arange(rows), b][:, None] * ws[0].repeat_interleave(B, 0)[:, b].T
    assert torch.equal(y, want.to(torch.bfloat16))


@pytest.mark.parametrize("bad", [[0, 5, 3, 9], [0, 4, 8, 11], [1, 4, 8, 9], [0, -2, 8, 9]], ids=str)
def test_offsets_that_are_no_prefix_sum_compute_nothing(moe, bad):
    xq, xs, wq, ws = forward_inputs([3, 3, 3], 128, 128)
    off = torch.tensor(bad, dtype=torch.int32, device="cuda")
    wsp = moe.workspace("grouped_linear_e4m3_block", N=9, D=128, E=3, Dff=128)
    y = torch.full((9, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    moe.moe_grouped_linear_e4m3_block(xq, xs, wq, ws, expert_offsets=off, y=y, ws=wsp)
    assert moe.read_device_error(wsp) == moe.MOE_ERR_DEVICE_BOUNDS and (y == 7).all()


def test_scale_indices_outside_count_as_zero(moe):
    xq, xs, wq, ws = forward_inputs([9], 128, 128)
    src = torch.arange(9, dtype=torch.int32, device="cuda")
    src[2], src[5] = -1, 9
    wsp = moe.workspace("combine")
    y = moe.moe_grouped_linear_e4m3_block(xq, xs, wq, ws, x_scale_index=src, ws=wsp)
    assert moe.read_device_error(wsp) == moe.MOE_ERR_DEVICE_BOUNDS
    zeroed = xs.clone()
    zeroed[2], zeroed[5] = 0, 0
    assert_within(y, *T.product(xq, zeroed, wq, ws, [9]), "y")


@pytest.mark.parametrize("kernel", ["1/1", "1/4", "2", "3"])
def test_withheld_load_ends_and_is_recorded(moe, monkeypatch, kernel):
    choose(monkeypatch, kernel)
    xq, xs, wq, ws = forward_inputs([300], 512, 256)
    wsp = moe.workspace("combine")
    moe.set_debug_flags(wsp, 1)
    moe.moe_grouped_linear_e4m3_block(xq, xs, wq, ws, ws=wsp)
    assert moe.read_device_error(wsp) == moe.MOE_ERR_DEVICE_TIMEOUT
    moe.clear_device_error(wsp)
    y = moe.moe_grouped_linear_e4m3_block(xq, xs, wq, ws, ws=wsp)
    assert moe.read_device_error(wsp) == 0
    assert_within(y, *T.product(xq, xs, wq, ws, [300]), "y")


@pytest.mark.parametrize("kernel", KERNELS)
def test_same_bits_every_time_and_in_a_graph(moe, monkeypatch, kernel):
    choose(monkeypatch, kernel)
    counts, D, F = [130, 0, 61, 300], 656, 528
    off = offsets_of(counts)
    xq, xs, wq, ws = forward_inputs(counts, D, F)
    (wb, wbs), (dyq, dys), seg = backward_inputs(moe, counts, D, F)
    wsp = moe.workspace("combine")

    def run(y, dx, dw):
        moe.moe_grouped_linear_e4m3_block(xq, xs, wq, ws, expert_offsets=off, y=y, ws=wsp)
        moe.moe_grouped_linear_e4m3_block_backward(wb, wbs, dyq, dys, *seg, expert_offsets=off, dx=dx, dw=dw, ws=wsp)

    def buffers():
        return [torch.empty(s, dtype=torch.bfloat16, device="cuda") for s in ((491, F), (491, D), (4, F, D))]

    first, again = buffers(), buffers()
    run(*first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(*again)
    for _ in range(3):
        graph.replay()
    for a, b in zip(first, again):
        assert torch.equal(a, b)
    assert moe.read_device_error(wsp) == 0


@pytest.mark.parametrize("kernel", ["1/1", "2", "3"])
def test_many_calls_of_ragged_tiles(moe, monkeypatch, kernel):
    """Tiles whose second half, last quarter or all but a row do not exist, in a long run of calls: no wait runs out and
    every call gives the same bits."""
    choose(monkeypatch, kernel)
    counts, D, F = [130, 1, 100, 256, 31, 385, 0, 97, 128], 2064, 1040
    off = offsets_of(counts)
    xq, xs, wq, ws = forward_inputs(counts, D, F)
    wsp = moe.workspace("combine")
    first = moe.moe_grouped_linear_e4m3_block(xq, xs, wq, ws, expert_offsets=off, ws=wsp)
    assert_within(first, *T.product(xq, xs, wq, ws, counts), "y")
    y = torch.empty_like(first)
    differs = torch.zeros((), dtype=torch.bool, device="cuda")
    for _ in range(1500):
        moe.moe_grouped_linear_e4m3_block(xq, xs, wq, ws, expert_offsets=off, y=y, ws=wsp)
        differs |= (y != first).any()
    assert moe.read_device_error(wsp) == 0 and not differs


def test_two_streams_at_once(moe):
    """Calls on two streams with a workspace each, many at a time."""
    sets = []
    for s in range(2):
        counts = [200, 31, 90]
        xq, xs, wq, ws = forward_inputs(counts, 528, 272, seed=10 + s)
        sets.append((torch.cuda.Stream(), xq, xs, wq, ws, offsets_of(counts), moe.workspace("combine"), []))
    torch.cuda.synchronize()
    for _ in range(8):
        for stream, xq, xs, wq, ws, off, wsp, out in sets:
            out.append(moe.moe_grouped_linear_e4m3_block(xq, xs, wq, ws, expert_offsets=off, ws=wsp, stream=stream))
    torch.cuda.synchronize()
    for _, xq, xs, wq, ws, _, wsp, out in sets:
        want = T.product(xq, xs, wq, ws, [200, 31, 90])
        assert moe.read_device_error(wsp) == 0
        for y in out:
            assert_within(y, *want, "y")
