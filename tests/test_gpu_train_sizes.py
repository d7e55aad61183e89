"""The training operators past 32-bit offsets and at their limits: many rows, many weights, many experts."""
import pytest
import torch

import train_reference as T
from dense_reference import H, U, assert_within

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
PAST = 2 ** 31


@pytest.fixture(scope="module")
def moe(cuda_device):
    from mixture_experts_layer_02_gb300 import moe
    yield moe
    torch.cuda.empty_cache()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def codes(g, *shape):
    """Codes 0x30 .. 0x3f with a sign: values of size 0.5 to 1.9."""
    return torch.randint(0x30, 0x40, shape, generator=g, device="cuda", dtype=torch.uint8) | (
        torch.randint(0, 2, shape, generator=g, device="cuda", dtype=torch.uint8) << 7)


def test_sort_gradients_past_32_bits(moe):
    N, D, K = 150_001, 7176, 2
    rows = N * K
    assert rows * D > PAST
    g = gen(1)
    y = torch.randint(-64, 64, (rows, D), generator=g, device="cuda", dtype=torch.int8).to(BF16)
    inv = torch.randperm(rows, generator=g, device="cuda").view(N, K).to(torch.int32)
    w = torch.rand((N, K), generator=g, device="cuda")
    dx = moe.moe_permute_backward(y, inv)
    some = torch.tensor([0, 1, N // 2, N - 1], device="cuda")
    want = y[inv[some].long()].double().sum(1)
    assert_within(dx[some], want, H * want.abs(), "dx")
    dout = dx
    dy, dw = moe.moe_combine_backward(dout, y, inv, w)
    for t in some.tolist():
        for k in range(K):
            r = int(inv[t, k])
            ref = w[t, k].double() * dout[t].double()
            assert_within(dy[r], ref, (H + 2 * U) * ref.abs(), "dy")
            a, b = dout[t].double(), y[r].double()
            assert abs(dw[t, k].double() - a @ b) <= (D + 2) * U * (a.abs() @ b.abs())
    last = inv.flatten().argmax().item()
    assert torch.isfinite(dy[-1]).all() and (dy[-1] != 0).any() and int(inv[last // K, last % K]) == rows - 1


def test_quantisers_past_32_bits(moe):
    rows, cols = 300_100, 7184
    assert rows * cols > PAST
    g = gen(2)
    src = torch.randint(-100, 100, (rows, cols), generator=g, device="cuda", dtype=torch.int8).to(BF16)
    off = torch.tensor([0, 100, 100, 299_900, rows], dtype=torch.int32, device="cuda")
    q, s, q_seg, s_seg = moe.moe_quantize_e4m3_segments(src, off)
    counts = off.diff().tolist()
    for e, a, b, pa, pb in T.spans(counts):
        if b == a:
            continue
        first = a + (b - a - 1) // 128 * 128  # the segment's last block
        want = T.quantize(src[first:b], 128, 1)
        at = pa + first - a
        assert torch.equal(q_seg[at:at + b - first], want[0]) and torch.equal(s_seg[at // 128:at // 128 + 1], want[1])
        assert (q_seg[at + b - first:pb] == 0).all()
        rows_want = T.quantize(src[first:b], 1, 128)
        assert torch.equal(q[first:b], rows_want[0]) and torch.equal(s[first:b], rows_want[1])
    tiles, scale = moe.moe_quantize_e4m3_block(src.view(1, rows, cols), block_rows=128)
    last = rows // 128 * 128
    want = T.quantize(src[last:], 128, 128)
    assert torch.equal(tiles[0, last:], want[0]) and torch.equal(scale[0, last // 128:], want[1])


@pytest.mark.parametrize("kernel", ["1", "2", "3", "4"])
def test_rows_past_32_bits(moe, monkeypatch, kernel):
    """A product whose rows' codes pass 2^31 bytes, its last rows among two experts."""
    monkeypatch.setenv("MOE_BLOCK_KERNEL", kernel)
    rows, D, F = 600_000, 4096, 32
    assert rows * D > PAST
    g = gen(3)
    if kernel == "4":  # a few rows an expert are meant; the last of many pass the limit all the same
        rows = 2 ** 19 + 40
    xq = codes(g, rows, D)
    xs = torch.rand((rows, D // 128), generator=g, device="cuda") + 0.5
    wq, ws = codes(g, 2, F, D), torch.rand((2, 1, D // 128), generator=g, device="cuda") + 0.5
    off = torch.tensor([0, rows - 20, rows], dtype=torch.int32, device="cuda")
    y = moe.moe_grouped_linear_e4m3_block(xq, xs, wq, ws, expert_offsets=off)
    for e, a, b in ((0, 0, 300), (0, rows - 320, rows - 20), (1, rows - 20, rows)):
        assert_within(y[a:b], *T.product(xq[a:b], xs[a:b], wq[e:e + 1], ws[e:e + 1], [b - a]), f"rows {a}..")


@pytest.mark.parametrize("kernel", ["1", "2", "3", "4"])
def test_weights_past_32_bits(moe, monkeypatch, kernel):
    """Weights of more than 2^31 codes: the last expert's, forward, and both gradients (the weight gradient has more
    than 2^31 elements too)."""
    monkeypatch.setenv("MOE_BLOCK_KERNEL", kernel)
    E, D, F, per = 48, 6160, 7440, 3
    assert E * D * F > PAST
    g = gen(4)
    wq = torch.empty((E, F, D), dtype=torch.uint8, device="cuda")
    for m in wq:
        m.copy_(codes(g, F, D))
    ws = torch.rand((E, T.blocks(F), T.blocks(D)), generator=g, device="cuda") + 0.5
    rows, counts = E * per, [per] * E
    off = torch.arange(0, rows + 1, per, dtype=torch.int32, device="cuda")
    xq, xs = codes(g, rows, D), torch.rand((rows, T.blocks(D)), generator=g, device="cuda") + 0.5
    y = moe.moe_grouped_linear_e4m3_block(xq, xs, wq, ws, expert_offsets=off)
    m = moe.segment_rows(rows, E)
    dyq, dys = codes(g, rows, F), torch.rand((rows, T.blocks(F)), generator=g, device="cuda") + 0.5
    seg = [codes(g, m, F), torch.rand((m // 128, F), generator=g, device="cuda") + 0.5, codes(g, m, D),
           torch.rand((m // 128, D), generator=g, device="cuda") + 0.5]
    for _, a, b, pa, pb in T.spans(counts):
        seg[0][pa + per:pb] = 0
        seg[2][pa + per:pb] = 0
    dx, dw = moe.moe_grouped_linear_e4m3_block_backward(wq, ws, dyq, dys, *seg, expert_offsets=off)
    for e in (0, E - 1):
        a, pa = e * per, e * 128
        assert_within(y[a:a + per], *T.product(xq[a:a + per], xs[a:a + per], wq[e:e + 1], ws[e:e + 1], [per]), f"y of {e}")
        cut = [seg[0][pa:pa + 128], seg[1][e:e + 1], seg[2][pa:pa + 128], seg[3][e:e + 1]]
        want_dx, want_dw = T.product_backward(dyq[a:a + per], dys[a:a + per], *cut, wq[e:e + 1], ws[e:e + 1], [per])
        assert_within(dx[a:a + per], *want_dx, f"dx of {e}")
        assert_within(dw[e], want_dw[0][0], want_dw[1][0], f"dw of {e}")


@pytest.mark.parametrize("kernel", ["1/1", "1/4", "2", "3", "4/2", ""])
def test_as_many_experts_as_there_can_be(moe, monkeypatch, kernel):
    if kernel:
        k, _, s = kernel.partition("/")
        monkeypatch.setenv("MOE_BLOCK_KERNEL", k)
        monkeypatch.setenv("MOE_BLOCK_SPLIT", s or "1")
    g = gen(5)
    E, D, F = 1024, 48, 32
    counts = torch.randint(0, 4, (E,), generator=g, device="cuda")
    counts[::7], counts[500], counts[1023] = 0, 300, 5
    off = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
    counts = counts.tolist()
    rows = sum(counts)
    xq, xs = codes(g, rows, D), torch.rand((rows, 1), generator=g, device="cuda")
    wq, ws = codes(g, E, F, D), torch.rand((E, 1, 1), generator=g, device="cuda")
    y = moe.moe_grouped_linear_e4m3_block(xq, xs, wq, ws, expert_offsets=off)
    assert_within(y, *T.product(xq, xs, wq, ws, counts), "y")
    dy = (torch.randn((rows, F), generator=g, device="cuda")).to(BF16)
    x = (torch.randn((rows, D), generator=g, device="cuda")).to(BF16)
    dyq, dxq = moe.moe_quantize_e4m3_segments(dy, off), moe.moe_quantize_e4m3_segments(x, off, both=False)
    dx, dw = moe.moe_grouped_linear_e4m3_block_backward(wq, ws, *dyq, *dxq[2:], expert_offsets=off)
    want_dx, want_dw = T.product_backward(*dyq, *dxq[2:], wq, ws, counts)
    assert_within(dx, *want_dx, "dx")
    assert_within(dw, *want_dw, "dw")


@pytest.mark.parametrize("kernel", ["1/1", "1/2", "2", "3", "4/4"])
def test_infinite_scales_and_nan_codes_stay_with_their_rows(moe, monkeypatch, kernel):
    """A NaN code or an infinite scale of one row reaches that row alone, and one of a weight's block its own columns; codes
    behind a matrix (the next expert's, NaN here) reach nothing, though boxes of 128 are read."""
    k, _, s = kernel.partition("/")
    monkeypatch.setenv("MOE_BLOCK_KERNEL", k)
    monkeypatch.setenv("MOE_BLOCK_SPLIT", s or "1")
    g = gen(6)
    D, F = 144, 272  # neither a multiple of 128: boxes reach past both
    xq, xs = codes(g, 200, D), torch.rand((200, 2), generator=g, device="cuda") + 0.5
    wq, ws = codes(g, 2, F, D), torch.rand((2, 3, 2), generator=g, device="cuda") + 0.5
    off = torch.tensor([0, 150, 200], dtype=torch.int32, device="cuda")
    clean = moe.moe_grouped_linear_e4m3_block(xq, xs, wq, ws, expert_offsets=off)
    xq[150:] = 0x7f
    wq[1] = 0x7f
    got = moe.moe_grouped_linear_e4m3_block(xq, xs, wq, ws, expert_offsets=off)
    assert torch.equal(got[:150], clean[:150]) and got[150:].isnan().all()
    xq[3, 7], xs[5, 1] = 0x7f, float("inf")
    got = moe.moe_grouped_linear_e4m3_block(xq, xs, wq, ws, expert_offsets=off)
    keep = [r for r in range(150) if r not in (3, 5)]
    assert got[3].isnan().all() and not got[5].isfinite().any() and torch.equal(got[keep], clean[keep])
    ws[0, 1, 0] = float("nan")  # columns 128 .. 255
    got = moe.moe_grouped_linear_e4m3_block(xq, xs, wq, ws, expert_offsets=off)
    assert got[keep][:, 128:256].isnan().all()
    assert torch.equal(got[keep][:, :128], clean[keep][:, :128]) and torch.equal(got[keep][:, 256:], clean[keep][:, 256:])
    dyq, dys = codes(g, 200, F), torch.rand((200, 3), generator=g, device="cuda") + 0.5
    m = moe.segment_rows(200, 2)
    seg = [codes(g, m, F), torch.ones((m // 128, F), device="cuda"), codes(g, m, D), torch.ones((m // 128, D), device="cuda")]
    seg[0][150:256], seg[2][150:256] = 0, 0
    seg[0][256:], seg[2][256:] = 0x7f, 0x7f
    ws[0, 1, 0] = 1.0
    dx, dw = moe.moe_grouped_linear_e4m3_block_backward(wq, ws, dyq, dys, *seg, expert_offsets=off)
    want_dx, want_dw = T.product_backward(dyq[:150], dys[:150], *[t[:256 if i % 2 == 0 else 2] for i, t in enumerate(seg)], wq[:1],
                                          ws[:1], [150])
    assert_within(dx[:150], *want_dx, "dx")
    assert dx[150:].isnan().all() and dw[1].isnan().all()
    assert_within(dw[0], want_dw[0][0], want_dw[1][0], "dw")
