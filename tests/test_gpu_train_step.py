"""A training step of the routed layer with block-scaled e4m3 products, as the operators are used together: every stage
against its 64-bit definition on what the stages before it wrote, in a stream of calls, in a graph, and its weights'
gradients against those of the unquantised layer."""
import pytest
import torch

import train_reference as T
from dense_reference import H, assert_within

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def moe(cuda_device):
    from mixture_experts_layer_02_gb300 import moe
    return moe


class Step:
    """out = x + sum_k w_k W2_k (silu(W1_k x) * W3_k x) and its gradient; W1 and W3 stacked as one product."""

    def __init__(self, moe, N, D, F, E, K, mode, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        normal = lambda *s, scale=1.0: (torch.randn(s, generator=g, device="cuda") * scale).to(BF16)
        self.moe, self.N, self.D, self.F, self.E, self.K, self.mode = moe, N, D, F, E, K, mode
        self.x, self.dout = normal(N, D), normal(N, D, scale=0.05)
        self.w_gate = normal(E, D, scale=D ** -0.5)
        self.w13, self.w2 = normal(E, 2 * F, D, scale=D ** -0.5), normal(E, D, F, scale=F ** -0.5)
        self.logits = torch.empty((N, E), dtype=torch.float32, device="cuda")
        self.q13, self.q2 = (moe.moe_quantize_e4m3_block(w, block_rows=128) for w in (self.w13, self.w2))
        self.ws = {op: moe.workspace(op, N=N, D=D, E=E, K=K) for op in ("route", "permute", "route_backward", "combine")}

    def forward(self):
        m, s = self.moe, self
        s.ids, s.w = m.moe_route(s.x, s.w_gate, None, s.K, s.mode, logits_out=s.logits, ws=s.ws["route"])
        s.off, s.src, s.inv, s.xp = m.moe_permute(s.x, s.ids, s.E, ws=s.ws["permute"])
        s.xq = m.moe_quantize_e4m3_segments(s.xp, s.off, ws=s.ws["combine"])
        s.gu = m.moe_grouped_linear_e4m3_block(s.xq[0], s.xq[1], *s.q13, expert_offsets=s.off, ws=s.ws["combine"])
        g, u = s.gu[:, :s.F].float(), s.gu[:, s.F:].float()
        s.h = (g * torch.sigmoid(g) * u).to(BF16)
        s.hq = m.moe_quantize_e4m3_segments(s.h, s.off, ws=s.ws["combine"])
        s.y = m.moe_grouped_linear_e4m3_block(s.hq[0], s.hq[1], *s.q2, expert_offsets=s.off, ws=s.ws["combine"])
        return m.moe_combine(s.y, s.inv, s.w, ws=s.ws["combine"])

    def backward(self):
        m, s = self.moe, self
        s.dy, s.dw = m.moe_combine_backward(s.dout, s.y, s.inv, s.w, ws=s.ws["combine"])
        s.dyq = m.moe_quantize_e4m3_segments(s.dy, s.off, ws=s.ws["combine"])
        s.dh, s.dw2 = m.moe_grouped_linear_e4m3_block_backward(*s.q2, *s.dyq, *s.hq[2:], expert_offsets=s.off, ws=s.ws["combine"])
        g, u, dh = s.gu[:, :s.F].float(), s.gu[:, s.F:].float(), s.dh.float()
        p = torch.sigmoid(g)
        s.dgu = torch.cat([dh * u * p * (1 + g * (1 - p)), dh * g * p], 1).to(BF16)
        s.dguq = m.moe_quantize_e4m3_segments(s.dgu, s.off, ws=s.ws["combine"])
        s.dxp, s.dw13 = m.moe_grouped_linear_e4m3_block_backward(*s.q13, *s.dguq, *s.xq[2:], expert_offsets=s.off, ws=s.ws["combine"])
        s.dxs = m.moe_permute_backward(s.dxp, s.inv, dresidual=s.dout, ws=s.ws["combine"])
        s.dx, s.dgate, s.dbias = m.moe_route_backward(s.dw, s.ids, s.w, s.logits, s.x, s.w_gate, s.mode, dresidual=s.dxs,
                                                      need_dbias=True, ws=s.ws["route_backward"])
        return s.dw2, s.dw13, s.dx, s.dgate, s.dbias

    def errors(self):
        return {op: self.moe.read_device_error(w) for op, w in self.ws.items() if self.moe.read_device_error(w)}


SIZES = [(1, 128, 144, 8, 2, 0), (77, 256, 272, 8, 2, 0), (300, 192, 80, 60, 6, 1), (512, 512, 256, 4, 2, 1)]


@pytest.mark.parametrize("N,D,F,E,K,mode", SIZES)
def test_every_stage(moe, N, D, F, E, K, mode):
    s = Step(moe, N, D, F, E, K, mode)
    s.forward()
    s.backward()
    assert not s.errors()
    counts = s.off.diff().tolist()
    for (v, q), name in (((s.xp, s.xq), "x"), ((s.h, s.hq), "h"), ((s.dy, s.dyq), "dy"), ((s.dgu, s.dguq), "dgu")):
        want = T.quantize(v, 1, 128)
        assert torch.equal(q[0], want[0]) and torch.equal(q[1], want[1]), name
        for e, a, b, pa, pb in T.spans(counts):
            if b > a:
                want = T.quantize(v[a:b], 128, 1)
                assert torch.equal(q[2][pa:pa + b - a], want[0]) and torch.equal(q[3][pa // 128:pb // 128], want[1]), name
                assert (q[2][pa + b - a:pb] == 0).all(), name
    assert_within(s.gu, *T.product(*s.xq[:2], *s.q13, counts), "gu")
    assert_within(s.y, *T.product(*s.hq[:2], *s.q2, counts), "y")
    (dy, e), (dw, ew), _ = T.combine_backward(s.dout, s.y, s.inv.cpu(), s.w)
    assert_within(s.dy, dy, e, "dy")
    assert_within(s.dw, dw, ew, "dw")
    want = T.product_backward(*s.dyq, *s.hq[2:], *s.q2, counts)
    assert_within(s.dh, *want[0], "dh")
    assert_within(s.dw2, *want[1], "dw2")
    want = T.product_backward(*s.dguq, *s.xq[2:], *s.q13, counts)
    assert_within(s.dxp, *want[0], "dxp")
    assert_within(s.dw13, *want[1], "dw13")
    assert_within(s.dxs, *T.permute_backward(s.dxp, s.inv.cpu(), s.dout), "dxs")
    want = T.route_backward(s.dw, s.ids, s.w, s.logits, s.x, s.w_gate, bool(mode), s.dxs)
    for got, (ref, e), name in zip((s.dx, s.dgate, s.dbias), want, ("dx", "dgate", "dbias")):
        assert_within(got, ref, e, name)


def test_gradients_point_where_the_unquantised_ones_do(moe):
    """Against autograd of the layer in 64 bits with the same choice of experts.  A code is off by at most 2^-4 of its
    value (or of the format's smallest), over all values about 2^-4 / sqrt 3 in the root mean square; a gradient here
    has up to six quantised operands behind it (x, W13, h, dy, W2, dgu), so sqrt(6) 2^-4 / sqrt 3 = 0.09 if they are
    independent, and 6 / sqrt 3 2^-4 = 0.22 if every one errs the same way."""
    s = Step(moe, 400, 256, 256, 8, 2, 0)
    s.forward()
    got = s.backward()
    x, g, w13, w2 = (t.double().requires_grad_() for t in (s.x, s.w_gate, s.w13, s.w2))
    logits = x @ g.T
    w = torch.softmax(torch.gather(logits, 1, s.ids.long()), 1)
    out = x.clone()
    for k in range(s.K):
        parts = []
        for t in range(s.N):
            e = int(s.ids[t, k])
            gu = w13[e] @ x[t]
            parts.append(w2[e] @ (gu[:s.F] * torch.sigmoid(gu[:s.F]) * gu[s.F:]))
        out = out + w[:, k:k + 1] * torch.stack(parts)
    want = torch.autograd.grad((out * s.dout.double()).sum(), (w2, w13, x, g))
    for a, b, name in zip(got, want, ("dw2", "dw13", "dx", "dgate")):
        off = (a.double() - b).norm() / b.norm()
        assert off <= 0.22 + 8 * H, (name, off.item())


@pytest.mark.parametrize("N,D,F,E,K,mode", SIZES[1:])
def test_stream_of_steps_and_graph_give_the_same_bits(moe, N, D, F, E, K, mode):
    s = Step(moe, N, D, F, E, K, mode)
    first = [s.forward(), *s.backward()]
    torch.cuda.synchronize()
    for _ in range(3):
        again = [s.forward(), *s.backward()]
    for a, b in zip(first, again):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = [s.forward(), *s.backward()]
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(first, captured):
        assert torch.equal(a, b)
    assert not s.errors()


def test_padded_paradigm_trains_too(moe):
    """Fixed capacity: the gradient's buffer is zero in rows without a token, so their products add nothing."""
    g = torch.Generator(device="cuda").manual_seed(3)
    N, D, F, E, K, cap = 90, 128, 144, 8, 2, 20
    x = torch.randn((N, D), generator=g, device="cuda").to(BF16)
    w = (torch.randn((E, F, D), generator=g, device="cuda") * D ** -0.5).to(BF16)
    ids = torch.rand((N, E), generator=g, device="cuda").topk(K, 1).indices.to(torch.int32)
    wt = torch.rand((N, K), generator=g, device="cuda")
    off, kept, slot, xp = moe.moe_permute_padded(x, ids, E, cap)
    assert (slot < 0).any() and (kept < cap).any()
    q, xs, xseg, xseg_s = moe.moe_quantize_e4m3_segments(xp, off)
    wq, ws = moe.moe_quantize_e4m3_block(w, block_rows=128)
    y = moe.moe_grouped_linear_e4m3_block(q, xs, wq, ws, expert_offsets=off)
    dout = torch.randn((N, F), generator=g, device="cuda").to(BF16)
    dy, _ = moe.moe_combine_backward(dout, y, slot, wt)
    dyq = moe.moe_quantize_e4m3_segments(dy, off)
    dx, dw = moe.moe_grouped_linear_e4m3_block_backward(wq, ws, *dyq, xseg, xseg_s, expert_offsets=off)
    counts = [cap] * E
    want_dx, want_dw = T.product_backward(*dyq, xseg, xseg_s, wq, ws, counts)
    assert_within(dx, *want_dx, "dx")
    assert_within(dw, *want_dw, "dw")
    assert_within(moe.moe_permute_backward(dx, slot), *T.permute_backward(dx, slot.cpu(), None), "dx of the tokens")
