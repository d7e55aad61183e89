"""CPU checks of the routed layer's training operators: refusals before anything reaches a GPU, workspace and buffer
sizes, rules of their sources, and the reference formulas of the GPU tests against differences and by hand."""
import ctypes

import pytest
import torch

import train_reference as T
from test_dense_rules_cpu import kernels, source

P = ctypes.c_void_p
X, Y, Z, W, V, S = (P(4096 * i) for i in range(1, 7))  # placeholders that pass the alignment check
BIG = 1 << 40


@pytest.fixture(scope="module")
def moe():
    from mixture_experts_layer_02_gb300 import build, moe
    build.build()
    moe.load()
    return moe


@pytest.fixture(scope="module")
def lib(moe):
    return moe.load()


# ------------------------------------------------------------------ refusals
@pytest.mark.parametrize("kw,status", [
    (dict(N=-1), 1), (dict(D=0), 1), (dict(D=12), 1), (dict(K=0), 1), (dict(K=33), 1), (dict(rows=-1), 1), (dict(ws=None), 1),
    (dict(ws_bytes=255), 3), (dict(inv=None), 1), (dict(inv=P(4100)), 1), (dict(N=1 << 30, K=8), 1), (dict(N=1 << 20, D=1 << 21), 1),
    (dict(x=None), 1), (dict(out=None), 1), (dict(out=P(8200)), 1),
])
def test_sort_gradient_refusals(lib, kw, status):
    a = dict(x=X, inv=Y, w=Z, N=4, D=64, K=2, rows=8, out=W, ws=S, ws_bytes=256) | kw
    assert lib.moe_permute_backward(a["x"], a["inv"], None, a["N"], a["D"], a["K"], a["rows"], a["out"], a["ws"], a["ws_bytes"],
                                    None) == status
    assert lib.moe_combine_backward(a["x"], X, a["inv"], a["w"], a["N"], a["D"], a["K"], a["rows"], a["out"], None, a["ws"],
                                    a["ws_bytes"], None) == status
    assert lib.moe_last_error_detail() != b""


def test_combine_gradient_needs_what_it_reads(lib):
    call = lambda y, w, dy, dw: lib.moe_combine_backward(X, y, Y, w, 4, 64, 2, 8, dy, dw, S, 256, None)
    assert call(None, Z, W, V) == 1  # dtopk_w is a product with y_perm
    assert call(Z, None, W, V) == 1
    assert call(Z, Z, None, P(4100)) == 1


@pytest.mark.parametrize("kw,status", [
    (dict(N=-1), 1), (dict(D=12), 1), (dict(E=0), 1), (dict(E=1025), 1), (dict(K=0), 1), (dict(K=9), 1), (dict(mode=2), 1),
    (dict(dw=None), 1), (dict(ids=None), 1), (dict(w=None), 1), (dict(logits=None, mode=1), 1), (dict(x=None), 1), (dict(wg=None), 1),
    (dict(dx=None, dg=None, db=None), 1), (dict(res=P(4104)), 1), (dict(db=P(4104)), 1), (dict(ws=None), 1), (dict(ws_bytes=256), 3),
])
def test_route_gradient_refusals(lib, kw, status):
    a = dict(dw=X, ids=Y, w=Z, logits=W, x=X, wg=Y, res=None, N=4, D=64, E=8, K=2, mode=0, dx=V, dg=W, db=Z, ws=S,
             ws_bytes=BIG) | kw
    assert lib.moe_route_backward(a["dw"], a["ids"], a["w"], a["logits"], a["x"], a["wg"], a["res"], a["N"], a["D"], a["E"], a["K"],
                                  a["mode"], a["dx"], a["dg"], a["db"], a["ws"], a["ws_bytes"], None) == status


@pytest.mark.parametrize("kw", [dict(mats=-1), dict(rows=-1), dict(cols=8), dict(cols=0), dict(cols=136), dict(block_rows=2),
                                dict(cols=2 ** 31 - 16), dict(rows=2 ** 31 - 1), dict(mats=1 << 20, rows=1 << 20), dict(src=None),
                                dict(q=None), dict(scale=None), dict(q=P(4097))])
def test_quantiser_refusals(lib, kw):
    a = dict(src=X, mats=1, rows=4, cols=64, block_rows=1, q=Y, scale=Z) | kw
    assert lib.moe_quantize_e4m3_block(a["src"], a["mats"], a["rows"], a["cols"], a["block_rows"], a["q"], a["scale"], None) == 1


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), 1), (dict(cols=24), 1), (dict(E=0), 1), (dict(E=1025), 1), (dict(off=None), 1), (dict(q=None), 1),
    (dict(scale=None), 1), (dict(q_seg=None), 1), (dict(s_seg=None), 1), (dict(src=None), 1), (dict(ws=None), 1),
    (dict(ws_bytes=0), 3), (dict(rows=2 ** 31 - 1), 1),
])
def test_segment_quantiser_refusals(lib, kw, status):
    a = dict(src=X, off=Y, rows=9, cols=64, E=3, q=Z, scale=W, q_seg=V, s_seg=X, ws=S, ws_bytes=256) | kw
    assert lib.moe_quantize_e4m3_segments(a["src"], a["off"], a["rows"], a["cols"], a["E"], a["q"], a["scale"], a["q_seg"], a["s_seg"],
                                          a["ws"], a["ws_bytes"], None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), 1), (dict(D=24), 1), (dict(F=8), 1), (dict(E=0), 1), (dict(E=1025), 1), (dict(off=None), 1), (dict(xq=None), 1),
    (dict(xs=None), 1), (dict(wq=None), 1), (dict(ws_=None), 1), (dict(y=None), 1), (dict(y=P(4098)), 1), (dict(ws=None), 1),
    (dict(ws_bytes=128), 3), (dict(n=8), 1), (dict(rows=2 ** 31 - 1, n=2 ** 31 - 1), 1), (dict(D=1 << 20, F=1 << 20), 1),
    (dict(D=(1 << 30) + 16), 1),
])
def test_block_product_refusals(lib, kw, status):
    a = dict(xq=X, xs=Y, idx=None, n=9, off=Z, rows=9, wq=W, ws_=V, E=3, D=64, F=64, y=X, ws=S, ws_bytes=256) | kw
    assert lib.moe_grouped_linear_e4m3_block(a["xq"], a["xs"], a["idx"], a["n"], a["off"], a["rows"], a["wq"], a["ws_"], a["E"], a["D"],
                                             a["F"], a["y"], a["ws"], a["ws_bytes"], None) == status
    if not {"xq", "xs", "y", "n"} & set(kw):
        assert lib.moe_grouped_linear_e4m3_block_backward(X, Y, X, Y, X, Y, a["off"], a["rows"], a["wq"], a["ws_"], a["E"], a["D"],
                                                          a["F"], W, V, a["ws"], a["ws_bytes"], None) == status


@pytest.mark.parametrize("missing", range(6))
def test_block_gradients_need_their_own_operands(lib, missing):
    ops = [X, Y, Z, W, V, X]
    ops[missing] = None
    call = lambda dx, dw: lib.moe_grouped_linear_e4m3_block_backward(*ops, Z, 9, X, Y, 3, 64, 64, dx, dw, S, 256, None)
    dx, dw = (V, None) if missing < 2 else (None, V)
    assert call(dx, dw) == 1
    assert call(None, None) == 1


def test_empty_calls_are_no_ops(lib):
    assert lib.moe_combine_backward(None, None, None, None, 0, 64, 2, 0, None, None, None, 0, None) == 0
    assert lib.moe_permute_backward(None, None, None, 0, 64, 2, 0, None, None, 0, None) == 0
    assert lib.moe_quantize_e4m3_block(None, 1, 0, 64, 1, None, None, None) == 0
    assert lib.moe_quantize_e4m3_segments(None, X, 0, 64, 3, None, None, None, None, None, 0, None) == 0
    assert lib.moe_grouped_linear_e4m3_block(None, None, None, 0, X, 0, None, None, 3, 64, 64, None, None, 0, None) == 0
    assert lib.moe_grouped_linear_e4m3_block_backward(None, None, None, None, None, None, X, 0, None, None, 3, 64, 64, Y, None, None,
                                                      0, None) == 0


# ------------------------------------------------------------------ the binding's own checks
def test_binding_names_what_does_not_fit(moe):
    z = lambda *s, d=torch.bfloat16: torch.zeros(s, dtype=d)
    with pytest.raises(ValueError, match="src: must be a contiguous CUDA tensor"):
        moe.moe_quantize_e4m3_block(z(4, 64))
    with pytest.raises(ValueError, match="src: expected"):
        moe.moe_quantize_e4m3_block(z(64))
    with pytest.raises(TypeError, match="src: expected torch.bfloat16"):
        moe.moe_quantize_e4m3_block(z(4, 64, d=torch.float32))
    with pytest.raises(ValueError, match="scale: expected shape"):
        moe.moe_quantize_e4m3_block(z(4, 64), scale=z(4, 2, d=torch.float32))
    with pytest.raises(ValueError, match="wq: expected"):
        moe.moe_grouped_linear_e4m3_block(z(4, 64, d=torch.uint8), z(4, 1, d=torch.float32), z(64, 64, d=torch.uint8), None)
    with pytest.raises(ValueError, match="w_scale: expected shape"):
        moe.moe_grouped_linear_e4m3_block(z(4, 64, d=torch.uint8), z(4, 1, d=torch.float32), z(1, 256, 64, d=torch.uint8),
                                          z(1, 1, 1, d=torch.float32))
    with pytest.raises(ValueError, match="inv_perm: expected"):
        moe.moe_permute_backward(z(4, 64), z(4, d=torch.int32))
    with pytest.raises(ValueError, match="logits: needed"):
        moe.moe_route_backward(z(4, 2, d=torch.float32), z(4, 2, d=torch.int32), z(4, 2, d=torch.float32), None, z(4, 64), z(8, 64),
                               moe.SIGMOID_NORM)


def test_sizes(moe):
    assert [moe.segment_rows(r, e) for r, e in ((0, 8), (1, 8), (2, 1), (128, 1), (129, 1), (9, 3), (32768, 256))] == \
        [0, 128, 128, 128, 256, 384, 65280]
    for rows, E in ((0, 3), (1, 1), (5, 256), (300, 4), (32768, 256)):
        assert moe.segment_rows(rows, E) == T.segment_rows(rows, E)
    for bad in ((-1, 4), (4, 0), (4, 1025)):
        with pytest.raises(ValueError):
            moe.segment_rows(*bad)
    # header, the gradient of the logits (rows of E rounded up to 8) and the bias's partial sums of 8 tokens
    assert moe.workspace_size("route_backward", N=100, D=64, E=60) == 256 + 12800 + 3328
    assert moe.workspace_size("route_backward", N=100, D=63, E=60) == 0
    assert moe.workspace_size("grouped_linear_e4m3_block", N=9, D=64, E=3, Dff=64) == 256
    assert moe.workspace_size("grouped_linear_e4m3_block_backward", N=9, D=65, E=3, Dff=64) == 0


# ------------------------------------------------------------------ rules of the sources
SOURCES = ["routing_grad.cu", "quant_block.cu", "block_gemm.cuh", "block_gemv.cu"]


@pytest.mark.parametrize("name", SOURCES)
def test_dependents_start_after_the_own_wait(name):
    """Two launches overlap at most: a launch lets the next one start only behind its own wait."""
    text = source(name)
    found = kernels(text)
    assert len(found) == text.count("__global__")
    for kernel, body in found:
        assert body.count("pdl_wait()") == 1, kernel
        assert 0 <= body.index("pdl_wait()") < body.index("pdl_trigger()"), kernel


@pytest.mark.parametrize("name", SOURCES)
def test_no_loads_through_the_non_coherent_path(name):
    text = source(name)
    for word in (".nc.", ".nc ", "__ldg", "__restrict__"):
        assert word not in text, word


# ------------------------------------------------------------------ the reference formulas
def test_reference_scale_rule_by_hand():
    top = torch.tensor([0.0, 448.0, 449.0, 896.0, 1.0, 1.75, 2.0 ** -130, 3e38], dtype=torch.float64)
    assert T.scale_of(top).tolist() == [2.0 ** -126, 1.0, 2.0, 2.0, 2.0 ** -8, 2.0 ** -8, 2.0 ** -126, 2.0 ** 120]


def test_reference_quantiser_by_hand():
    v = torch.zeros((130, 144), dtype=torch.bfloat16)
    v[0, 0], v[0, 130], v[129, 0] = 448.0, 1.0, 3.0
    q, s = T.quantize(v, 1, 128)
    assert s[0].tolist() == [1.0, 2.0 ** -8] and s[1].tolist() == [2.0 ** -126] * 2 and s[129, 0] == 2.0 ** -7
    assert torch.equal(T.values(q, s, 1, 128), v.double())
    q, s = T.quantize(v, 128, 128)
    assert s.tolist() == [[1.0, 2.0 ** -8], [2.0 ** -7, 2.0 ** -126]] and torch.equal(T.values(q, s, 128, 128), v.double())
    q, s = T.quantize(v, 128, 1)
    assert s[0, 0] == 1.0 and s[1, 0] == 2.0 ** -7 and s[0, 130] == 2.0 ** -8


def test_reference_product_gradients_are_those_of_the_product():
    """The gradients' definitions against autograd of the forward definition, on operands that all forms hold exactly."""
    g = torch.Generator().manual_seed(0)
    counts, D, F = [3, 0, 130], 32, 48
    rows = sum(counts)
    x = torch.randint(-8, 9, (rows, D), generator=g).to(torch.bfloat16)
    w = torch.randint(-8, 9, (3, F, D), generator=g).to(torch.bfloat16)
    dy = torch.randint(-8, 9, (rows, F), generator=g).to(torch.bfloat16)
    wq = [T.quantize(m, 128, 128) for m in w]
    wq, ws = torch.stack([q for q, _ in wq]), torch.stack([s for _, s in wq])
    seg = T.segment_rows(rows, 3)

    def segments(v):
        q, s = torch.zeros((seg, v.shape[1]), dtype=torch.uint8), torch.ones((seg // 128, v.shape[1]))
        for _, a, b, pa, pb in T.spans(counts):
            if b > a:
                q[pa:pa + b - a], s[pa // 128:pb // 128] = T.quantize(v[a:b], 128, 1)
        return q, s

    xl, wl = x.double().requires_grad_(), w.double().requires_grad_()
    y = torch.cat([xl[a:b] @ wl[e].T for e, a, b, _, _ in T.spans(counts)])
    want = torch.autograd.grad((y * dy.double()).sum(), (xl, wl))
    assert torch.equal(T.product(*T.quantize(x, 1, 128), wq, ws, counts)[0], y.detach())
    (dx, _), (dw, _) = T.product_backward(*T.quantize(dy, 1, 128), *segments(dy), *segments(x), wq, ws, counts)
    assert torch.equal(dx, want[0]) and torch.equal(dw, want[1])


def test_reference_sort_gradients_are_those_of_the_sums():
    g = torch.Generator().manual_seed(1)
    N, D, K = 5, 8, 3
    y = torch.randn((N * K, D), generator=g).double().requires_grad_()
    w = torch.rand((N, K), generator=g).double().requires_grad_()
    x = torch.randn((N, D), generator=g).double().requires_grad_()
    inv = torch.randperm(N * K, generator=g).view(N, K)
    dout = torch.randn((N, D), generator=g).double()
    out = (w.unsqueeze(2) * y[inv]).sum(1)
    want = torch.autograd.grad((out * dout).sum(), (y, w))
    (dy, _), (dw, _), named = T.combine_backward(dout, y.detach(), inv, w.detach())
    assert named.all() and torch.allclose(dy, want[0], rtol=1e-12) and torch.allclose(dw, want[1], rtol=1e-12)
    x_perm = torch.empty_like(y).index_copy(0, inv.flatten(), x.repeat_interleave(K, 0))
    want_x, = torch.autograd.grad((x_perm * y.detach()).sum(), x)
    assert torch.allclose(T.permute_backward(y.detach(), inv, None)[0], want_x, rtol=1e-12)
