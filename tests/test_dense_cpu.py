"""CPU checks of the dense operators: refusals of the C entry points before
anything reaches a GPU, workspace sizes, and the reference formulas of the GPU
tests against finite differences."""
import ctypes

import pytest
import torch

import dense_reference as R

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    from mixture_experts_layer_02_gb300 import build, moe
    build.build()
    return moe.load()


# placeholders that pass the alignment check; no call below may reach a launch
X, Y, Z, W = P(4096), P(8192), P(12288), P(16384)


def norm(lib, x=X, residual=None, weight=W, N=4, D=64, eps=1e-6, y=Y, yq=None, y_scale=None, out=None):
    return lib.moe_rmsnorm(x, residual, weight, N, D, eps, y, yq, y_scale, out, None)


@pytest.mark.parametrize("kw,status", [
    (dict(N=-1), 1), (dict(D=0), 1), (dict(D=12), 1), (dict(D=1 << 20), 2), (dict(eps=-1.0), 1),
    (dict(eps=float("nan")), 1), (dict(x=None), 1), (dict(weight=None), 1), (dict(x=P(4100)), 1), (dict(y=P(8200)), 1),
    (dict(residual=P(4104)), 1), (dict(y=None), 1), (dict(yq=Z), 1), (dict(y_scale=Z), 1),
])
def test_norm_refusals(lib, kw, status):
    assert norm(lib, **kw) == status
    assert lib.moe_last_error_detail() != b""


def test_empty_forward_calls_are_no_ops(lib):
    assert norm(lib, N=0, x=None) == 0
    assert lib.moe_gated_linear(None, None, None, 0, 64, 64, 2, None, None, None, None, 0, None) == 0
    assert lib.moe_linear(None, None, None, None, 0, 64, 64, 0, None, None, None, 0, None) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(N=-1), 1), (dict(D=4), 1), (dict(D=65), 1), (dict(F=0), 1), (dict(F=60), 1), (dict(fn=5), 1), (dict(fn=-1), 1),
    (dict(x=None), 1), (dict(w=None), 1), (dict(w=P(16386)), 1), (dict(out=None), 1), (dict(ws=None), 1),
    (dict(ws=P(24584)), 1), (dict(ws_bytes=255), 3), (dict(D=1 << 30, F=1 << 30), 1),
])
def test_product_refusals(lib, kw, status):
    a = dict(x=X, w=W, out=Y, N=4, D=64, F=64, fn=2, ws=P(24576), ws_bytes=256) | kw
    got = lib.moe_gated_linear(a["x"], a["w"], a["w"], a["N"], a["D"], a["F"], a["fn"], a["out"], None, None, a["ws"],
                               a["ws_bytes"], None)
    assert got == status
    got = lib.moe_linear(a["x"], a["w"], None, None, a["N"], a["D"], a["F"], a["fn"], a["out"], None, a["ws"],
                         a["ws_bytes"], None)
    assert got == status


def test_backward_refusals(lib):
    big = 1 << 30
    # dw1 without dw3
    assert lib.moe_gated_linear_backward(X, X, W, W, X, X, 4, 64, 64, 2, Y, Z, None, P(24576), big, None) == 1
    # g missing; workspace too small
    assert lib.moe_gated_linear_backward(X, X, W, W, None, X, 4, 64, 64, 2, Y, Z, Z, P(24576), big, None) == 1
    assert lib.moe_gated_linear_backward(X, X, W, W, X, X, 4, 64, 64, 2, Y, Z, Z, P(24576), 256, None) == 3
    # an activation without its pre-activation
    assert lib.moe_linear_backward(X, X, W, None, 4, 64, 64, 2, Y, Z, None, P(24576), big, None) == 1
    assert lib.moe_linear_backward(X, X, W, None, 4, 64, 64, 0, Y, Z, None, P(24576), 256, None) == 3
    # norm: dx missing, workspace too small
    assert lib.moe_rmsnorm_backward(X, X, W, None, 4, 64, 1e-6, None, Z, P(24576), big, None) == 1
    assert lib.moe_rmsnorm_backward(X, X, W, None, 4, 64, 1e-6, Y, Z, P(24576), 256, None) == 3


def test_workspace_sizes(lib):
    from mixture_experts_layer_02_gb300 import moe
    assert moe.workspace_size("gated_linear", N=7, D=64, Dff=72) == 256
    assert moe.workspace_size("linear", N=7, D=64, Dff=72) == 256
    assert moe.workspace_size("linear", N=7, D=60, Dff=72) == 0
    assert moe.workspace_size("gated_linear_backward", N=100, D=64, Dff=72) >= 256 + 2 * 100 * 72 * 2
    assert moe.workspace_size("linear_backward", N=100, D=64, Dff=72) >= 256 + 100 * 72 * 2
    assert moe.workspace_size("rmsnorm_backward", N=100, D=64) >= 256 + 64 * 4
    assert moe.workspace_size("rmsnorm_backward", N=100, D=65536) == 0


def test_binding_refuses_what_the_kernels_cannot_take():
    from mixture_experts_layer_02_gb300 import moe
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.ones(64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        moe.moe_rmsnorm(x, w)
    with pytest.raises(TypeError, match="expected torch.bfloat16"):
        moe.moe_rmsnorm(x.float(), w)
    with pytest.raises(ValueError, match="rows, width"):
        moe.moe_linear(x[0], torch.zeros(8, 64, dtype=torch.bfloat16))


# ------------------------------------------------------------------ the reference against differences
def _difference(f, t, direction, step=1e-5):
    return (f(t + step * direction) - f(t - step * direction)) / (2 * step)


@pytest.mark.parametrize("fn", sorted(R.FNS))
def test_reference_gradients_against_differences(fn):
    torch.manual_seed(1)
    n, d, f = 5, 16, 24
    x, w1, w3 = torch.randn(n, d).double(), torch.randn(f, d).double() / 4, torch.randn(f, d).double() / 4
    up = torch.randn(n, f).double()
    g, u = x @ w1.T, x @ w3.T
    (dx, _), (dw1, _), (dw3, _) = R.gated_backward(up, x, w1, w3, g, u, fn)

    def loss(x, w1, w3):
        return (R.act(x @ w1.T, fn) * (x @ w3.T) * up).sum()

    for grad, t, put in ((dx, x, lambda v: loss(v, w1, w3)), (dw1, w1, lambda v: loss(x, v, w3)),
                         (dw3, w3, lambda v: loss(x, w1, v))):
        v = torch.randn_like(t)
        assert abs((grad * v).sum() - _difference(put, t, v)) <= 1e-6 * (grad.norm() * v.norm())
    b = torch.randn(f).double()
    (dx, _), (dw, _), (db, _) = R.linear_backward(up, x, w1, x @ w1.T + b, fn)
    for grad, t, put in ((dx, x, lambda v: (R.act(v @ w1.T + b, fn) * up).sum()),
                         (dw, w1, lambda v: (R.act(x @ v.T + b, fn) * up).sum()),
                         (db, b, lambda v: (R.act(x @ w1.T + v, fn) * up).sum())):
        v = torch.randn_like(t)
        assert abs((grad * v).sum() - _difference(put, t, v)) <= 1e-6 * (grad.norm() * v.norm())


def test_reference_norm_gradient_against_differences():
    torch.manual_seed(2)
    s, w, up, down = (torch.randn(*sh).double() for sh in ((6, 24), (24,), (6, 24), (6, 24)))
    dx, dw, _, _ = R.norm_backward(up, s, w, down)
    for grad, t, put in ((dx, s, lambda v: (R.norm(v, w)[1] * up + v * down).sum()),
                         (dw, w, lambda v: (R.norm(s, v)[1] * up).sum())):
        v = torch.randn_like(t)
        assert abs((grad * v).sum() - _difference(put, t, v)) <= 1e-6 * (grad.norm() * v.norm())


def test_reference_scale_rule():
    y = torch.tensor([[448.0, 1.0], [448.5, 0.0], [1.0, -0.5], [0.0, 0.0], [-896.0, 3.0]]).double()
    assert R.norm_scale(y).tolist() == [1.0, 2.0, 2.0 ** -8, 2.0 ** -126, 2.0]
