"""The feed-forward block example: the dense operators with the MoE layer, as they are used together."""
import dataclasses
import os
import sys

import pytest
import torch

import dense_reference as R

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module")
def block(cuda_device):
    import ffn_block
    from mixture_experts_layer_02_gb300 import synth
    wl = dataclasses.replace(synth.WORKLOADS["qwen3_N1"], name="block", N=64, D=512, E=16, Dff=256)
    return ffn_block.Block.make(wl, shared=264)


def tokens(n, d, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn((n, d), generator=g, device="cuda").to(torch.bfloat16)


@pytest.mark.parametrize("n", [1, 3, 64])
def test_forward_is_the_layer_plus_the_shared_expert(block, n):
    from mixture_experts_layer_02_gb300 import moe
    wl = block.wl
    x, res = tokens(n, wl.D, 1), tokens(n, wl.D, 2)
    out, s = block.forward(x, res)
    s64, y64 = R.norm(x, block.norm, res)
    assert torch.equal(s, s64.float().to(torch.bfloat16))
    y = moe.moe_rmsnorm(x, block.norm, residual=res)[0]
    layer = moe.moe_layer_forward_e4m3(y, block.w_gate, None, block.experts, wl.K, wl.mode, wl.act)
    h = (R.act(y64 @ block.w1.double().T, "silu") * (y64 @ block.w3.double().T)) @ block.w2.double().T
    got, want = out.double() - h, layer.double()
    # the layer call quantises the bf16 rows, the block the norm's fp32 rows: codes may differ by one step,
    # 2^-4 relative each, over hundreds of terms of random sign; h and y round to bf16 on both sides
    assert (got - want).norm() <= 0.05 * (want.norm() + h.norm())


def test_dense_gradients_match_the_formulas(block):
    wl = block.wl
    x, res, dout = tokens(48, wl.D, 1), tokens(48, wl.D, 2), tokens(48, wl.D, 3)
    out, kept = block.dense(x, res)
    got = block.dense_backward(dout, kept)
    leaves = [t.double().requires_grad_() for t in (x, block.norm, block.w1, block.w3, block.w2)]
    lx, ln, l1, l3, l2 = leaves
    s = lx + res.double()
    y = s * (s.square().mean(1, keepdim=True) + 1e-6).rsqrt() * ln
    g = y @ l1.T
    ref = s + (g * torch.sigmoid(g) * (y @ l3.T)) @ l2.T
    assert (out.double() - ref).norm() <= 4 * R.H * ref.norm()
    want = torch.autograd.grad((ref * dout.double()).sum(), leaves)
    for a, b, name in zip(got, want, ("dx", "dnorm", "dw1", "dw3", "dw2")):
        # a handful of bf16 roundings on the way (y, g, u, h, dh, dg, du, the gradient), each 2^-8 at most
        assert (a.double() - b).norm() <= 8 * R.H * b.norm(), name


def test_training_lowers_the_loss(block):
    import ffn_block
    b = ffn_block.Block.make(block.wl, shared=512, seed=5)
    x, res, target = (tokens(64, b.wl.D, s) for s in (11, 12, 13))
    losses = [b.train_step(x, res, target, lr=5.0).item() for _ in range(12)]
    assert losses[-1] < 0.9 * losses[0], losses
