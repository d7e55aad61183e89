"""The feed-forward block example keeps its workspaces: a kernel that gave up is not lost."""
import dataclasses
import os
import sys

import pytest
import torch

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


def test_check_tells_of_a_kernel_that_gave_up(block):
    from mixture_experts_layer_02_gb300 import moe
    x, res = tokens(64, block.wl.D, 1), tokens(64, block.wl.D, 2)
    want, _ = block.forward(x, res)
    block.check()
    for op in ("gated_linear", "linear"):
        moe.set_debug_flags(block.kept[op][-1], 1)
        block.forward(x, res)
        with pytest.raises(moe.MoEError, match=op):
            block.check()
        block.check()  # told once
        assert torch.equal(block.forward(x, res)[0], want)
    block.check()


def test_check_covers_the_gradients_and_outgrown_workspaces(block):
    from mixture_experts_layer_02_gb300 import moe
    small, large = (tokens(n, block.wl.D, 3) for n in (40, 200))
    _, kept = block.dense(small, small)
    for op in ("linear_backward", "gated_linear_backward", "rmsnorm_backward"):
        block.kept = {}
        block.dense_backward(small, kept)
        ws = block.kept[op][-1]
        moe.set_debug_flags(ws, 1)
        block.dense_backward(small, kept)
        _, more = block.dense(large, large)
        block.dense_backward(large, more)  # needs a larger workspace: the error stays in the one before
        with pytest.raises(moe.MoEError, match=op):
            block.check()
        block.check()
    grads = block.dense_backward(small, kept)
    block.check()
    assert all(g.isfinite().all() for g in grads)
