"""A pre-norm feed-forward block: routed e4m3 experts beside a dense shared expert.

    s      = x + residual                      \\
    y      = norm(s) * weight                   > one launch, y also as e4m3 codes
    yq, sc = e4m3(y)                           /
    routed = sum_k w_k expert_k(yq)            the MoE layer on the norm's own codes
    out    = routed + W2 (silu(W1 y) * W3 y)   the shared expert, its sum in the epilogue

``out`` and ``s`` are the next block's x and residual.  ``Block.train_step``
runs the norm and the shared expert forward and backward and applies plain
gradient descent (the routed experts are inference only).  The block keeps its
workspaces, so that ``Block.check`` can say whether a kernel gave up: a call
without one drops the error word with it.

    python examples/ffn_block.py [--tokens N]
"""
from __future__ import annotations

import argparse
import dataclasses
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from mixture_experts_layer_02_gb300 import moe, synth  # noqa: E402


@dataclasses.dataclass
class Block:
    wl: synth.Workload         # sizes and scoring of the routed experts
    shared: int                # hidden width of the shared expert
    norm: torch.Tensor         # [D]
    w_gate: torch.Tensor       # [E, D]
    experts: dict              # e4m3 codes and scales of the routed experts
    w1: torch.Tensor           # [shared, D]
    w3: torch.Tensor
    w2: torch.Tensor           # [D, shared]
    kept: dict = dataclasses.field(default_factory=dict)  # workspaces of each operation, the largest last

    @classmethod
    def make(cls, wl: synth.Workload, shared: int, seed: int = 0, device="cuda") -> "Block":
        inp = synth.make_inputs(wl, seed=seed, device=device)
        g = torch.Generator(device=device)
        g.manual_seed(seed + 77)

        def normal(rows, cols):
            return (torch.randn((rows, cols), generator=g, device=device) * cols ** -0.5).to(torch.bfloat16)

        return cls(wl, shared, torch.ones(wl.D, dtype=torch.bfloat16, device=device), inp["w_gate"],
                   moe.quantize_experts_e4m3(inp["w1"], inp["w3"], inp["w2"]), normal(shared, wl.D), normal(shared, wl.D),
                   normal(wl.D, shared))

    def ws(self, op: str, N: int, **sizes) -> torch.Tensor:
        """A workspace for ``op``, made anew only where the last one is too small."""
        have = self.kept.setdefault(op, [])
        if not have or have[-1].numel() < moe.workspace_size(op, N=N, **sizes):
            have.append(moe.workspace(op, N=N, **sizes))
        return have[-1]

    def check(self):
        """Wait for the GPU; raise if a kernel of this block recorded an error since the last check."""
        for op, have in self.kept.items():
            for w in have:
                status = moe.read_device_error(w)
                if status != moe.MOE_OK:
                    moe.clear_device_error(w)
                    raise moe.MoEError(op, status, "recorded by a kernel of this block")

    def routed(self, y, yq, scale):
        """The MoE layer on the norm's bf16 rows (router) and codes (experts)."""
        wl, e, N = self.wl, self.experts, y.shape[0]
        ids, w = moe.moe_route(y, self.w_gate, None, wl.K, wl.mode, ws=self.ws("route", N, D=wl.D, E=wl.E, K=wl.K))
        offsets, src, inv, rows = moe.moe_permute_e4m3(yq, ids, wl.E, ws=self.ws("permute", N, E=wl.E))
        y_perm = moe.moe_grouped_ffn_e4m3(rows, scale, src, offsets, e["w1q"], e["s1"], e["w3q"], e["s3"], e["w2q"], e["s2"],
                                          wl.act, ws=self.ws("ffn", N * wl.K, D=wl.D, E=wl.E, K=1, Dff=wl.Dff))[3]
        return moe.moe_combine(y_perm, inv, w, ws=self.ws("combine", 0))

    def dense_ws(self, op: str, y) -> torch.Tensor:
        up = op.startswith("gated")
        D, F = (self.wl.D, self.shared) if up else (self.shared, self.wl.D)
        return self.ws(op, y.shape[0], D=D, Dff=F)

    def forward(self, x, residual):
        """(out, s) of N tokens, one or many."""
        y, yq, scale, s = moe.moe_rmsnorm(x, self.norm, residual=residual, quantize=True)
        h, _, _ = moe.moe_gated_linear(y, self.w1, self.w3, ws=self.dense_ws("gated_linear", y))
        out, _ = moe.moe_linear(h, self.w2, residual=self.routed(y, yq, scale), ws=self.dense_ws("linear", y))
        return out, s

    def dense(self, x, residual):
        """The block without its routed experts, and what its backward pass keeps."""
        y, _, _, s = moe.moe_rmsnorm(x, self.norm, residual=residual)
        h, g, u = moe.moe_gated_linear(y, self.w1, self.w3, save=True, ws=self.dense_ws("gated_linear", y))
        out, _ = moe.moe_linear(h, self.w2, residual=s, ws=self.dense_ws("linear", y))
        return out, (y, s, h, g, u)

    def dense_backward(self, dout, kept):
        """Gradients (dx, dnorm, dw1, dw3, dw2) of the dense block; dx is x's and the residual's."""
        y, s, h, g, u = kept
        dh, dw2, _ = moe.moe_linear_backward(dout, h, self.w2, ws=self.dense_ws("linear_backward", y))
        dy, dw1, dw3 = moe.moe_gated_linear_backward(dh, y, self.w1, self.w3, g, u,
                                                     ws=self.dense_ws("gated_linear_backward", y))
        dx, dnorm = moe.moe_rmsnorm_backward(dy, s, self.norm, dresidual=dout,
                                             ws=self.ws("rmsnorm_backward", y.shape[0], D=self.wl.D))
        return dx, dnorm, dw1, dw3, dw2

    def train_step(self, x, residual, target, lr: float) -> torch.Tensor:
        """One step of gradient descent on mean squared error; returns the loss."""
        out, kept = self.dense(x, residual)
        off = out.float() - target.float()
        _, dnorm, dw1, dw3, dw2 = self.dense_backward((2.0 * off / off.numel()).to(torch.bfloat16), kept)
        for p, d in ((self.norm, dnorm), (self.w1, dw1), (self.w3, dw3), (self.w2, dw2)):
            p.copy_(p.float() - lr * d.float())
        return off.square().mean()


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--tokens", type=int, default=64)
    a = ap.parse_args()
    wl = dataclasses.replace(synth.WORKLOADS["qwen3_N1"], name="block", N=a.tokens, D=512, E=16, Dff=256)
    block = Block.make(wl, shared=1024)
    x, residual = (synth.make_tokens(wl, seed=3, device="cuda", step=i) for i in (0, 1))
    out, s = block.forward(x, residual)
    one, _ = block.forward(x[:1], residual[:1])
    print(f"{a.tokens} tokens: out {tuple(out.shape)}, rms {out.float().square().mean().sqrt():.4f}; "
          f"token 0 alone differs by {(one - out[:1]).abs().max().item():.4f}")
    target = synth.make_tokens(wl, seed=3, device="cuda", step=2)
    for step in range(20):
        loss = block.train_step(x, residual, target, lr=5.0)
        if step % 5 == 0 or step == 19:
            print(f"step {step:2d}  loss {loss.item():.4f}")
    block.check()


if __name__ == "__main__":
    main()
