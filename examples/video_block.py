"""Train one small transformer block on video tokens: the fused query
up-projection with positions on three axes, a rotary key that the heads share,
the gated feed-forward block, and AdamW with MXFP8 moments.

    python examples/video_block.py [--steps 30] [--state-bits 8]

Every product but the attention itself (plain torch operations here) runs in
the library. Positions (frame, row, column) are gathered once into a table per
token, which the fused projection reads like any other; the shared key's
gradient is the inverse rotation of the heads' sum.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import up_proj_gemm_gb300 as mlaq  # noqa: E402
from up_proj_gemm_gb300 import autograd as mlaq_grad  # noqa: E402

bf16 = torch.bfloat16
FRAMES, ROWS, COLS = 4, 8, 8
K, H, DN, DR, DV, F = 128, 4, 32, 32, 32, 512
SECTIONS = (8, 4, 4)  # pairs that follow the frame, the row and the column


def positions(device):
    """int32 [3, T]: frame, row and column of every token."""
    f, r, c = torch.meshgrid(torch.arange(FRAMES), torch.arange(ROWS), torch.arange(COLS), indexing="ij")
    return torch.stack([f.flatten(), r.flatten(), c.flatten()]).to(torch.int32).to(device)


class Block:
    """Parameters and forward pass of the block."""

    def __init__(self, device, seed=0):
        g = torch.Generator().manual_seed(seed)

        def param(*shape):
            w = torch.randn(shape, generator=g) * shape[-1] ** -0.5
            return w.to(bf16).to(device).requires_grad_()

        self.w_q = param(H * (DN + DR), K)
        self.w_k, self.w_v = param(H * DN, K), param(H * DV, K)
        self.w_rope = param(DR, K)
        self.w_out = param(K, H * DV)
        self.w_gate_up, self.w_down = param(2 * F, K), param(K, F)
        freq = 10000.0 ** (-torch.arange(0, DR, 2, dtype=torch.float64) / DR)
        angle = torch.arange(64, dtype=torch.float64)[:, None] * torch.cat([freq, freq])
        self.cos, self.sin = angle.cos().float().to(device), angle.sin().float().to(device)
        self.pos, self.axes = positions(device), mlaq.rope_sections(SECTIONS)
        # the tables of this clip, for the fused projection
        self.clip_cos, self.clip_sin = mlaq.rope_axes_table(self.cos, self.sin, self.pos, self.axes, DR)

    def parameters(self):
        return [self.w_q, self.w_k, self.w_v, self.w_rope, self.w_out, self.w_gate_up, self.w_down]

    def __call__(self, x):
        T = x.shape[0]
        q = mlaq_grad.q_up_proj(x, self.w_q, self.clip_cos, self.clip_sin, H, DN, DR)
        k_rope = mlaq_grad.rope_axes((x @ self.w_rope.t()).view(T, 1, DR), self.cos, self.sin, self.pos, self.axes, DR,
                                     heads=H)
        k = torch.cat([(x @ self.w_k.t()).view(T, H, DN), k_rope], -1)
        v = (x @ self.w_v.t()).view(T, H, DV)
        score = torch.einsum("qhd,khd->hqk", q.float(), k.float()) * (DN + DR) ** -0.5
        mixed = torch.einsum("hqk,khd->qhd", score.softmax(-1), v.float()).to(bf16)
        x = x + mixed.reshape(T, H * DV) @ self.w_out.t()
        return x + mlaq_grad.gated_ffn(x.contiguous(), self.w_gate_up, self.w_down, act="silu")


def train(steps=30, state_bits=8, device="cuda:0", seed=0):
    """The losses of `steps` steps towards a fixed target (one value a step)."""
    block = Block(device, seed)
    g = torch.Generator().manual_seed(seed + 1)
    T = FRAMES * ROWS * COLS
    x = torch.randn((T, K), generator=g).to(bf16).to(device)
    target = torch.randn((T, K), generator=g).to(device)
    opt = mlaq.AdamW(block.parameters(), lr=2e-2, betas=(0.9, 0.95), weight_decay=0.01, state_bits=state_bits,
                     masters=True, seed=seed)
    losses = []
    for _ in range(steps):
        loss = (block(x).float() - target).square().mean()
        loss.backward()
        opt.step()
        for p in block.parameters():
            p.grad = None
        losses.append(loss.detach())
    return torch.stack(losses).tolist()


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=30)
    ap.add_argument("--state-bits", type=int, default=8, choices=(8, 32))
    a = ap.parse_args()
    for i, v in enumerate(train(a.steps, a.state_bits)):
        print(f"step {i:3d}  loss {v:.4f}")


if __name__ == "__main__":
    main()
