#!/usr/bin/env python3
"""Trains one attention block in 4 bits: the operators of a step together, as a training loop calls them.

  x -> QKV product (MXFP4) -> rotary on its packed output -> attention -> projection (MXFP4)
    -> dropout -> + x

and back: the dropout's gradient from the same draws, both linears' gradients quantized with stochastic
rounding in both views, dgrad and wgrad accumulated into the flat fp32 gradient buffer, the rotary gradient in
place on the packed dQKV, then the fused AdamW sweep and the 4-bit weights written again from the masters.
Attention itself is the caller's: here torch's, causal, through autograd.

The shape is the layer workload's at TP = 2 (hidden 2048, 4 groups of 4 queries, a key and a value of 64) with
fewer tokens.  The block learns one sequence by heart (random targets for random inputs); the loss falls.

    python examples/mxfp4_attention_block.py [--steps N] [--tokens T]
"""
from __future__ import annotations

import argparse
import sys
from pathlib import Path

import torch

sys.path.insert(0, str(Path(__file__).resolve().parents[1]))
import param_buffers_gb300 as gtp  # noqa: E402


class AttentionBlock:
    """One block over `tokens` tokens (one sequence) and its flat parameter and gradient buffers."""

    def __init__(self, tokens, hidden=2048, groups=4, queries=4, head_dim=64, p=0.1, lr=1e-3, seed=0, device="cuda"):
        self.T, self.H, self.G, self.Q, self.D, self.p = tokens, hidden, groups, queries, head_dim, p
        self.qkv_rows, self.proj_cols = groups * (queries + 2) * head_dim, groups * queries * head_dim
        self.seed, self.step_count, self.dev = seed, 0, device
        shapes = {"qkv": (self.qkv_rows, hidden), "proj": (hidden, self.proj_cols)}
        self.layout = gtp.gtp_buffer_layout([gtp.ParamDesc(r * c) for r, c in shapes.values()],
                                            gtp.LayoutConfig(40_000_000, 2, True))
        numel = self.layout.buffers[0]["numel"]
        zeros = lambda dt=torch.float32: torch.zeros(numel, dtype=dt, device=device)
        self.grad, self.master, self.m, self.v = zeros(), zeros(), zeros(), zeros()
        self.param = zeros(torch.bfloat16)
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        self.weights, self.start = {}, {}
        for (name, (r, c)), at in zip(shapes.items(), self.layout.index):
            w = self.master[at["start"]:at["end"]].view(r, c)
            w.copy_(torch.randn(r, c, generator=g, device=device) * c ** -0.5)
            self.start[name] = at["start"]
            self.weights[name] = (w, *gtp.gtp_mxfp4_views(r, c, device))  # master, rowwise, columnwise view
        self.hp = gtp.AdamHparams(lr=lr, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.0)
        self.turns, self.scale = gtp.gtp_rotary_turns(
            gtp.RotaryConfig(head_dim, base=500000.0, scaling="bands", factor=32.0))
        bf16 = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device=device)
        self.qkv, self.dqkv = (bf16(tokens, groups, queries + 2, head_dim) for _ in range(2))
        self.y, self.out, self.dy, self.dx = (bf16(tokens, hidden) for _ in range(4))
        self.da = bf16(tokens, self.proj_cols)
        self.views = {k: gtp.gtp_mxfp4_views(tokens, n, device)
                      for k, n in (("x", hidden), ("a", self.proj_cols), ("dy", hidden), ("dqkv", self.qkv_rows))}
        self.quantize_weights()

    def quantize_weights(self):
        for w, row, col in self.weights.values():
            gtp.gtp_mxfp4_quantize(w, row=row, col=col)

    def rng(self, use):
        """One offset a use and step: the forward and the backward of a use agree, no two uses do."""
        return gtp.Rng(self.seed, 4 * self.step_count + use)

    def rotate(self, qkv, inverse):
        heads = qkv[:, :, :self.Q + 1]  # the queries and the key of every group
        gtp.gtp_rotary(heads, heads, self.turns, scale=self.scale, inverse=inverse)

    def forward(self, x):
        T, G, Q, D = self.T, self.G, self.Q, self.D
        row, col = self.views["x"]
        gtp.gtp_mxfp4_quantize(x, row=row, col=col)
        gtp.gtp_linear_fprop_mxfp4(*row, *self.weights["qkv"][1], self.qkv.view(T, -1))
        self.rotate(self.qkv, inverse=False)
        # attention, the caller's part: [groups, queries, tokens, head_dim], keys and values shared by a group
        q, k, v = (t.permute(1, 2, 0, 3).detach().requires_grad_()
                   for t in (self.qkv[:, :, :Q], self.qkv[:, :, Q:Q + 1], self.qkv[:, :, Q + 1:]))
        with torch.enable_grad():
            a = torch.nn.functional.scaled_dot_product_attention(q, k.expand_as(q), v.expand_as(q), is_causal=True)
            a = a.permute(2, 0, 1, 3).reshape(T, -1)
        self.tape = (a, (q, k, v))
        row, col = self.views["a"]
        gtp.gtp_mxfp4_quantize(a.detach(), row=row, col=col)
        gtp.gtp_linear_fprop_mxfp4(*row, *self.weights["proj"][1], self.y)
        gtp.gtp_dropout_add(self.y, x, self.out, self.p, self.rng(0))
        return self.out

    def backward(self, dout):
        """Accumulates both weight gradients and returns the input's."""
        T, Q = self.T, self.Q
        gtp.gtp_dropout_grad(dout, self.dy, self.p, self.rng(0))
        row, col = self.views["dy"]
        gtp.gtp_mxfp4_quantize(self.dy, row=row, col=col, rng=self.rng(1))
        gtp.gtp_linear_dgrad_mxfp4(*row, *self.weights["proj"][2], self.da)
        gtp.gtp_linear_wgrad_accum_mxfp4(*col, *self.views["a"][1], self.grad, self.start["proj"])
        a, inputs = self.tape
        dq, dk, dv = torch.autograd.grad(a, inputs, self.da)
        for part, d in ((slice(0, Q), dq), (slice(Q, Q + 1), dk), (slice(Q + 1, Q + 2), dv)):
            self.dqkv[:, :, part].copy_(d.permute(2, 0, 1, 3))
        self.rotate(self.dqkv, inverse=True)
        row, col = self.views["dqkv"]
        gtp.gtp_mxfp4_quantize(self.dqkv.view(T, -1), row=row, col=col, rng=self.rng(2))
        gtp.gtp_linear_dgrad_mxfp4(*row, *self.weights["qkv"][2], self.dx)
        gtp.gtp_linear_wgrad_accum_mxfp4(*col, *self.views["x"][1], self.grad, self.start["qkv"])
        return self.dx.add_(dout)

    def update(self):
        """The fused sweep (AdamW, cast, zeroed gradients), then the 4-bit weights from the masters."""
        self.step_count += 1
        gtp.gtp_adam_step_flat(self.grad, self.master, self.m, self.v, self.param, self.layout.c_buckets,
                               [1.0] * len(self.layout.buckets), self.hp, step=self.step_count)
        self.quantize_weights()


def train(steps=60, tokens=512, report=10, **block):
    """Trains the block and returns the losses; an output equal to the input has a loss of 1."""
    b = AttentionBlock(tokens, **block)
    g = torch.Generator(device=b.dev)
    g.manual_seed(b.seed + 1)
    x = torch.randn(tokens, b.H, generator=g, device=b.dev).bfloat16()
    target = x.float() + torch.randn(tokens, b.H, generator=g, device=b.dev)
    losses = []
    for step in range(steps):
        diff = b.forward(x).float() - target
        loss = diff.square().mean()
        b.backward((diff * (2.0 / diff.shape[0])).bfloat16())
        b.update()
        losses.append(loss)
        if report and (step + 1) % report == 0:
            print(f"step {step + 1}: loss {loss.item():.4f}")
    return [v.item() for v in losses], b


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--tokens", type=int, default=512)
    args = ap.parse_args()
    train(args.steps, args.tokens)
