"""The 4-bit attention block of examples/: the operators together in a training loop."""
import importlib.util
from pathlib import Path

import pytest
import torch

pytestmark = pytest.mark.gpu
spec = importlib.util.spec_from_file_location(
    "mxfp4_attention_block", Path(__file__).resolve().parents[1] / "examples" / "mxfp4_attention_block.py")
example = importlib.util.module_from_spec(spec)
spec.loader.exec_module(example)

SMALL = dict(hidden=256, groups=2, queries=2, head_dim=32, p=0.05, lr=3e-3)


def test_forward_is_reproducible_and_dropout_repeats_in_the_backward():
    x = torch.randn(131, 256, device="cuda").bfloat16()
    a, b = (example.AttentionBlock(131, seed=5, **SMALL) for _ in range(2))
    assert torch.equal(a.forward(x), b.forward(x))
    a.backward(torch.ones_like(x))
    assert torch.equal(a.out[a.dy == 0], x[a.dy == 0])  # where the gradient was dropped, nothing was added
    assert 0.02 < (a.dy == 0).float().mean().item() < 0.09
    a.step_count += 1
    assert not torch.equal(a.forward(x), b.out)  # the next step draws anew


def test_gradient_against_the_block_in_fp32():
    """The input's and the weights' gradients of the 4-bit block agree with autograd of the same block in fp32 as
    far as 4-bit operands allow: each quantized operand is off by about 10 % of its norm at random, so a chain
    of products keeps the direction (cosine above 0.9)."""
    torch.manual_seed(0)
    T = 256
    b = example.AttentionBlock(T, seed=3, **{**SMALL, "p": 0.0})
    x = torch.randn(T, 256, device="cuda").bfloat16()
    dout = torch.randn(T, 256, device="cuda").bfloat16()
    b.forward(x)
    dx = b.backward(dout)
    ws = {n: w[0].clone().requires_grad_() for n, w in b.weights.items()}
    xf = x.float().requires_grad_()
    qkv = (xf @ ws["qkv"].t()).view(T, 2, 4, 32)
    half = 16
    ang = torch.arange(T, device="cuda", dtype=torch.float64)[:, None] * torch.tensor(
        [t / 2.0 ** 64 * 2 * torch.pi for t in b.turns], dtype=torch.float64, device="cuda")
    c, s = ang.cos().float()[:, None, None], ang.sin().float()[:, None, None]
    u, v = qkv[:, :, :3, :half], qkv[:, :, :3, half:]
    rot = torch.cat((u * c - v * s, u * s + v * c), -1)
    q, k, val = (t.permute(1, 2, 0, 3) for t in (rot[:, :, :2], rot[:, :, 2:3], qkv[:, :, 3:]))
    att = (q @ k.transpose(-1, -2)) * 32 ** -0.5
    att = att.masked_fill(torch.ones(T, T, dtype=torch.bool, device="cuda").triu(1), float("-inf")).softmax(-1) @ val
    out = att.permute(2, 0, 1, 3).reshape(T, -1) @ ws["proj"].t() + xf
    grads = torch.autograd.grad(out, (xf, ws["qkv"], ws["proj"]), dout.float())
    cos = lambda p, r: torch.nn.functional.cosine_similarity(p.flatten().float(), r.flatten(), 0).item()
    view = lambda n: b.grad[b.start[n]:b.start[n] + ws[n].numel()]
    assert cos(b.out, out.detach()) > 0.9
    for got, ref in ((dx, grads[0]), (view("qkv"), grads[1]), (view("proj"), grads[2])):
        assert cos(got, ref) > 0.9


def test_the_loss_falls():
    losses, _ = example.train(steps=60, tokens=128, report=0, seed=1, **SMALL)
    assert sum(losses[-10:]) < 0.9 * sum(losses[:10])
