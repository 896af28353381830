"""Rotary positions on the GPU against the float64 oracle.

Tolerance per element, from the arithmetic: the angle is kept to 2^-24 of half a turn (an fp32 with a
32-bit integer's top 24 bits), 2^-24 pi; sincospi is good to 1 ulp (2^-23 relative to values up to 1);
two products and a sum round three times more.  With m = scale * hypot(a, b) of the pair:
8 * 2^-23 m, plus half an ulp of bf16 (2^-8 of the value) where that is the type."""
import numpy as np
import pytest
import torch

import param_buffers_gb300 as gtp
from oracle import rotary as RO

pytestmark = pytest.mark.gpu
DEV = "cuda"


def pair_size(x, half, interleaved):
    m = np.abs(x)
    if interleaved:
        h = np.hypot(x[..., 0:2 * half:2], x[..., 1:2 * half:2])
        m[..., 0:2 * half:2] = m[..., 1:2 * half:2] = h
    else:
        h = np.hypot(x[..., :half], x[..., half:2 * half])
        m[..., :half] = m[..., half:2 * half] = h
    return m


def check(got, x, positions, turns, layout, scale=1.0, inverse=False):
    """got, x: torch [T, H, D]."""
    half = len(turns)
    xin = x.double().cpu().numpy()
    ref = RO.rotate(xin, positions, list(turns), layout == "interleaved", scale, inverse)
    out = got.double().cpu().numpy()
    tol = 8 * 2.0 ** -23 * abs(scale) * pair_size(xin.copy(), half, layout == "interleaved")
    if got.dtype == torch.bfloat16:
        tol += 2.0 ** -8 * np.abs(ref) * (1 + 2.0 ** -6)
    assert np.all(np.abs(out - ref) <= tol + 2.0 ** -133)
    assert np.array_equal(out[..., 2 * half:], xin[..., 2 * half:])


DIMS = [(64, 64), (128, 128), (128, 64), (80, 32), (33, 2), (65, 64), (256, 256), (36, 12)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("D,rot", DIMS)
@pytest.mark.parametrize("T", [1, 37])
def test_against_the_oracle(T, D, rot, layout, dtype):
    g = torch.Generator().manual_seed(T + D)
    x = torch.randn(T, 5, D, generator=g).to(dtype).to(DEV)
    turns, _ = gtp.gtp_rotary_turns(gtp.RotaryConfig(rot, 500000.0, "bands", 32.0))
    pos = torch.randint(0, 1 << 20, (T,), generator=g, dtype=torch.int32)
    out = torch.full_like(x, float("nan"))
    gtp.gtp_rotary(x, out, turns, positions=pos.to(DEV), layout=layout)
    check(out, x, pos.tolist(), turns, layout)
    back = torch.empty_like(x)
    gtp.gtp_rotary(x, back, turns, positions=pos.to(DEV).long(), layout=layout, inverse=True, scale=0.5)
    check(back, x, pos.tolist(), turns, layout, 0.5, True)
    same = x.clone()
    gtp.gtp_rotary(same, same, turns, positions=pos.to(DEV), layout=layout)
    assert torch.equal(same, out)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_packed_projection_in_place(dtype):
    """Queries and the key of every group of a packed QKV product turn; values stay."""
    T, G, P, D = 70, 4, 6, 64
    qkv = torch.randn(T, G, P, D, device=DEV).to(dtype)
    before = qkv.clone()
    turns, _ = gtp.gtp_rotary_turns(gtp.RotaryConfig(64))
    heads = qkv[:, :, :P - 1]
    gtp.gtp_rotary(heads, heads, turns, pos0=5, tokens_per_position=2, positions_per_sequence=20)
    pos = [5 + (t // 2) % 20 for t in range(T)]
    assert torch.equal(qkv[:, :, P - 1], before[:, :, P - 1])
    check(qkv[:, :, :P - 1].reshape(T, -1, D), before[:, :, :P - 1].reshape(T, -1, D), pos, turns, "half")


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("shift", [0, 1, 3, 8])
def test_strides_and_alignment(layout, shift):
    T, H, D, rot = 9, 3, 48, 32
    store = torch.randn(T * 400 + 16, device=DEV).to(torch.bfloat16)
    x = store.as_strided((T, H, D), (400 if shift != 3 else 397, 100, 1), shift)
    room = torch.zeros(T * 311 + 16, device=DEV, dtype=torch.bfloat16)
    out = room.as_strided((T, H, D), (311, 101, 1), shift)       # odd strides
    wide = torch.zeros(H, T, D, device=DEV, dtype=torch.bfloat16).transpose(0, 1)   # heads outermost
    turns, _ = gtp.gtp_rotary_turns(gtp.RotaryConfig(rot))
    gtp.gtp_rotary(x, out, turns, layout=layout)
    gtp.gtp_rotary(x, wide, turns, layout=layout)
    check(out, x, range(T), turns, layout)
    assert torch.equal(out, wide)
    mask = torch.ones_like(room, dtype=torch.bool)
    mask.as_strided((T, H, D), (311, 101, 1), shift).fill_(False)
    assert not room[mask].any()                                  # nothing outside the heads


def test_positions_far_out_and_negative():
    pos = torch.tensor([0, -1, 1 << 31, -(1 << 40), (1 << 62) + 12345, 131071], device=DEV)
    x = torch.randn(6, 2, 64, device=DEV)
    out = torch.empty_like(x)
    turns, _ = gtp.gtp_rotary_turns(gtp.RotaryConfig(64))
    gtp.gtp_rotary(x, out, turns, positions=pos)
    check(out, x, pos.tolist(), turns, "half")


def test_gradient_by_differences():
    """<g, rotate(x)> moves by <inverse rotate(g), h>: the map is linear, so any step serves."""
    T, H, D = 11, 4, 32
    x, g, h = (torch.randn(T, H, D, device=DEV) for _ in range(3))
    turns, scale = gtp.gtp_rotary_turns(gtp.RotaryConfig(32, 10000.0, "ramp", 8.0, 1.0, 32.0, 2048))
    f = lambda v: (gtp.gtp_rotary(v, o := torch.empty_like(v), turns, scale=scale, pos0=9), o.double())[1]
    dg = torch.empty_like(g)
    gtp.gtp_rotary(g, dg, turns, scale=scale, pos0=9, inverse=True)
    diff = float((g.double() * (f(x + h) - f(x - h))).sum()) / 2
    want = float((dg.double() * ((x + h).double() - (x - h).double())).sum()) / 2
    # both sides: 1408 terms of order |g||h|, each off by a few fp32 roundings
    assert abs(diff - want) <= 1408 * 16 * 2.0 ** -23 * scale * 4


def test_long_batch_and_empty():
    T, H, D = 20001, 20, 64
    x = torch.randn(T, H, D, device=DEV).to(torch.bfloat16)
    out = torch.empty_like(x)
    turns, _ = gtp.gtp_rotary_turns(gtp.RotaryConfig(64))
    gtp.gtp_rotary(x, out, turns)
    rows = [0, 1, 8191, 8192, 20000]
    check(out[rows], x[rows], rows, turns, "half")
    gtp.gtp_rotary(x[:0], out[:0], turns)


def test_side_stream_and_captured_positions():
    """On a stream of its own, captured once: each replay turns by the positions on the device then."""
    x = torch.randn(9, 3, 64, device=DEV)
    out = torch.empty_like(x)
    pos = torch.arange(9, dtype=torch.int32, device=DEV)
    turns, _ = gtp.gtp_rotary_turns(gtp.RotaryConfig(64))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    gtp.gtp_rotary(x, out, turns, positions=pos, stream=side)
    side.synchronize()
    check(out, x, pos.tolist(), turns, "half")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        gtp.gtp_rotary(x, out, turns, positions=pos)
    for step in (1, 2):
        pos.add_(1000)
        graph.replay()
        torch.cuda.synchronize()
        check(out, x, pos.tolist(), turns, "half")
