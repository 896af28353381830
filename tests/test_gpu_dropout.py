"""Dropout with the residual add and its gradient on the GPU against the float64 oracle.

The mask is compared bit for bit.  A value is x * scale (one fp32 rounding, the scale itself rounded:
2^-23 relative in all) plus the residual (one more, 2^-24 of the sum), then half a bf16 ulp (2^-8)
where the output is bf16."""
import numpy as np
import pytest
import torch

import param_buffers_gb300 as gtp
from oracle import dropout as DO

pytestmark = pytest.mark.gpu
DEV = "cuda"
B, F = torch.bfloat16, torch.float32


def check(got, x, p, rng, residual=None):
    xin = x.double().cpu().numpy()
    res = None if residual is None else residual.double().cpu().numpy()
    ref = DO.dropout(xin, p, rng, res)
    out = got.double().cpu().numpy()
    kept = np.abs(DO.dropout(xin, p, rng))
    tol = 2.0 ** -23 * kept + (0 if res is None else 2.0 ** -24 * (np.abs(ref) + 2.0 ** -22 * kept))
    if got.dtype == B:
        tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
    assert np.all(np.abs(out - ref) <= tol + 2.0 ** -133)
    return ref


@pytest.mark.parametrize("xd,od", [(B, B), (B, F), (F, F), (F, B)])
@pytest.mark.parametrize("R,C", [(1, 1), (1, 8), (3, 7), (5, 33), (64, 2048), (257, 1000), (2, 70001)])
@pytest.mark.parametrize("p", [0.0, 0.1, 0.5])
def test_forward_and_gradient(R, C, xd, od, p):
    g = torch.Generator().manual_seed(R + C)
    x = torch.randn(R, C, generator=g).to(xd).to(DEV)
    res = torch.randn(R, C, generator=g).to(od).to(DEV)
    rng = (0xFEDCBA9876543210, 3 + (1 << 33))
    out = torch.full((R, C), float("nan"), dtype=od, device=DEV)
    gtp.gtp_dropout_add(x, res, out, p, rng)
    check(out, x, p, rng, res)
    gtp.gtp_dropout_add(x, None, out, p, rng)
    check(out, x, p, rng)
    dx = torch.full((R, C), float("nan"), dtype=xd, device=DEV)
    gtp.gtp_dropout_grad(res, dx, p, rng)
    check(dx, res, p, rng)


def test_mask_is_the_generator_s_and_the_same_in_both_directions():
    x = torch.ones(100, 515, device=DEV)
    rng = gtp.Rng(42, 7)
    out, dx = torch.empty_like(x), torch.empty_like(x)
    gtp.gtp_dropout_add(x, None, out, 0.3, rng)
    gtp.gtp_dropout_grad(x, dx, 0.3, rng)
    keep = DO.keep((42, 7), 100, 515, 0.3)
    assert np.array_equal(out.cpu().numpy() != 0, keep) and torch.equal(out, dx)
    # a shard of the rows from an offset of its own draws its own mask; the same offset draws the same
    word = torch.full((1,), 5, dtype=torch.int64, device=DEV)
    gtp.gtp_dropout_add(x, None, out, 0.3, gtp.Rng(42, 2, word))
    assert np.array_equal(out.cpu().numpy() != 0, keep)


def test_dropped_elements_contribute_nothing():
    x = torch.full((40, 64), float("nan"), device=DEV)
    x[::2] = float("inf")
    res = torch.randn(40, 64, device=DEV)
    out = torch.empty_like(res)
    gtp.gtp_dropout_add(x, res, out, 0.5, (1, 1))
    keep = torch.from_numpy(DO.keep((1, 1), 40, 64, 0.5)).to(DEV)
    assert torch.equal(out[~keep], res[~keep])
    assert not torch.isfinite(out[keep]).any()
    gtp.gtp_dropout_add(x, res, out, 1.0, (1, 1))
    assert torch.equal(out, res)
    gtp.gtp_dropout_grad(x, out, 1.0, (1, 1))
    assert not out.any()


@pytest.mark.parametrize("xd,od", [(B, B), (B, F), (F, F), (F, B)])
@pytest.mark.parametrize("pad,shift", [(0, 0), (8, 0), (5, 0), (1, 3), (16, 8)])
def test_strides_alignment_and_in_place(xd, od, pad, shift):
    R, C = 33, 72
    xs = torch.randn(R, C + pad + shift, device=DEV).to(xd)
    rs = torch.randn(R, C + 2 * pad + shift, device=DEV).to(od)
    os = torch.full((R, C + pad + 2 * shift), 7.0, device=DEV).to(od)
    x, res, out = xs[:, shift:shift + C], rs[:, shift:shift + C], os[:, 2 * shift:2 * shift + C]
    gtp.gtp_dropout_add(x, res, out, 0.2, (8, 8))
    check(out, x, 0.2, (8, 8), res)
    assert torch.all(os[:, :2 * shift] == 7) and torch.all(os[:, 2 * shift + C:] == 7)
    onto = res.clone()
    gtp.gtp_dropout_add(x, onto, onto, 0.2, (8, 8))
    assert torch.equal(onto, out)
    if xd == od:
        inplace = x.clone()
        gtp.gtp_dropout_grad(inplace, inplace, 0.2, (8, 8))
        check(inplace, x, 0.2, (8, 8))


def test_gradient_by_differences():
    x, h, g = (torch.randn(50, 96, device=DEV) for _ in range(3))
    f = lambda v: (gtp.gtp_dropout_add(v, x, o := torch.empty_like(v), 0.25, (4, 4)), o.double())[1]
    dx = torch.empty_like(x)
    gtp.gtp_dropout_grad(g, dx, 0.25, (4, 4))
    diff = float((g.double() * (f(x + h) - f(x - h))).sum()) / 2
    want = float((dx.double() * ((x + h).double() - (x - h).double())).sum()) / 2
    assert abs(diff - want) <= 4800 * 2.0 ** -20      # 4800 terms, a few fp32 roundings of order-1 values each


def test_large_rows_and_empty():
    x = torch.randn(20000, 512, device=DEV).to(B)
    out = torch.empty_like(x)
    gtp.gtp_dropout_add(x, x, out, 0.1, (2, 3))
    rows = np.array([0, 1, 8191, 19999])
    keep = DO.PH.draws(2, 3, 20000, 512, 16, 0)[rows] >= DO.threshold(0.1)
    moved = ((out - x)[rows].cpu().float().numpy() != 0) | (x[rows].cpu().float().numpy() == 0)
    # 0.1 of an ulp-sized x could round away: bf16 keeps x + 1.11 x apart from x always
    assert np.array_equal(moved, keep | (x[rows].cpu().float().numpy() == 0))
    gtp.gtp_dropout_add(x[:0], x[:0], out[:0], 0.1, (2, 3))


def test_side_stream_and_captured_offset():
    """On a stream of its own, captured once: each replay draws at the device's offset, both ways."""
    x, r = torch.randn(40, 100, device=DEV), torch.randn(40, 100, device=DEV)
    out, dx = torch.empty_like(x), torch.empty_like(x)
    word = torch.zeros(1, dtype=torch.int64, device=DEV)
    rng = gtp.Rng(6, 1 << 33, word)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    gtp.gtp_dropout_add(x, r, out, 0.3, rng, stream=side)
    gtp.gtp_dropout_grad(x, dx, 0.3, rng, stream=side)
    side.synchronize()
    check(out, x, 0.3, (6, 1 << 33), r)
    check(dx, x, 0.3, (6, 1 << 33))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        gtp.gtp_dropout_add(x, r, out, 0.3, rng)
        gtp.gtp_dropout_grad(x, dx, 0.3, rng)
    for step in (3, 4):
        word.fill_(step)
        graph.replay()
        torch.cuda.synchronize()
        check(out, x, 0.3, (6, (1 << 33) + step), r)
        check(dx, x, 0.3, (6, (1 << 33) + step))
