"""The token embedding and its gradient on the GPU against the float64 oracle.

Lookup: one fp32 product (2^-24), half a bf16 step (2^-8) where the output is bf16.  Gradient of a row with n tokens:
n additions and the scale's product in fp32 (2^-24 each, of the terms' magnitudes), the addition to the buffer (2^-24 of
the result), and 2^-8 of the result where the buffer is bf16."""
import numpy as np
import pytest
import torch

import param_buffers_gb300 as gtp
from oracle import embedding as E

pytestmark = pytest.mark.gpu
DEV = "cuda"
B, F = torch.bfloat16, torch.float32


def f64(t):
    return t.double().cpu().numpy()


def make_ids(T, rows, first, kind="mixed", wide=True, seed=0):
    g = torch.Generator().manual_seed(seed + T + rows)
    if kind == "one row":
        ids = torch.full((T,), first + rows // 2)
    elif kind == "none":
        ids = torch.full((T,), first + rows)
    else:  # half of them in the shard, some nowhere at all, a frequent one
        ids = torch.randint(max(0, first - rows // 2), first + rows + max(1, rows // 2), (T,), generator=g)
        ids[::5] = first
        ids[3::17] = -1
    if not wide:
        return ids.to(torch.int32)
    ids[6::29] = -(1 << 63)  # an int64 that wraps where it is subtracted from
    ids[7::29] = (1 << 63) - 1
    return ids


def check_lookup(out, ids, table, first, scale):
    ref = E.lookup(ids.tolist(), f64(table), first, float(np.float32(scale)))
    tol = 2.0 ** -24 * np.abs(ref)
    if out.dtype == B:
        tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
    assert np.all(np.abs(f64(out) - ref) <= tol)


def check_gradient(got, before, ids, dout, first, rows, scale):
    grad, mass, n = E.gradient(ids.tolist(), f64(dout), rows, first, float(np.float32(scale)))
    ref = f64(before).reshape(rows, -1) + grad
    tol = (n[:, None] + 1) * 2.0 ** -24 * mass * (1 + 2.0 ** -20) + 2.0 ** -24 * (np.abs(ref) + 2.0 ** -10 * mass)
    if got.dtype == B:
        tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
    out = f64(got).reshape(rows, -1)
    assert np.all(np.abs(out - ref) <= np.where(n[:, None] > 0, tol, 0))  # rows without a token keep their bits


@pytest.mark.parametrize("td,od", [(B, B), (B, F), (F, F), (F, B)])
@pytest.mark.parametrize("T,rows,C,first", [(1, 5, 8, 0), (1, 1, 1, 7), (37, 100, 2048, 100), (130, 17, 1535, 3),
                                            (300, 64, 24, 1 << 40), (5, 3, 9001, 2)])
def test_lookup(T, rows, C, first, td, od):
    for wide in (True, False):
        if not wide and first > 1 << 30:
            continue
        ids = make_ids(T, rows, first, wide=wide).to(DEV)
        table = torch.randn(rows, C, device=DEV).to(td)
        out = torch.full((T, C), float("nan"), dtype=od, device=DEV)
        gtp.gtp_embedding(ids, table, out, first_row=first, scale=1.7)
        check_lookup(out, ids, table, first, 1.7)


def test_lookup_strides_empty_and_infinite_scale():
    table = torch.randn(20, 80, device=DEV).to(B)[:, 3:67]
    out = torch.full((9, 100), 5.0, device=DEV)
    ids = torch.arange(-2, 7, device=DEV)
    gtp.gtp_embedding(ids, table, out[:, 1:65], scale=float("inf"))
    assert torch.all(out[:2, 1:65] == 0) and torch.all(torch.isinf(out[2:, 1:65]))
    assert torch.all(out[:, :1] == 5) and torch.all(out[:, 65:] == 5)
    gtp.gtp_embedding(ids[:0], table, out[:0, :64])
    gtp.gtp_embedding(ids, table[:0], out[:, :64])
    assert torch.all(out[:, :64] == 0)  # a shard without rows


@pytest.mark.parametrize("dd,gd", [(B, F), (F, F), (B, B), (F, B)])
@pytest.mark.parametrize("T,rows,C,first,offset", [(1, 5, 8, 0, 0), (1, 1, 1, 7, 3), (64, 10, 16, 0, 64), (65, 33, 40, 5, 1),
                                                   (1111, 401, 1000, 401, 8), (700, 3, 77, 2, 5), (16, 50, 2056, 0, 0), (63, 30, 24, 0, 8),
                                                   (66, 30, 24, 0, 8), (62, 9, 333, 4, 1), (130, 40, 2051, 0, 3)])
def test_gradient(T, rows, C, first, offset, dd, gd):
    for kind in ("mixed", "one row", "none"):
        ids = make_ids(T, rows, first, kind, wide=T % 2 == 1).to(DEV)
        dout = torch.randn(T, C, device=DEV).to(dd)
        grad = torch.randn(offset + rows * C + 11, device=DEV).to(gd)
        before = grad.clone()
        ws = torch.empty(gtp.gtp_embedding_grad_workspace_bytes(T, rows, C), dtype=torch.uint8, device=DEV)
        ws.fill_(0x7F)
        gtp.gtp_embedding_grad_accum(dout, ids, grad, offset, rows, ws, first_row=first, scale=0.7)
        end = offset + rows * C
        check_gradient(grad[offset:end], before[offset:end], ids, dout, first, rows, 0.7)
        assert torch.equal(grad[:offset], before[:offset]) and torch.equal(grad[end:], before[end:])


@pytest.mark.parametrize("T,rows", [(16384, 500), (16385, 500), (40000, 70000), (9000, 500000), (10241, 700), (12200, 20),
                                    (12288, 500), (12289, 500), (2560, 900), (2561, 900),
                                    (32768, 300), (32769, 300), (131072, 300), (131073, 70000), (70000, 17000000)])
def test_gradient_both_ways_of_sorting(T, rows):
    """Around the borders between counting and the radix sort, and keys of one to four digits."""
    C = 8
    g = torch.Generator().manual_seed(T)
    ids = torch.randint(-10, rows + 10, (T,), generator=g)
    ids[T // 3:T // 2] = rows - 1  # a row of thousands of tokens, over many tiles
    ids = ids.to(DEV)
    dout = torch.randn(T, C, device=DEV)
    before = torch.randn(rows * C, device=DEV)
    ws = torch.empty(gtp.gtp_embedding_grad_workspace_bytes(T, rows, C), dtype=torch.uint8, device=DEV)
    grads = []
    for _ in range(2):
        grad = before.clone()
        gtp.gtp_embedding_grad_accum(dout, ids, grad, 0, rows, ws)
        grads.append(grad)
    assert torch.equal(*grads)  # the same bits again
    check_gradient(grads[0], before, ids, dout, 0, rows, 1.0)


def test_gradient_strides_and_difference():
    """A strided dout; and the gradient is the lookup's: <dout, lookup(table)> changes by it along a direction."""
    T, rows, C = 90, 30, 48
    ids = make_ids(T, rows, 30).to(DEV)
    dout = torch.randn(T, C + 5, device=DEV)[:, 2:2 + C]
    ws = torch.empty(gtp.gtp_embedding_grad_workspace_bytes(T, rows, C), dtype=torch.uint8, device=DEV)
    grad = torch.zeros(rows * C, device=DEV)
    gtp.gtp_embedding_grad_accum(dout, ids, grad, 0, rows, ws, first_row=30, scale=3.0)
    check_gradient(grad, torch.zeros_like(grad), ids, dout, 30, rows, 3.0)
    along = torch.randn(rows, C, device=DEV)
    out = torch.empty(T, C, device=DEV)
    gtp.gtp_embedding(ids, along, out, first_row=30, scale=3.0)  # the lookup is linear in the table
    a, b = (out.double() * dout.double()).sum(), (grad.double().view(rows, C) * along.double()).sum()
    mass = (out.double() * dout.double()).abs().sum()
    assert abs(a - b) <= 2.0 ** -20 * mass


def test_captured_on_a_side_stream():
    T, rows, C = 500, 64, 256
    ids = make_ids(T, rows, 0).to(DEV)
    table, dout = torch.randn(rows, C, device=DEV), torch.randn(T, C, device=DEV)
    out, grad = torch.empty(T, C, device=DEV), torch.zeros(rows * C, device=DEV)
    ws = torch.empty(gtp.gtp_embedding_grad_workspace_bytes(T, rows, C), dtype=torch.uint8, device=DEV)
    want_out, want = torch.empty_like(out), torch.zeros_like(grad)
    gtp.gtp_embedding(ids, table, want_out)
    gtp.gtp_embedding_grad_accum(dout, ids, want, 0, rows, ws)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        gtp.gtp_embedding(ids, table, out)
        gtp.gtp_embedding_grad_accum(dout, ids, grad, 0, rows, ws)
    for _ in range(2):
        grad.zero_()
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want_out) and torch.equal(grad, want)
