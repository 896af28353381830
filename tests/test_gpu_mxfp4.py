"""MXFP4 on the GPU against the oracle: both views bit for bit under both roundings, the values, and
the three products.

Tolerances.  Codes, scale bytes (padding included) and values: equal.  A product's terms are exact in
fp32 (E2M1 products have 4 bits, the scales are powers of two), so a bf16 output is off the float64
product by one rounding (2^-8 relative) and the fp32 accumulation, at most 2^-23 of the terms'
absolute sum a term; the accumulate by the same without the bf16 rounding, plus one fp32 rounding
of the sum for each of at most 8 splits (2^-24 of |main_grad| + the absolute sum)."""
import numpy as np
import pytest
import torch

import param_buffers_gb300 as gtp
from oracle import floats as F
from oracle import mxfp4 as MX
from oracle.sf_layout import tile_scales

pytestmark = pytest.mark.gpu
DEV = "cuda"


def buffers(rows, cols):
    """Views prefilled with a pattern, so that an unwritten byte shows."""
    views = gtp.gtp_mxfp4_views(rows, cols, DEV)
    for v in views:
        for t in v:
            t.fill_(0xAB)
    return views


def bits(t):
    return t.detach().cpu().contiguous().view(torch.int16).numpy().view(np.uint16)


def source(R, C, seed, dtype):
    rng = np.random.default_rng(seed)
    x = (rng.standard_normal((R, C)) * np.exp2(rng.integers(-14, 10, size=(R, 1)))).astype(np.float32)
    flat = x.reshape(-1)
    special = [0.0, -0.0, np.nan, np.inf, -np.inf, 1e-40, -1e-45, 3e38, -3.4e38, 6.0, 0.25, 0.75, 1.25, 2.5, 5.0]
    for i, v in enumerate(special):
        if flat.size > 40 * i + 7:
            flat[40 * i + 7] = v
    t = torch.from_numpy(x)
    return t.to(torch.bfloat16) if dtype == "bf16" else t


def oracle_in(x):
    return (bits(x), True) if x.dtype == torch.bfloat16 else (x.cpu().numpy(), False)


def check_view(got, want):
    codes, scales = want
    assert np.array_equal(got[1].cpu().numpy(), tile_scales(scales))
    assert np.array_equal(got[0].cpu().numpy(), codes)


SIZES = [(1, 1), (1, 32), (32, 1), (3, 31), (5, 33), (127, 65), (128, 128), (129, 160), (257, 2048), (1000, 296)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rng", [None, (0x123456789ABCDEF0, 77 + (5 << 32))], ids=["nearest", "stochastic"])
@pytest.mark.parametrize("R,C", SIZES)
def test_both_views_bit_exact(R, C, rng, dtype):
    x = source(R, C, R * 1000 + C, dtype)
    a, bf = oracle_in(x)
    row, col = buffers(R, C)
    gtp.gtp_mxfp4_quantize(x.to(DEV), row=row, col=col, rng=rng)
    check_view(row, MX.quantize_rowwise(a, bf, rng))
    check_view(col, MX.quantize_columnwise(a, bf, rng))
    # one view at a time writes the same bytes
    row1, col1 = buffers(R, C)
    gtp.gtp_mxfp4_quantize(x.to(DEV), row=row1, rng=rng)
    gtp.gtp_mxfp4_quantize(x.to(DEV), col=col1, rng=rng)
    for u, v in zip(row + col, row1 + col1):
        assert torch.equal(u, v)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pad,shift", [(0, 1), (3, 0), (24, 0), (7, 5)])
def test_strided_and_unaligned_sources(dtype, pad, shift):
    R, C = 130, 200
    x = source(R, C, 3, dtype)
    big = torch.full((R, C + pad + shift), 7.0, dtype=x.dtype, device=DEV)
    view = big[:, shift:shift + C]
    view.copy_(x)
    a, bf = oracle_in(x)
    row, col = buffers(R, C)
    gtp.gtp_mxfp4_quantize(view, row=row, col=col, rng=(1, 2))
    check_view(row, MX.quantize_rowwise(a, bf, (1, 2)))
    check_view(col, MX.quantize_columnwise(a, bf, (1, 2)))


def test_ties_saturation_and_both_scale_rules():
    x = np.zeros((2, 64), np.float32)
    x[0, :12] = [4.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.9, -7.9, -0.25, -5.0]   # nearest: scale 1
    x[1, :4] = [6.0, 6.0000005, 3.0, 1.0]                                               # stochastic: scale 2, not 1
    for rng in (None, (9, 9)):
        row, col = buffers(2, 64)
        gtp.gtp_mxfp4_quantize(torch.from_numpy(x).to(DEV), row=row, col=col, rng=rng)
        check_view(row, MX.quantize_rowwise(x, rng=rng))
        check_view(col, MX.quantize_columnwise(x, rng=rng))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rng", [None, (31, 5)], ids=["nearest", "stochastic"])
def test_blocks_of_every_exponent(rng, dtype):
    """One row, and one block of a column, for each power of two that a block's amax can have."""
    exps = np.arange(-149, 128)
    g = np.random.default_rng(12)
    m = (g.uniform(-1, 1, size=(exps.size, 64)) * np.exp2(-g.integers(0, 30, size=(exps.size, 64)))).astype(np.float32)
    m[:, ::32] = 1.75
    rows = torch.from_numpy(np.ldexp(m, exps[:, None]).astype(np.float32))
    cols = torch.from_numpy(np.ldexp(m.T[:32], exps[None]).astype(np.float32)).contiguous()
    for x in (rows, cols):
        x = x.to(torch.bfloat16) if dtype == "bf16" else x
        a, bf = oracle_in(x)
        row, col = buffers(*x.shape)
        gtp.gtp_mxfp4_quantize(x.to(DEV), row=row, col=col, rng=rng)
        check_view(row, MX.quantize_rowwise(a, bf, rng))
        check_view(col, MX.quantize_columnwise(a, bf, rng))


def test_stochastic_mean_and_device_offset():
    """The mean over many offsets approaches the source; an offset on the device adds to the host's."""
    x = source(64, 96, 8, "f32").nan_to_num(0, 0, 0)
    x[x.abs() > 1e30] = 0
    d = x.to(DEV)
    total = torch.zeros(64, 96, dtype=torch.float64, device=DEV)
    row, col = buffers(64, 96)
    out = torch.empty(64, 96, device=DEV)
    word = torch.zeros(1, dtype=torch.int64, device=DEV)
    n = 2000
    for k in range(n):
        word.fill_(k)
        gtp.gtp_mxfp4_quantize(d, row=row, rng=gtp.Rng(5, 1000, word))
        gtp.gtp_mxfp4_dequantize(*row, out)
        total += out.double()
    e = MX.scale_exponent(x.numpy().reshape(64, 3, 32).__abs__().max(-1).astype(np.float64), True)
    step = np.repeat(np.exp2(e), 32, axis=1)           # half a step of the widest spacing, 2
    # a draw's deviation is at most half a step: six sigma of the mean, plus the 1/512-step grain
    err = np.abs(total.cpu().numpy() / n - x.numpy())
    assert np.all(err <= 2 * step * (6 * 0.5 / np.sqrt(n) + 1 / 512))
    gtp.gtp_mxfp4_quantize(d, row=row, rng=(5, 1000 + n - 1))
    last = torch.empty_like(out)
    gtp.gtp_mxfp4_dequantize(*row, last)
    assert torch.equal(last, out)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("R,C", [(1, 1), (3, 33), (129, 160), (300, 2048)])
def test_values(R, C, dtype):
    rng = np.random.default_rng(R + C)
    B = -(-C // 32)
    codes = rng.integers(0, 256, (R, 16 * B)).astype(np.uint8)
    scales = rng.integers(0, 253, (R, B)).astype(np.uint8)
    scales.reshape(-1)[::5] = 0xFF
    scales.reshape(-1)[1::7] = 0
    out = torch.full((R, C), 3.0, dtype=dtype, device=DEV)
    gtp.gtp_mxfp4_dequantize(torch.from_numpy(codes).to(DEV), torch.from_numpy(tile_scales(scales)).to(DEV), out)
    want = MX.dequantize(codes, scales, C)
    got = out.double().cpu().numpy()
    assert np.array_equal(got, want, equal_nan=True)


# --------------------------------------------------------------------------- products

def operand(R, K, seed, device=DEV):
    """A random view: packed codes and scale bytes (padding blocks' codes zero), with its values."""
    rng = np.random.default_rng(seed)
    x = (rng.standard_normal((R, K)) * np.exp2(rng.integers(-4, 4, size=(R, 1)))).astype(np.float32)
    p, s = MX.quantize_rowwise(x)
    return (torch.from_numpy(p).to(device), torch.from_numpy(tile_scales(s)).to(device)), MX.dequantize(p, s, K)


def check_bf16(Y, A, B):
    ref, mass = A @ B.T, np.abs(A) @ np.abs(B).T
    got = F.bf16_bits_to_f64(bits(Y))
    assert np.all(np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) * (1 + 2.0 ** -7) + A.shape[1] * 2.0 ** -23 * mass + 2.0 ** -133)


@pytest.mark.parametrize("M,N,K", [(1, 8, 1), (1, 8, 32), (3, 24, 33), (128, 256, 256), (129, 264, 288), (200, 8, 1000),
                                   (257, 512, 2048), (1, 1536, 2048), (700, 1000, 520)])
def test_forward_and_dgrad(M, N, K):
    (Xq, X), (Wq, W) = operand(M, K, 1), operand(N, K, 2)
    Y = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device=DEV)
    gtp.gtp_linear_fprop_mxfp4(*Xq, *Wq, Y)
    check_bf16(Y, X, W)
    if K % 8 == 0:
        (dYq, dY), (Wtq, Wt) = operand(M, N, 3), operand(K, N, 4)
        dX = torch.full((M, K), float("nan"), dtype=torch.bfloat16, device=DEV)
        gtp.gtp_linear_dgrad_mxfp4(*dYq, *Wtq, dX)
        check_bf16(dX, dY, Wt)


@pytest.mark.parametrize("M", [1, 2, 3, 4, 5, 7, 8, 9])
@pytest.mark.parametrize("N,K", [(8, 8), (40, 40), (136, 104), (264, 1064), (1288, 4200), (128, 9000)])
def test_few_rows(M, N, K):
    """Single tokens and a few, around the size at which they take their own kernel: lengths that end inside a
    block, an atom of scales and a warp's step, rows that end inside a tile of 128."""
    (Xq, X), (Wq, W) = operand(M, K, 11), operand(N, K, 12)
    Y = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device=DEV)
    gtp.gtp_linear_fprop_mxfp4(*Xq, *Wq, Y)
    check_bf16(Y, X, W)
    (dYq, dY), (Wtq, Wt) = operand(M, N, 13), operand(K, N, 14)
    dX = torch.full((M, K), float("nan"), dtype=torch.bfloat16, device=DEV)
    gtp.gtp_linear_dgrad_mxfp4(*dYq, *Wtq, dX)
    check_bf16(dX, dY, Wt)


def test_few_rows_extreme_scales_and_nan():
    """Exponents of the two blocks that meet inside the range although one alone is at its end; NaN scales."""
    M, N, K = 2, 16, 64
    g = np.random.default_rng(15)
    xc, wc = (g.integers(0, 256, (r, K // 2)).astype(np.uint8) for r in (M, N))
    xs, ws = np.full((M, 2), 254, np.uint8), np.full((N, 2), 3, np.uint8)
    xs[1] = 0
    ws[1::2] = 252
    A, W = MX.dequantize(xc, xs, K), MX.dequantize(wc, ws, K)
    dev = lambda c, s: (torch.from_numpy(c).to(DEV), torch.from_numpy(tile_scales(s)).to(DEV))
    Y = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
    gtp.gtp_linear_fprop_mxfp4(*dev(xc, xs), *dev(wc, ws), Y)
    keep = np.array([[n % 2 == (0 if m == 0 else 1) for n in range(N)] for m in range(M)])  # the others pass 2^127 or vanish
    got, ref, mass = F.bf16_bits_to_f64(bits(Y)), A @ W.T, np.abs(A) @ np.abs(W).T
    bound = 2.0 ** -8 * np.abs(ref) * (1 + 2.0 ** -7) + K * 2.0 ** -23 * mass + 2.0 ** -133
    assert np.all(np.abs(got - ref)[keep] <= bound[keep])
    assert not np.isnan(got[keep]).any()  # the others may hold Inf - Inf of two blocks
    ws[3, 1] = 0xFF
    gtp.gtp_linear_fprop_mxfp4(*dev(xc, xs), *dev(wc, ws), Y)
    assert torch.isnan(Y[:, 3]).all() and torch.isnan(Y).cpu().numpy()[keep].sum() == 1


@pytest.mark.parametrize("M,N,K,off", [(1, 4, 4, 0), (32, 128, 64, 64), (33, 129, 68, 4), (1111, 160, 96, 128),
                                       (8192, 256, 256, 64), (4100, 1536, 264, 0)])
def test_wgrad_accumulates_into_the_view(M, N, K, off):
    (dYq, dY), (Xq, X) = operand(N, M, 5), operand(K, M, 6)
    rng = np.random.default_rng(7)
    g0 = rng.standard_normal(off + N * K + 77).astype(np.float32)
    grad = torch.from_numpy(g0).to(DEV)
    gtp.gtp_linear_wgrad_accum_mxfp4(*dYq, *Xq, grad, off)
    gtp.gtp_linear_wgrad_accum_mxfp4(*dYq, *Xq, grad, off)
    got = grad.cpu().numpy()
    assert np.array_equal(got[:off], g0[:off]) and np.array_equal(got[off + N * K:], g0[off + N * K:])
    prod, mass = dY @ X.T, np.abs(dY) @ np.abs(X).T
    ref = g0[off:off + N * K].reshape(N, K).astype(np.float64) + 2 * prod
    bound = 2 * M * 2.0 ** -23 * mass + 2 * 8 * 2.0 ** -24 * (np.abs(g0[off:off + N * K].reshape(N, K)) + 2 * mass)
    assert np.all(np.abs(got[off:off + N * K].reshape(N, K) - ref) <= bound)


def test_nan_blocks_stay_in_their_rows():
    """A NaN block makes NaN of its own row's outputs only, although the next row tile's scales follow
    the contraction's last atom in memory (129 rows, 288 = one stage and one block)."""
    x = np.random.default_rng(0).standard_normal((300, 288)).astype(np.float32)
    x[128, 3] = np.nan            # first row of the second tile, its first block
    x[299, 287] = np.inf          # the last row's last block
    p, s = MX.quantize_rowwise(x)
    Xq = (torch.from_numpy(p).to(DEV), torch.from_numpy(tile_scales(s)).to(DEV))
    Wq, W = operand(264, 288, 1)
    Y = torch.empty(300, 264, dtype=torch.bfloat16, device=DEV)
    gtp.gtp_linear_fprop_mxfp4(*Xq, *Wq, Y)
    bad = torch.isnan(Y).cpu().numpy()
    assert bad[128].all() and bad[299].all() and bad.sum() == 2 * 264
    Yt = torch.empty(264, 300 - 4, dtype=torch.bfloat16, device=DEV)   # the same rows as the second operand
    gtp.gtp_linear_fprop_mxfp4(*Wq, Xq[0][4:].contiguous(), torch.from_numpy(tile_scales(s[4:])).to(DEV), Yt)
    bad = torch.isnan(Yt).cpu().numpy()
    assert bad[:, 124].all() and bad[:, 295].all() and bad.sum() == 2 * 264


def test_empty_sizes():
    Y = torch.full((5, 16), 3.0, dtype=torch.bfloat16, device=DEV)
    e = lambda r: (torch.empty(r, 0, dtype=torch.uint8, device=DEV), torch.empty(0, dtype=torch.uint8, device=DEV))
    gtp.gtp_linear_fprop_mxfp4(*e(5), *e(16), Y)
    assert not Y.any()
    grad = torch.ones(64, device=DEV)
    gtp.gtp_linear_wgrad_accum_mxfp4(*e(8), *e(8), grad, 0)
    assert torch.all(grad == 1)
    row, col = gtp.gtp_mxfp4_views(0, 40, DEV)
    gtp.gtp_mxfp4_quantize(torch.empty(0, 40, device=DEV), row=row, col=col)
    gtp.gtp_mxfp4_dequantize(*row, torch.empty(0, 40, device=DEV))


def test_a_linear_through_quantize_and_products():
    """Quantize, forward, stochastic backward: each product equals the oracle's of the oracle's own views."""
    M, N, K = 333, 160, 96
    g = np.random.default_rng(3)
    X, Wt, dY = (torch.from_numpy(g.standard_normal(s).astype(np.float32)).to(torch.bfloat16)
                 for s in ((M, K), (N, K), (M, N)))
    xr, xc = buffers(M, K)
    wr, wc = buffers(N, K)
    yr, yc = buffers(M, N)
    rng = (21, 4)
    gtp.gtp_mxfp4_quantize(X.to(DEV), row=xr, col=xc)
    gtp.gtp_mxfp4_quantize(Wt.to(DEV), row=wr, col=wc)
    gtp.gtp_mxfp4_quantize(dY.to(DEV), row=yr, col=yc, rng=rng)
    Y, dX = torch.empty(M, N, dtype=torch.bfloat16, device=DEV), torch.empty(M, K, dtype=torch.bfloat16, device=DEV)
    grad = torch.zeros(N * K, device=DEV)
    gtp.gtp_linear_fprop_mxfp4(*xr, *wr, Y)
    gtp.gtp_linear_dgrad_mxfp4(*yr, *wc, dX)
    gtp.gtp_linear_wgrad_accum_mxfp4(*yc, *xc, grad, 0)
    val = lambda q, n: MX.dequantize(*q, n)
    check_bf16(Y, val(MX.quantize_rowwise(bits(X), True), K), val(MX.quantize_rowwise(bits(Wt), True), K))
    check_bf16(dX, val(MX.quantize_rowwise(bits(dY), True, rng), N), val(MX.quantize_columnwise(bits(Wt), True), N))
    A, B = val(MX.quantize_columnwise(bits(dY), True, rng), M), val(MX.quantize_columnwise(bits(X), True), M)
    got = grad.cpu().numpy().reshape(N, K)
    assert np.all(np.abs(got - A @ B.T) <= (M * 2.0 ** -23 + 8 * 2.0 ** -24) * (np.abs(A) @ np.abs(B).T))


def test_graph_capture_and_side_stream():
    """Captured once and replayed with the step count on the device: every replay draws anew."""
    x = torch.randn(256, 192, device=DEV)
    row, col = buffers(256, 192)
    word = torch.zeros(1, dtype=torch.int64, device=DEV)
    gtp.gtp_mxfp4_quantize(x, row=row, col=col, rng=gtp.Rng(3, 0, word))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        gtp.gtp_mxfp4_quantize(x, row=row, col=col, rng=gtp.Rng(3, 0, word))
    for step in (1, 2):
        word.fill_(step)
        graph.replay()
        torch.cuda.synchronize()
        check_view(row, MX.quantize_rowwise(x.cpu().numpy(), rng=(3, step)))
        check_view(col, MX.quantize_columnwise(x.cpu().numpy(), rng=(3, step)))
