"""The 4-bit step's operators on arrays of more than 2^31 elements or 2^32 bytes: offsets that pass 32 bits.
Sampled rows and columns, the first and the last among them, at the tolerances of the operators' own tests."""
import numpy as np
import pytest
import torch

import param_buffers_gb300 as gtp
from oracle import dropout as DO
from oracle import floats as F
from oracle import mxfp4 as MX
from oracle import philox as PH
from oracle import rotary as RO
from oracle.sf_layout import tile_scales

pytestmark = pytest.mark.gpu
DEV = "cuda"
B = torch.bfloat16


@pytest.fixture(autouse=True)
def free():
    yield
    torch.cuda.empty_cache()


def bits(t):
    return t.detach().cpu().contiguous().view(torch.int16).numpy().view(np.uint16)


def scale_rows(tiled, rows, blocks):
    """The scale bytes of some rows out of the tiled order."""
    r = torch.tensor(rows, device=DEV)[:, None]
    b = torch.arange(blocks, device=DEV)[None, :]
    words = (blocks + 3) // 4
    return tiled[((r >> 7) * words + (b >> 2)) * 512 + (r & 31) * 16 + ((r >> 5) & 3) * 4 + (b & 3)].cpu().numpy()


@pytest.mark.parametrize("C", [32784, 32783])
def test_quantize_and_values(C):
    R = 65600
    x = torch.empty(R, C, dtype=B, device=DEV).normal_()
    row, col = gtp.gtp_mxfp4_views(R, C, DEV)
    gtp.gtp_mxfp4_quantize(x, row=row, col=col)
    rows, cols = [0, 127, 65535, 65536, R - 1], [0, 32767, C - 1]
    codes, scales = MX.quantize_rowwise(bits(x[rows]), True)
    assert np.array_equal(row[0][rows].cpu().numpy(), codes)
    assert np.array_equal(scale_rows(row[1], rows, -(-C // 32)), scales)
    t, s = MX.quantize_rowwise(bits(x[:, cols].t()), True)
    assert np.array_equal(col[0][cols].cpu().numpy(), t)
    assert np.array_equal(scale_rows(col[1], cols, -(-R // 32)), s)
    gtp.gtp_mxfp4_dequantize(*row, x)
    assert np.array_equal(x[rows].double().cpu().numpy(), MX.dequantize(codes, scales, C))


def test_product_and_accumulate():
    M, N, K = 70000, 30728, 64
    g = np.random.default_rng(4)
    A, W = (MX.quantize_rowwise(g.standard_normal((r, K)).astype(np.float32)) for r in (M, N))
    up = lambda q: (torch.from_numpy(q[0]).to(DEV), torch.from_numpy(tile_scales(q[1])).to(DEV))
    Y = torch.empty(M, N, dtype=B, device=DEV)
    gtp.gtp_linear_fprop_mxfp4(*up(A), *up(W), Y)
    rows = [0, 255, 34953, M - 1]
    a, w = MX.dequantize(*A, K)[rows], MX.dequantize(*W, K)
    ref, mass = a @ w.T, np.abs(a) @ np.abs(w).T
    got = F.bf16_bits_to_f64(bits(Y[rows]))
    assert np.all(np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) * (1 + 2.0 ** -7) + K * 2.0 ** -23 * mass + 2.0 ** -133)
    del Y
    n, k, off = 200, 136, (1 << 31) + 4
    P, Q = (MX.quantize_rowwise(g.standard_normal((r, 96)).astype(np.float32)) for r in (n, k))
    grad = torch.zeros(off + n * k + 4, device=DEV)
    gtp.gtp_linear_wgrad_accum_mxfp4(*up(P), *up(Q), grad, off)
    p, q = MX.dequantize(*P, 96), MX.dequantize(*Q, 96)
    got = grad[off:off + n * k].view(n, k).double().cpu().numpy()
    assert np.all(np.abs(got - p @ q.T) <= (96 * 2.0 ** -23 + 8 * 2.0 ** -24) * (np.abs(p) @ np.abs(q).T))
    assert not grad[:off].any() and not grad[off + n * k:].any()


def test_one_token_over_many_rows():
    N, K = 1100000, 8192
    codes = torch.empty(N, K // 2, dtype=torch.uint8, device=DEV).random_(0, 256)
    scales = torch.empty(gtp.gtp_mxfp4_views(N, K, "meta")[0][1].numel(), dtype=torch.uint8, device=DEV).random_(120, 130)
    x = MX.quantize_rowwise(np.random.default_rng(5).standard_normal((1, K)).astype(np.float32))
    Y = torch.empty(1, N, dtype=B, device=DEV)
    gtp.gtp_linear_fprop_mxfp4(torch.from_numpy(x[0]).to(DEV), torch.from_numpy(tile_scales(x[1])).to(DEV), codes, scales, Y)
    rows = [0, 31, 1048575, 1048576, N - 1]
    a = MX.dequantize(*x, K)
    w = MX.dequantize(codes[rows].cpu().numpy(), scale_rows(scales, rows, K // 32), K)
    ref, mass = a @ w.T, np.abs(a) @ np.abs(w).T
    got = F.bf16_bits_to_f64(bits(Y[:, rows]))
    assert np.all(np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) * (1 + 2.0 ** -7) + K * 2.0 ** -23 * mass + 2.0 ** -133)


def test_rotary():
    T, H, D = 262145, 64, 128
    x = torch.empty(T, H, D, dtype=B, device=DEV).normal_()
    rows = [0, 131072, 262143, T - 1]
    before = x[rows].double().cpu().numpy()
    turns, _ = gtp.gtp_rotary_turns(gtp.RotaryConfig(D))
    gtp.gtp_rotary(x, x, turns)
    ref = RO.rotate(before, rows, list(turns), False)
    size = np.hypot(before[..., :D // 2], before[..., D // 2:])
    tol = 8 * 2.0 ** -23 * np.concatenate([size, size], -1) + 2.0 ** -8 * np.abs(ref) * (1 + 2.0 ** -6) + 2.0 ** -133
    assert np.all(np.abs(x[rows].double().cpu().numpy() - ref) <= tol)


@pytest.mark.parametrize("C", [32776, 32771])
def test_dropout(C):
    R, p, rng = 65601, 0.25, (77, 5)
    x = torch.empty(R, C, dtype=B, device=DEV).normal_()
    out = torch.empty_like(x)
    gtp.gtp_dropout_add(x, None, out, p, rng)
    rows = [0, 65535, 65536, R - 1]
    w = PH.philox(*rng, np.arange(-(-C // 8), dtype=np.uint64)[None, :], np.array(rows, np.uint64)[:, None])
    keep = (w.astype("<u4").view("<u2").reshape(len(rows), -1)[:, :C] >= DO.threshold(p))
    ref = np.where(keep, x[rows].double().cpu().numpy() * (65536 / (65536 - DO.threshold(p))), 0)
    tol = 2.0 ** -23 * np.abs(ref)
    got = out[rows].double().cpu().numpy()
    assert np.all(np.abs(got - ref) <= tol + 2.0 ** -8 * (np.abs(ref) + tol) + 2.0 ** -133)
    assert np.array_equal(got != 0, keep & (x[rows].double().cpu().numpy() != 0))
