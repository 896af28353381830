"""MXFP4 products over more output tiles than the GPU has CTA pairs, each tile several passes of the operand ring: whole
waves of full-width tiles, the accumulator handed from one tile to the next through the staging buffers, and the
half-width tiles of a last partial wave.  Every element, against float64; bounds as in test_gpu_mxfp4.py."""
import numpy as np
import pytest
import torch

import param_buffers_gb300 as gtp
from oracle import floats as F
from oracle import mxfp4 as MX
from oracle.sf_layout import tile_scales

pytestmark = pytest.mark.gpu
DEV = "cuda"
TILE, STAGE = 256, 256        # a CTA pair's output tile; contraction elements of a stage of the ring


def operand(R, K, seed):
    """A view of random values with its float64 values."""
    rng = np.random.default_rng(seed)
    x = (rng.standard_normal((R, K)) * np.exp2(rng.integers(-4, 4, size=(R, 1)))).astype(np.float32)
    p, s = MX.quantize_rowwise(x)
    return (torch.from_numpy(p).to(DEV), torch.from_numpy(tile_scales(s)).to(DEV)), MX.dequantize(p, s, K)


def waves(rows, cols):
    """(whole waves, tiles of the last partial one) of an output on this GPU."""
    pairs = torch.cuda.get_device_properties(0).multi_processor_count // 2
    return divmod(-(-rows // TILE) * -(-cols // TILE), pairs)


# 100 tiles, 24 of them in half-width tiles behind one wave; 196, two waves and 44 whole tiles
@pytest.mark.parametrize("M,N,K", [(2400, 2392, 2100), (3500, 3480, 1700)])
@pytest.mark.parametrize("call", ["fprop", "dgrad"])
def test_stores_of_several_waves(M, N, K, call):
    assert waves(M, N)[0] >= 1 and waves(M, N)[1] and -(-K // STAGE) > 6
    (Aq, A), (Bq, B) = operand(M, K, 1), operand(N, K, 2)
    D = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device=DEV)
    getattr(gtp, f"gtp_linear_{call}_mxfp4")(*Aq, *Bq, D)
    ref, mass = A @ B.T, np.abs(A) @ np.abs(B).T
    got = F.bf16_bits_to_f64(D.cpu().view(torch.int16).numpy().view(np.uint16))
    assert np.all(np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) * (1 + 2.0 ** -7) + K * 2.0 ** -23 * mass + 2.0 ** -133)


# 90 tiles of five stages, 14 of them in half-width tiles; 156 of nine, two waves and four such tiles; 50 split in
# three over the contraction, so that a pair's units are parts of different tiles
@pytest.mark.parametrize("M,N,K", [(1100, 2560, 2056), (2100, 3200, 2900), (3500, 2500, 1200)])
def test_accumulates_of_several_units_a_pair(M, N, K):
    full, last = waves(N, K)
    assert full >= 1 and last or -(-M // STAGE) > 12
    (dYq, dY), (Xq, X) = operand(N, M, 3), operand(K, M, 4)
    off, guard = 64, 96
    g0 = np.random.default_rng(5).standard_normal(off + N * K + guard).astype(np.float32)
    grad = torch.from_numpy(g0).to(DEV)
    gtp.gtp_linear_wgrad_accum_mxfp4(*dYq, *Xq, grad, off)
    gtp.gtp_linear_wgrad_accum_mxfp4(*dYq, *Xq, grad, off)
    got = grad.cpu().numpy()
    assert np.array_equal(got[:off], g0[:off]) and np.array_equal(got[off + N * K:], g0[off + N * K:])
    old = g0[off:off + N * K].reshape(N, K).astype(np.float64)
    prod, mass = dY @ X.T, np.abs(dY) @ np.abs(X).T
    bound = 2 * M * 2.0 ** -23 * mass + 2 * 8 * 2.0 ** -24 * (np.abs(old) + 2 * mass)
    assert np.all(np.abs(got[off:off + N * K].reshape(N, K) - (old + 2 * prod)) <= bound)
