"""Refusals of the embedding, the norm and the orthogonalised update (host only: every call below fails its checks, or has
nothing to do, before any CUDA call, so the addresses are never used)."""
import ctypes as C

import pytest

from param_buffers_gb300 import abi

pytestmark = pytest.mark.skipif(not abi.LIB_PATH.exists(), reason="libgtp.so not built")
F32, BF16, U8 = abi.GTP_F32, abi.GTP_BF16, abi.GTP_U8
OK, ARG, SHAPE, ALIGN, DTYPE, RANGE, CAPACITY = (abi.GTP_OK, abi.GTP_E_ARG, abi.GTP_E_SHAPE, abi.GTP_E_ALIGN,
                                                 abi.GTP_E_DTYPE, abi.GTP_E_RANGE, abi.GTP_E_CAPACITY)


def at(k):
    """Addresses far apart."""
    return 0x1000000000 * (k + 1)


def test_struct_sizes():
    assert C.sizeof(abi.gtp_embedding_desc) == 96 == len(abi.EMBEDDING_DESC_PACK(*[0] * 9, 0.0, *[0] * 4))
    assert C.sizeof(abi.gtp_embedding_grad_desc) == 104 == len(abi.EMBEDDING_GRAD_DESC_PACK(*[0] * 10, 0.0, *[0] * 4))
    assert C.sizeof(abi.gtp_rmsnorm_desc) == 160 == len(abi.RMSNORM_DESC_PACK(*[0] * 16, 0.0, *[0] * 6))
    assert C.sizeof(abi.gtp_rmsnorm_grad_desc) == 144 == len(abi.RMSNORM_GRAD_DESC_PACK(*[0] * 20))
    assert C.sizeof(abi.gtp_muon_hparams) == 56 == len(abi.MUON_HPARAMS_PACK(*[0] * 13))


def lookup(**change):
    d = dict(ids=at(0), table=at(1), out=at(2), tokens=10, first_row=0, rows=100, cols=64, table_ld=64, out_ld=64, scale=1.0,
             ids64=1, table_dtype=BF16, out_dtype=BF16, reserved=0)
    assert set(change) <= set(d)
    return abi.load().gtp_embedding(C.byref(abi.gtp_embedding_desc(**{**d, **change})), None)


@pytest.mark.parametrize("change,status", [
    (dict(reserved=1), ARG), (dict(table_dtype=U8), DTYPE), (dict(out_dtype=abi.GTP_F16), DTYPE), (dict(ids64=2), ARG), (dict(tokens=-1), ARG),
    (dict(rows=-1), ARG), (dict(cols=-1), ARG), (dict(first_row=-1), ARG), (dict(tokens=(1 << 30) + 1), SHAPE),
    (dict(rows=1 << 30, cols=1 << 11, table_ld=1 << 11, out_ld=1 << 11), SHAPE), (dict(table_ld=63), ARG), (dict(out_ld=63), ARG),
    (dict(table_ld=1 << 45), SHAPE), (dict(ids=None), ARG), (dict(table=None), ARG), (dict(out=None), ARG),
    (dict(ids=at(0) + 4), ALIGN), (dict(ids64=0, ids=at(0) + 2), ALIGN), (dict(table=at(1) + 1), ALIGN),
    (dict(out=at(2) + 1), ALIGN), (dict(out=at(1) + 128), ARG), (dict(out=at(0) + 16), ARG),
    (dict(tokens=0, ids=None, out=None), OK), (dict(cols=0), OK)])
def test_embedding(change, status):
    assert lookup(**change) == status, abi.load().gtp_last_error()


def lookup_grad(workspace=at(3), bytes=1 << 20, **change):
    d = dict(ids=at(0), dout=at(1), grad_data=at(2), tokens=10, first_row=0, rows=100, cols=64, dout_ld=64, grad_offset=64,
             grad_numel_total=6464, scale=1.0, ids64=1, dout_dtype=BF16, grad_dtype=F32, reserved=0)
    assert set(change) <= set(d)
    return abi.load().gtp_embedding_grad_accum(C.byref(abi.gtp_embedding_grad_desc(**{**d, **change})), workspace, bytes, None)


@pytest.mark.parametrize("change,status", [
    (dict(reserved=-1), ARG), (dict(dout_dtype=U8), DTYPE), (dict(grad_dtype=U8), DTYPE), (dict(ids64=-1), ARG), (dict(rows=-1), ARG),
    (dict(first_row=-5), ARG), (dict(dout_ld=3), ARG), (dict(grad_offset=65), RANGE), (dict(grad_offset=-1), RANGE), (dict(grad_numel_total=-1), RANGE),
    (dict(grad_numel_total=1 << 62, grad_offset=1 << 61), RANGE), (dict(workspace=None), ARG), (dict(grad_data=None), ARG), (dict(ids=None), ARG),
    (dict(dout=None), ARG), (dict(workspace=at(3) + 8), ALIGN), (dict(grad_data=at(2) + 2), ALIGN), (dict(dout=at(1) + 1), ALIGN),
    (dict(bytes=100), CAPACITY), (dict(grad_data=at(1)), ARG), (dict(workspace=at(2) + 1024), ARG), (dict(workspace=at(0)), ARG),
    (dict(workspace=at(1) + 32), ARG), (dict(workspace=at(3) + 16), ALIGN), (dict(tokens=0), OK), (dict(rows=0), OK)])
def test_embedding_gradient(change, status):
    assert lookup_grad(**change) == status, abi.load().gtp_last_error()


def test_workspace_sizes():
    lib = abi.load()
    for fn in (lib.gtp_embedding_grad_workspace_bytes, lib.gtp_orthogonalize_workspace_bytes):
        assert fn(-1, 1, 1) == fn(1, -1, 1) == fn(1, 1, -1) == -1 and fn(0, 8, 8) == fn(1, 8, 0) == 0
    assert lib.gtp_embedding_grad_workspace_bytes(8192, 64128, 2048) > 0
    assert lib.gtp_embedding_grad_workspace_bytes((1 << 30) + 1, 1, 1) == -1
    assert lib.gtp_rmsnorm_grad_workspace_bytes(-1, 1) == lib.gtp_rmsnorm_grad_workspace_bytes(1, 16385) == -1
    assert lib.gtp_rmsnorm_grad_workspace_bytes(0, 8) == 0 < lib.gtp_rmsnorm_grad_workspace_bytes(1, 1)
    assert lib.gtp_orthogonalize_workspace_bytes(65, 8, 8) == lib.gtp_orthogonalize_workspace_bytes(1, 65537, 8) == -1
    assert lib.gtp_orthogonalize_workspace_bytes(1, 46341, 46341) == -1


def norm(**change):
    d = dict(x=at(0), residual=at(1), weight=at(2), sum=at(3), y=at(4), rstd=at(5), row_codes=at(6), row_scales=at(7),
             col_codes=at(8), col_scales=at(9), rows=64, cols=96, x_ld=96, residual_ld=96, sum_ld=96, y_ld=96, eps=1e-5,
             x_dtype=BF16, residual_dtype=BF16, weight_dtype=BF16, y_dtype=BF16, tiled_scales=0, reserved=0)
    assert set(change) <= set(d)
    return abi.load().gtp_rmsnorm(C.byref(abi.gtp_rmsnorm_desc(**{**d, **change})), None)


@pytest.mark.parametrize("change,status", [
    (dict(reserved=1), ARG), (dict(tiled_scales=2), ARG), (dict(eps=-1.0), ARG), (dict(eps=float("nan")), ARG),
    (dict(eps=float("inf")), ARG), (dict(x_dtype=U8), DTYPE), (dict(residual_dtype=U8), DTYPE), (dict(weight_dtype=9), DTYPE),
    (dict(y_dtype=U8), DTYPE), (dict(rows=-1), ARG), (dict(cols=-1), ARG), (dict(rows=(1 << 30) + 1), SHAPE),
    (dict(cols=16416), SHAPE), (dict(rows=63), SHAPE), (dict(cols=80), SHAPE), (dict(rows=32 * 65536), SHAPE),
    (dict(sum=None), ARG), (dict(residual=None), ARG), (dict(row_scales=None), ARG), (dict(col_codes=None), ARG),
    (dict(rstd=None), ARG), (dict(x=None), ARG), (dict(weight=None), ARG), (dict(x=at(0) + 1), ALIGN), (dict(rstd=at(5) + 2), ALIGN),
    (dict(x_ld=95), ARG), (dict(sum_ld=95), ARG), (dict(x_ld=1 << 50), SHAPE), (dict(x=at(0) + 8), ALIGN),
    (dict(x_ld=100), ALIGN), (dict(weight=at(2) + 4), ALIGN), (dict(row_codes=at(6) + 4), ALIGN), (dict(col_codes=at(8) + 8), ALIGN),
    (dict(y=at(0) + 192), ARG), (dict(sum=at(1) + 192), ARG), (dict(y=at(1)), ARG), (dict(y=at(3)), ARG), (dict(rstd=at(2)), ARG),
    (dict(row_codes=at(4)), ARG), (dict(col_scales=at(9), row_scales=at(9)), ARG), (dict(row_codes=at(8) + 64), ARG),
    (dict(residual=None, sum=None, y=at(0)), ARG),
    (dict(residual=None, sum=None, y=None, rstd=None, row_codes=None, row_scales=None, col_codes=None, col_scales=None), ARG),
    (dict(rows=0), OK), (dict(cols=0), OK)])
def test_norm(change, status):
    assert norm(**change) == status, abi.load().gtp_last_error()


def test_null_descriptors():
    assert abi.load().gtp_embedding(None, None) == ARG and abi.load().gtp_embedding_grad_accum(None, at(1), 1 << 20, None) == ARG
    assert abi.load().gtp_rmsnorm(None, None) == ARG and abi.load().gtp_rmsnorm_grad(None, at(1), 1 << 20, None) == ARG


def norm_grad(workspace=at(8), bytes=1 << 20, **change):
    d = dict(dy=at(0), sum=at(1), weight=at(2), dsum=at(3), rstd=at(4), dx=at(5), grad_data=at(6), rows=10, cols=96, dy_ld=96,
             sum_ld=96, dsum_ld=96, dx_ld=96, grad_offset=4, grad_numel_total=100, dy_dtype=BF16, sum_dtype=BF16,
             weight_dtype=F32, grad_dtype=F32, reserved=0)
    assert set(change) <= set(d)
    return abi.load().gtp_rmsnorm_grad(C.byref(abi.gtp_rmsnorm_grad_desc(**{**d, **change})), workspace, bytes, None)


@pytest.mark.parametrize("change,status", [
    (dict(reserved=7), ARG), (dict(dy_dtype=U8), DTYPE), (dict(sum_dtype=U8), DTYPE), (dict(weight_dtype=U8), DTYPE),
    (dict(grad_dtype=U8), DTYPE), (dict(rows=-1), ARG), (dict(cols=16385), SHAPE), (dict(grad_offset=5), RANGE),
    (dict(grad_offset=-1), RANGE), (dict(dy=None), ARG), (dict(sum=None), ARG), (dict(dx=None), ARG), (dict(weight=None), ARG),
    (dict(rstd=None), ARG), (dict(grad_data=None), ARG), (dict(workspace=None), ARG), (dict(workspace=at(8) + 8), ALIGN),
    (dict(bytes=64), CAPACITY), (dict(rstd=at(4) + 1), ALIGN), (dict(grad_data=at(6) + 2), ALIGN), (dict(dx=at(5) + 1), ALIGN),
    (dict(dx_ld=90), ARG), (dict(dx=at(0) + 2), ARG), (dict(dx=at(3), dx_ld=97), ARG), (dict(dx=at(2)), ARG),
    (dict(grad_data=at(5)), ARG), (dict(workspace=at(1)), ARG), (dict(grad_data=at(4)), ARG), (dict(workspace=at(6)), ARG),
    (dict(dy_dtype=F32, dx=at(0)), ARG), (dict(rows=0), OK), (dict(cols=0), OK)])
def test_norm_gradient(change, status):
    assert norm_grad(**change) == status, abi.load().gtp_last_error()


@pytest.mark.parametrize("args,status", [
    ((at(0), at(1), 0, 4, 64, at(2), U8), DTYPE), ((at(0), at(1), 2, 4, 64, at(2), F32), ARG), ((at(0), at(1), 0, -4, 64, at(2), F32), ARG),
    ((at(0), at(1), 0, 4, 48, at(2), F32), SHAPE), ((at(0), at(1), 0, 1 << 30, 1 << 20, at(2), F32), SHAPE),
    ((None, at(1), 0, 4, 64, at(2), F32), ARG), ((at(0), None, 0, 4, 64, at(2), F32), ARG), ((at(0), at(1), 0, 4, 64, None, F32), ARG),
    ((at(0) + 8, at(1), 0, 4, 64, at(2), F32), ALIGN), ((at(0), at(1), 0, 4, 64, at(2) + 2, F32), ALIGN),
    ((at(0), at(1), 0, 4, 64, at(0) + 128, BF16), ARG), ((at(0), at(1), 1, 4, 64, at(1) + 256, BF16), ARG), ((at(0), at(1), 0, 0, 64, None, F32), OK)])
def test_mxfp8_dequantize(args, status):
    assert abi.load().gtp_mxfp8_dequantize(*args, None) == status


ABC = abi.COEFFICIENTS_PACK(3.4445, -4.7750, 2.0315)
ORTHO = dict(src=at(0), src_dt=F32, src_ld=64, src_plane=2048, dst=at(1), dst_dt=BF16, dst_ld=64, dst_plane=2048, count=2, rows=32,
             cols=64, coefficients=ABC, steps=5, workspace=at(2), bytes=1 << 24)


@pytest.mark.parametrize("change,status", [
    (dict(src_dt=U8), DTYPE), (dict(dst_dt=U8), DTYPE), (dict(count=-1), ARG), (dict(count=65), CAPACITY), (dict(rows=-1), ARG),
    (dict(cols=65537), SHAPE), (dict(rows=40000, cols=60000), SHAPE), (dict(coefficients=None), ARG), (dict(steps=0), ARG),
    (dict(steps=17), ARG), (dict(coefficients=abi.COEFFICIENTS_PACK(float("nan"), 0, 0)), ARG),
    (dict(coefficients=abi.COEFFICIENTS_PACK(3.0, 0, 0)), ARG), (dict(coefficients=abi.COEFFICIENTS_PACK(100.0, -100.0, 1.0)), ARG),
    (dict(src=None), ARG), (dict(dst=None), ARG), (dict(workspace=None), ARG), (dict(src_ld=63), ARG), (dict(dst_ld=63), ARG),
    (dict(src_plane=-1), ARG), (dict(dst_plane=2047), ARG), (dict(src_ld=1 << 43), SHAPE), (dict(src=at(0) + 2), ALIGN),
    (dict(dst=at(1) + 1), ALIGN), (dict(workspace=at(2) + 16), ALIGN), (dict(bytes=1000), CAPACITY), (dict(workspace=at(0)), ARG),
    (dict(workspace=at(1) + 4096), ARG), (dict(count=0), OK), (dict(rows=0), OK)])
def test_orthogonalize(change, status):
    assert abi.load().gtp_orthogonalize(*{**ORTHO, **change}.values(), None) == status, abi.load().gtp_last_error()


def muon(offsets=(0, 2048), hparams=None, **change):
    a = dict(grad=at(0), grad_dt=F32, momentum=at(1), master=at(2), param=at(3), numel=4096, count=2, rows=32, cols=64,
             workspace=at(4), bytes=1 << 24)
    a.update(change)
    h = abi.gtp_muon_hparams(lr=1e-3, momentum=0.9, weight_decay=0.1, scale=1.0, grad_factor=1.0,
                             coefficients=(3.4445, -4.7750, 2.0315), steps=5, nesterov=1, zero_grad_after=1)
    for k, v in (hparams or {}).items():
        setattr(h, k, v)
    o = None if offsets is None else (C.c_int64 * len(offsets))(*offsets)
    return abi.load().gtp_muon_step(a["grad"], a["grad_dt"], a["momentum"], a["master"], a["param"], a["numel"], o, a["count"],
                                    a["rows"], a["cols"], C.byref(h), a["workspace"], a["bytes"], None)


@pytest.mark.parametrize("change,status", [
    (dict(grad_dt=U8), DTYPE), (dict(count=-1), ARG), (dict(count=65), CAPACITY), (dict(numel=-1), ARG), (dict(grad=None), ARG),
    (dict(momentum=None), ARG), (dict(master=None), ARG), (dict(offsets=None), ARG), (dict(offsets=(0, 2049)), RANGE),
    (dict(offsets=(0, -1)), RANGE), (dict(offsets=(0, 2047)), RANGE), (dict(offsets=(100, 0)), RANGE), (dict(grad=at(0) + 2), ALIGN),
    (dict(param=at(3) + 1), ALIGN), (dict(workspace=None), ARG), (dict(workspace=at(4) + 128), ALIGN), (dict(bytes=5), CAPACITY),
    (dict(momentum=at(0)), ARG), (dict(param=at(2) + 64), ARG), (dict(workspace=at(3)), ARG),
    (dict(hparams=dict(lr=-1.0)), ARG), (dict(hparams=dict(momentum=1.0)), ARG), (dict(hparams=dict(weight_decay=float("nan"))), ARG),
    (dict(hparams=dict(scale=float("inf"))), ARG), (dict(hparams=dict(grad_factor=float("nan"))), ARG), (dict(hparams=dict(steps=0)), ARG),
    (dict(hparams=dict(nesterov=2)), ARG), (dict(hparams=dict(zero_grad_after=-1)), ARG), (dict(hparams=dict(reserved=1)), ARG),
    (dict(hparams=dict(grad_scale=at(5) + 2)), ALIGN), (dict(hparams=dict(grad_scale=at(1) + 16)), ARG),
    (dict(offsets=(), count=0), OK), (dict(rows=0), OK)])
def test_muon_step(change, status):
    assert muon(**change) == status, abi.load().gtp_last_error()


def test_muon_step_without_hyper_parameters():
    assert abi.load().gtp_muon_step(at(0), F32, at(1), at(2), at(3), 10, (C.c_int64 * 1)(0), 1, 2, 2, None, at(4), 1 << 20, None) == ARG
