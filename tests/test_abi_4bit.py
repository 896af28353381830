"""The C ABI of the MXFP4, rotary and dropout entry points without a GPU: bad arguments are refused on the host before
a device is touched, and the host-only frequencies agree with the oracle.  Fake addresses; nothing launches."""
import ctypes as C
import math

import pytest

from oracle import rotary as RO
from param_buffers_gb300 import abi

pytestmark = pytest.mark.skipif(not abi.LIB_PATH.exists(), reason="libgtp.so not built")

ALIGNED = 0x100000        # never dereferenced: every call using it fails validation first or has nothing to do


def test_mxfp4_argument_errors():
    """Bad sizes, types, alignments and overlaps of the MXFP4 calls are refused on the host."""
    lib = abi.load()
    a = [ALIGNED + k * (1 << 24) for k in range(6)]
    q = lambda src=a[0], dt=abi.GTP_F32, r=64, c=96, ld=96, rc=a[1], rs=a[2], cc=a[3], cs=a[4], rng=None: \
        lib.gtp_mxfp4_quantize(src, dt, r, c, ld, rc, rs, cc, cs, rng, None)
    assert q(dt=abi.GTP_F16) == abi.GTP_E_DTYPE
    assert q(r=-1) == abi.GTP_E_ARG and q(c=-1) == abi.GTP_E_ARG
    assert q(r=(1 << 30) + 1) == abi.GTP_E_SHAPE and q(r=1 << 29, c=1 << 29, ld=1 << 29) == abi.GTP_E_SHAPE
    assert q(ld=95) == abi.GTP_E_ARG and q(ld=(1 << 40) + 1) == abi.GTP_E_SHAPE
    assert q(src=None) == abi.GTP_E_ARG and q(src=a[0] + 2) == abi.GTP_E_ALIGN
    assert q(rc=None) == abi.GTP_E_ARG and q(cs=None) == abi.GTP_E_ARG            # half a view
    assert q(rc=None, rs=None, cc=None, cs=None) == abi.GTP_E_ARG
    assert q(rc=a[1] + 8) == abi.GTP_E_ALIGN and q(cs=a[4] + 4) == abi.GTP_E_ALIGN
    assert q(rc=a[0] + 64 * 96 * 4 - 16) == abi.GTP_E_ARG                          # codes over the source's end
    assert q(cs=a[2]) == abi.GTP_E_ARG                                              # one buffer for both scales
    assert q(rng=C.byref(abi.gtp_rng(1, 2, a[5] + 4))) == abi.GTP_E_ALIGN
    assert q(r=0, src=None, rc=None, rs=None, cc=None, cs=None) == abi.GTP_OK
    d = lambda co=a[0], s=a[1], r=64, c=96, o=a[2], dt=abi.GTP_BF16: lib.gtp_mxfp4_dequantize(co, s, r, c, o, dt, None)
    assert d(dt=abi.GTP_U8) == abi.GTP_E_DTYPE and d(r=-1) == abi.GTP_E_ARG and d(co=None) == abi.GTP_E_ARG
    assert d(co=a[0] + 8) == abi.GTP_E_ALIGN and d(o=a[2] + 1) == abi.GTP_E_ALIGN
    assert d(o=a[0] + 64 * 48 - 2) == abi.GTP_E_ARG and d(o=a[1]) == abi.GTP_E_ARG
    f = lambda fn=lib.gtp_linear_fprop_mxfp4, x=a[0], xs=a[1], w=a[2], ws=a[3], y=a[4], M=64, N=64, K=96: \
        fn(x, xs, w, ws, y, M, N, K, None)
    assert f(M=-1) == abi.GTP_E_ARG and f(N=(1 << 30) + 8) == abi.GTP_E_SHAPE
    assert f(N=12) == abi.GTP_E_ALIGN and f(y=None) == abi.GTP_E_ARG and f(x=None) == abi.GTP_E_ARG
    assert f(xs=a[1] + 4) == abi.GTP_E_ALIGN and f(y=a[4] + 8) == abi.GTP_E_ALIGN
    assert f(M=1 << 30, N=1 << 30) == abi.GTP_E_SHAPE
    assert f(y=a[0] + 64 * 48 - 16) == abi.GTP_E_ARG and f(y=a[3]) == abi.GTP_E_ARG
    assert f(fn=lib.gtp_linear_dgrad_mxfp4, K=12) == abi.GTP_E_ALIGN                # dX's rows
    assert f(M=0, x=None, xs=None, y=None) == abi.GTP_OK
    w = lambda off=0, total=64 * 96, g=a[4], M=33, N=64, K=96: \
        lib.gtp_linear_wgrad_accum_mxfp4(a[0], a[1], a[2], a[3], g, off, total, M, N, K, None)
    assert w(off=4) == abi.GTP_E_RANGE and w(off=-4) == abi.GTP_E_ARG and w(off=2, total=10 ** 6) == abi.GTP_E_ALIGN
    assert w(K=94, total=10 ** 6) == abi.GTP_E_ALIGN and w(g=None) == abi.GTP_E_ARG and w(g=a[1]) == abi.GTP_E_ARG
    assert w(M=0) == abi.GTP_OK


def test_rotary_argument_errors():
    lib = abi.load()
    turns = (C.c_uint64 * 32)()
    a = [ALIGNED + k * (1 << 24) for k in range(4)]

    def r(**kw):
        v = dict(src=a[0], dst=a[1], positions=None, pos0=0, tokens_per_position=1, positions_per_sequence=0, tokens=8,
                 src_token=384, src_group=0, src_head=64, dst_token=384, dst_group=0, dst_head=64,
                 turns=C.addressof(turns), groups=1, heads=6, head_dim=64, rot_dim=64, dtype=abi.GTP_BF16,
                 positions64=0, interleaved=0, inverse=0, scale=1.0, reserved=0)
        v.update(kw)
        return lib.gtp_rotary(C.byref(abi.gtp_rotary_desc(**v)), None)
    assert lib.gtp_rotary(None, None) == abi.GTP_E_ARG
    assert r(dtype=abi.GTP_F16) == abi.GTP_E_DTYPE
    for bad in (dict(reserved=1), dict(inverse=2), dict(interleaved=-1), dict(tokens=-1), dict(turns=None),
                dict(scale=float("inf")), dict(tokens_per_position=0), dict(positions_per_sequence=-1),
                dict(src=None), dict(dst=None), dict(src_head=-64),
                dict(dst_head=63), dict(dst_token=383),                    # heads of dst on one another
                dict(dst=a[0] + 128), dict(dst=a[0], dst_token=400),       # over the source, not in place
                dict(positions=a[1] + 64)):
        assert r(**bad) == abi.GTP_E_ARG, bad
    for bad in (dict(rot_dim=63), dict(rot_dim=66), dict(rot_dim=0), dict(head_dim=0),
                dict(head_dim=512, rot_dim=258), dict(tokens=(1 << 32) + 1), dict(heads=1 << 21),
                dict(heads=1 << 15, head_dim=1 << 16)):              # 2^31 elements in a token's heads
        assert r(**bad) == abi.GTP_E_SHAPE, bad
    assert r(src=a[0] + 1) == abi.GTP_E_ALIGN and r(positions=a[2] + 2) == abi.GTP_E_ALIGN
    assert r(positions=a[2] + 4, positions64=1) == abi.GTP_E_ALIGN
    assert r(tokens=0, src=None) == abi.GTP_OK
    assert C.sizeof(abi.gtp_rotary_desc) == 152 and C.sizeof(abi.gtp_rotary_config) == 56 and C.sizeof(abi.gtp_rng) == 24


def test_rotary_turns_against_the_oracle_and_errors():
    lib = abi.load()
    names = ("unscaled", "linear", "base", "bands", "ramp")
    for rot in (2, 64, 96, 256):
        for code, name in enumerate(names):
            if rot == 2 and name == "base":
                continue
            cfg = abi.gtp_rotary_config(500000.0, 8.0, 1.0, 4.0, 8192, rot, code)
            turns, scale = (C.c_uint64 * (rot // 2))(), C.c_float()
            assert lib.gtp_rotary_turns(C.byref(cfg), turns, C.byref(scale)) == abi.GTP_OK
            f, s = RO.frequencies(rot, 500000.0, name, 8.0, 1.0, 4.0, 8192)
            # in units of 2^-64 turn: half a unit is the format's own rounding; on both sides float64 pow and a
            # few products, 16 roundings of 2^-53
            for t, v in zip(turns, f):
                units = v / (2 * math.pi) * 2.0 ** 64
                assert abs(t - units) <= 0.5 + 16 * 2.0 ** -53 * units
            assert scale.value == pytest.approx(s, rel=2.0 ** -23)
    turns, scale = (C.c_uint64 * 128)(), C.c_float()

    def e(base=1e4, factor=2.0, low=1.0, high=4.0, ctx=8192, rot=64, scaling=0, r=0):
        cfg = abi.gtp_rotary_config(base, factor, low, high, ctx, rot, scaling, (C.c_int32 * 2)(r, 0))
        return lib.gtp_rotary_turns(C.byref(cfg), turns, C.byref(scale))
    assert e(rot=63) == e(rot=0) == e(rot=258) == e(rot=2, scaling=2) == abi.GTP_E_SHAPE
    for bad in (dict(base=1.0), dict(base=float("nan")), dict(scaling=5), dict(scaling=-1), dict(factor=0.5, scaling=1),
                dict(ctx=0, scaling=3), dict(low=4.0, scaling=4), dict(r=1)):
        assert e(**bad) == abi.GTP_E_ARG, bad
    assert lib.gtp_rotary_turns(None, turns, C.byref(scale)) == abi.GTP_E_ARG


def test_dropout_argument_errors():
    lib = abi.load()
    a = [ALIGNED + k * (1 << 24) for k in range(4)]
    rng = abi.gtp_rng(1, 2)

    def d(x=a[0], xd=abi.GTP_BF16, xl=64, res=a[1], rl=64, out=a[2], od=abi.GTP_F32, ol=64, r=8, c=64, p=0.1,
          g=C.byref(rng)):
        return lib.gtp_dropout_add(x, xd, xl, res, rl, out, od, ol, r, c, p, g, None)
    assert d(xd=abi.GTP_U8) == d(od=abi.GTP_F16) == abi.GTP_E_DTYPE
    assert d(r=-1) == d(p=-0.1) == d(p=1.5) == d(p=float("nan")) == d(g=None) == d(xl=63) == d(rl=63) == d(ol=0) \
        == d(x=None) == d(out=None) == abi.GTP_E_ARG
    assert d(r=(1 << 30) + 1) == d(xl=(1 << 40) + 1) == abi.GTP_E_SHAPE
    assert d(x=a[0] + 1) == d(out=a[2] + 2) == d(g=C.byref(abi.gtp_rng(1, 2, a[3] + 4))) == abi.GTP_E_ALIGN
    assert d(out=a[0]) == abi.GTP_E_ARG                                  # another type over the input
    assert d(out=a[1] + 256) == abi.GTP_E_ARG                            # part of the residual
    assert d(out=a[1], ol=72) == abi.GTP_E_ARG                           # the residual with other strides
    assert d(r=0, x=None, out=None) == abi.GTP_OK
    g = lambda o=a[2], dt=abi.GTP_BF16, ld=64: lib.gtp_dropout_grad(a[0], abi.GTP_BF16, 64, o, dt, ld, 8, 64, 0.1,
                                                                    C.byref(rng), None)
    assert g(o=a[0] + 64) == g(o=a[0], dt=abi.GTP_F32) == g(ld=63) == abi.GTP_E_ARG
