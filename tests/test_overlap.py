"""Which outputs count as overlapping an input: columns side by side in one buffer and heads of one packed tensor do not.
The host's rule against a byte-by-byte count (no GPU), and the entry points' refusals."""
import ctypes as C
import random
import shutil
import subprocess
from pathlib import Path

import pytest

from param_buffers_gb300 import abi

ROOT = Path(__file__).resolve().parents[1]
CSRC = ROOT / "param_buffers_gb300" / "csrc"

PROGRAM = r"""
#include <cstdio>
#include "byte_range.h"
int main() {
  long long v[16];
  while (true) {
    for (auto &e : v)
      if (std::scanf("%lld", &e) != 1) return 0;
    gtp::Runs r[2];
    for (int i = 0; i < 2; ++i) {
      r[i].begin = uintptr_t(v[8 * i]);
      r[i].bytes = v[8 * i + 1];
      for (int k = 0; k < 3; ++k) r[i].dim[k] = {v[8 * i + 2 + 2 * k], v[8 * i + 3 + 2 * k]};
    }
    std::printf("%d\n", int(gtp::overlap(r[0], r[1])));
  }
}
"""


def places(begin, nbytes, dims):
    at = [begin]
    for stride, n in dims:
        at = [a + k * stride for a in at for k in range(n)]
    return {a + b for a in at for b in range(nbytes)}


@pytest.mark.skipif(shutil.which("g++") is None, reason="no host compiler")
def test_exact_on_the_same_strides_and_by_spans_otherwise(tmp_path):
    (tmp_path / "main.cpp").write_text(PROGRAM)
    exe = tmp_path / "overlap"
    subprocess.run(["g++", "-std=c++17", f"-I{CSRC}", str(tmp_path / "main.cpp"), "-o", str(exe)], check=True)
    rnd, cases, want = random.Random(0), [], []
    for _ in range(4000):
        nb, ns, strides, span = rnd.randint(1, 9), [rnd.randint(1, 4) for _ in range(3)], [], 0
        other = rnd.choice([nb, rnd.randint(1, 9)])
        span = max(nb, other)
        for n in ns:                                    # each stride clears what the smaller ones span
            strides.append(span + rnd.choice([0, 0, 1, 5, 20]))
            span += (n - 1) * strides[-1]
        dims = list(zip(strides, ns))
        rnd.shuffle(dims)
        begin, there = 5000, 5000 + rnd.randint(-2 * span, 2 * span)
        dims2 = dims if rnd.random() < 0.8 else [(s + (1 if n > 1 else 7), n) for s, n in dims]
        a, b = places(begin, nb, dims), places(there, other, dims2)
        alike = all(n == 1 or s == t for (s, n), (t, _) in zip(dims, dims2))
        hulls = max(min(a), min(b)) <= min(max(a), max(b))
        want.append(bool(a & b) if alike else hulls)
        cases.append([begin, nb, *(v for d in dims for v in d), there, other, *(v for d in dims2 for v in d)])
    text = "\n".join(" ".join(map(str, c)) for c in cases)
    got = [v == "1" for v in subprocess.run([str(exe)], input=text, check=True, capture_output=True,
                                            text=True).stdout.split()]
    assert got == want and 500 < sum(want) < 3500


@pytest.mark.skipif(not abi.LIB_PATH.exists(), reason="libgtp.so not built")
def test_columns_that_share_elements_are_refused():
    """Fake addresses; every call fails its checks."""
    lib, at, rng = abi.load(), 0x100000, abi.gtp_rng(1, 2)

    def drop(out, ld=256, x=at, res=None, cols=64, od=abi.GTP_BF16):
        return lib.gtp_dropout_add(x, abi.GTP_BF16, 256, res, 256, out, od, ld, 8, cols, 0.1, C.byref(rng), None)
    for off in (2, 126, 512 - 126, 512, 7 * 512 + 126):
        assert drop(at + off) == abi.GTP_E_ARG
    assert drop(at + 128, ld=264) == abi.GTP_E_ARG                       # other strides: what they span
    assert drop(at + (1 << 24) + 100, x=at, res=at + (1 << 24)) == abi.GTP_E_ARG


@pytest.mark.gpu
def test_columns_side_by_side_are_taken():
    """Input, residual and output as columns of one buffer, an fp32 output between bf16 rows, and heads rotated into other
    heads of the packed tensor: the same results as into buffers of their own."""
    import torch

    import param_buffers_gb300 as gtp
    for dt, n in ((torch.bfloat16, 64), (torch.float32, 72), (torch.bfloat16, 37)):
        buf = torch.randn(50, 3 * n, device="cuda").to(dt)
        x, res, out = (buf[:, k * n:(k + 1) * n] for k in range(3))
        x0, res0, own = x.clone(), res.clone(), torch.empty(50, n, dtype=dt, device="cuda")
        gtp.gtp_dropout_add(x0, res0, own, 0.3, (5, 6))
        gtp.gtp_dropout_add(x, res, out, 0.3, (5, 6))
        assert torch.equal(out, own) and torch.equal(x, x0) and torch.equal(res, res0)
        gtp.gtp_dropout_grad(x, res, 0.3, (5, 7))
        gtp.gtp_dropout_grad(x0, own, 0.3, (5, 7))
        assert torch.equal(res, own) and torch.equal(x, x0)
    store = torch.zeros(40, 192, device="cuda")
    out, x = store[:, :64], store.view(torch.bfloat16)[:, 128:192]
    x.copy_(torch.randn(40, 64))
    x0, own = x.clone(), torch.empty(40, 64, device="cuda")
    gtp.gtp_dropout_add(x, None, out, 0.3, (8, 9))
    gtp.gtp_dropout_add(x0, None, own, 0.3, (8, 9))
    assert torch.equal(out, own) and torch.equal(x, x0)
    qkv = torch.randn(33, 4, 6, 64, device="cuda").bfloat16()
    before = qkv.clone()
    turns, _ = gtp.gtp_rotary_turns(gtp.RotaryConfig(64))
    own = torch.empty(33, 4, 2, 64, dtype=torch.bfloat16, device="cuda")
    gtp.gtp_rotary(before[:, :, :2], own, turns)
    gtp.gtp_rotary(qkv[:, :, :2], qkv[:, :, 3:5], turns)
    assert torch.equal(qkv[:, :, 3:5], own)
    for keep in (slice(0, 3), slice(5, 6)):
        assert torch.equal(qkv[:, :, keep], before[:, :, keep])
