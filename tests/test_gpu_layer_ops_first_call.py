"""The first call of a process may be one that is captured: each operator in a fresh process, captured before anything has run
it, replayed, and compared with an eager call."""
import subprocess
import sys
from pathlib import Path

import pytest

pytestmark = pytest.mark.gpu
ROOT = Path(__file__).resolve().parents[1]
SETUP = """
import torch
import param_buffers_gb300 as gtp
D, B = "cuda", torch.bfloat16
u8 = lambda *s: torch.empty(*s, dtype=torch.uint8, device=D)
T, V, C = 3000, 500, 512
x, w = torch.randn(T // 8 // 32 * 32, C, device=D), torch.randn(C, device=D)
R = x.shape[0]
ids, table, dout = torch.randint(0, V, (T,), device=D), torch.randn(V, C, device=D), torch.randn(T, C, device=D)
out, grad, rstd = torch.zeros(T, C, device=D), torch.zeros(V * C, device=D), torch.ones(R, device=D)
y, dx, gw = torch.zeros(R, C, device=D), torch.zeros(R, C, device=D), torch.zeros(C, device=D)
row, col = (u8(R, C), u8(R, C // 32)), (u8(C, R), u8(C, R // 32))
value = torch.zeros(R, C, device=D)
"""
CALLS = {
    "embedding": ("", "gtp.gtp_embedding(ids, table, out)", "out"),
    "embedding_grad": ("ws = u8(gtp.gtp_embedding_grad_workspace_bytes(T, V, C))",
                       "grad.zero_(); gtp.gtp_embedding_grad_accum(dout, ids, grad, 0, V, ws)", "grad"),
    "norm": ("", "gtp.gtp_rmsnorm(x, w, 1e-5, y=y, rstd=rstd, row=row, col=col); gtp.gtp_mxfp8_dequantize(*row, value)", "y, *col, value"),
    "norm_grad": ("ws = u8(gtp.gtp_rmsnorm_grad_workspace_bytes(R, C))",
                  "gw.zero_(); gtp.gtp_rmsnorm_grad(y, x, rstd, w, dx, gw, 0, ws)", "dx, gw"),
    "orthogonalize": ("ws = u8(gtp.gtp_orthogonalize_workspace_bytes(1, R, C)); o = torch.zeros(R, C, device=D)",
                      "gtp.gtp_orthogonalize(x, o, ws)", "o"),
    "orthogonalize_small": ("s = x[:100].contiguous(); ws = u8(gtp.gtp_orthogonalize_workspace_bytes(1, 100, C)); o = torch.zeros(100, C, device=D)",
                            "gtp.gtp_orthogonalize(s, o, ws)", "o"),
}


@pytest.mark.parametrize("name", list(CALLS))
def test_captured_first(name):
    prepare, call, outputs = CALLS[name]
    body = [SETUP, prepare, "torch.cuda.synchronize()", "g = torch.cuda.CUDAGraph()", "with torch.cuda.graph(g):", f"    {call}",
            "g.replay()", "torch.cuda.synchronize()", f"got = [t.clone() for t in ({outputs},)]", call, "torch.cuda.synchronize()",
            f"assert all(torch.equal(a, b) for a, b in zip(got, ({outputs},)))", "assert gtp.gtp_wait_timeouts() == 0", "print('same')"]
    r = subprocess.run([sys.executable, "-c", "\n".join(body)], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("same"), r.stderr[-2000:]
