"""Equal calls give equal bits, whatever the workspace held before and whatever runs beside them: each operator of the layer's
sides many times over, its workspace filled anew, half of the time beside another stream's products."""
import pytest
import torch

import param_buffers_gb300 as gtp

pytestmark = pytest.mark.gpu
DEV = "cuda"
B, F = torch.bfloat16, torch.float32
FILLS = [0, 0xFF, 0x7F, 0x01, 0x80, 0x3C, 0xFF, 0]


def repeat(go, outputs, ws):
    """go() once for each fill of the workspace; outputs() are what it writes."""
    side, busy = torch.cuda.Stream(), torch.randn(2048, 2048, device=DEV).to(B)
    want = None
    for k, fill in enumerate(FILLS):
        ws.fill_(fill)
        for t in outputs:
            t.fill_(float("nan") if t.is_floating_point() else 0xAA)
        if k & 1:
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                for _ in range(20):
                    busy @ busy
        go()
        torch.cuda.synchronize()
        got = [t.clone() for t in outputs]
        want = want or got
        assert all(torch.equal(a, b) for a, b in zip(got, want)), k
    assert gtp.gtp_wait_timeouts() == 0


@pytest.mark.parametrize("count,R,C", [(1, 512, 256), (1, 84, 26), (3, 128, 500), (1, 777, 1111), (2, 1536, 2048), (1, 2048, 520)])
@pytest.mark.parametrize("od", [B, F])
def test_orthogonalize(count, R, C, od):
    src, out = 1e-3 * torch.randn(count, R, C, device=DEV), torch.empty(count, R, C, dtype=od, device=DEV)
    ws = torch.empty(gtp.gtp_orthogonalize_workspace_bytes(count, R, C), dtype=torch.uint8, device=DEV)
    repeat(lambda: gtp.gtp_orthogonalize(src, out, ws), [out], ws)


@pytest.mark.parametrize("count,R,C", [(1, 777, 1111), (8, 300, 200), (3, 40, 70)])
def test_step(count, R, C):
    n = count * R * C
    start = [1e-3 * torch.randn(n, device=DEV), 1e-3 * torch.randn(n, device=DEV), torch.randn(n, device=DEV)]
    grad, m, p = (t.clone() for t in start)
    param = torch.empty(n, dtype=B, device=DEV)
    ws = torch.empty(gtp.gtp_orthogonalize_workspace_bytes(count, R, C), dtype=torch.uint8, device=DEV)

    def go():
        for t, s in zip((grad, m, p), start):
            t.copy_(s)
        gtp.gtp_muon_step(grad, m, p, param, [k * R * C for k in range(count)], R, C, gtp.MuonHparams(), ws)
    repeat(go, [grad, m, p, param], ws)


@pytest.mark.parametrize("T,V,C", [(50, 97, 512), (1111, 401, 1000), (8192, 6000, 256), (40000, 300, 77)])
def test_embedding_gradient(T, V, C):
    ids = torch.randint(-V // 2, V + V // 2, (T,), device=DEV)
    ids[T // 2:T // 2 + T // 4] = V // 3
    dout, start = torch.randn(T, C, device=DEV), torch.randn(V * C, device=DEV)
    grad = start.clone()
    ws = torch.empty(gtp.gtp_embedding_grad_workspace_bytes(T, V, C), dtype=torch.uint8, device=DEV)

    def go():
        grad.copy_(start)
        gtp.gtp_embedding_grad_accum(dout, ids, grad, 0, V, ws)
    repeat(go, [grad], ws)


@pytest.mark.parametrize("R,C", [(1312, 2048), (640, 1280), (320, 4096), (1301, 2047)])
def test_norm_and_its_gradient(R, C):
    x, res, dy = (torch.randn(R, C, device=DEV).to(B) for _ in range(3))
    w, start = 1 + 0.2 * torch.randn(C, device=DEV), torch.randn(C, device=DEV)
    out, y, dx, rstd, grad = (torch.empty(s, dtype=t, device=DEV) for s, t in (((R, C), B), ((R, C), B), ((R, C), B), ((R,), F), ((C,), F)))
    u8 = lambda *s: torch.empty(*s, dtype=torch.uint8, device=DEV)
    views = dict(row=(u8(R, C), u8(R, C // 32)), col=(u8(C, R), u8(C, R // 32))) if C % 32 == 0 else {}
    ws = u8(gtp.gtp_rmsnorm_grad_workspace_bytes(R, C))

    def go():
        grad.copy_(start)
        gtp.gtp_rmsnorm(x, w, 1e-5, residual=res, sum=out, y=y, rstd=rstd, **views)
        gtp.gtp_rmsnorm_grad(dy, out, rstd, w, dx, grad, 0, ws, dsum=y)
    repeat(go, [out, y, rstd, dx, grad, *(t for v in views.values() for t in v)], ws)
