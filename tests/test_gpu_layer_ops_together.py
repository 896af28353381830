"""The embedding, the norms, the orthogonalised update and the operators between them, one step of a small network as a
training loop runs it, on the GPU against float64.

  ids -> embedding (fp32 stream h0) -> norm (MXFP8 views) -> MXFP8 product -> norm of (product + h0) -> loss <y2, dout>

and back into one flat gradient buffer, then the orthogonalised step of the linear's weight and the fused AdamW sweep of the
other buffer.  Each value is compared with the formula on the operands that the GPU itself rounded (its bf16 tensors, its
views' values), so what is left are the outputs' roundings: half a bf16 step, 2^-8, of each bf16 tensor on the way (the
product, dgrad's output), below 2^-8 of its norm; three of them follow one another at most, and fp32 sums below 2^-15 besides:
2e-2 of the norm bounds every chain, 1e-4 those all in fp32."""
import numpy as np
import pytest
import torch

import param_buffers_gb300 as gtp
from oracle import adamw as A
from oracle import embedding as E
from oracle import mxfp8 as MX
from oracle import orthogonalize as O
from oracle import rmsnorm as N

pytestmark = pytest.mark.gpu
DEV = "cuda"
B, F, U8 = torch.bfloat16, torch.float32, torch.uint8
EPS, SCALE = 1e-5, 16.0


def f64(t):
    return t.double().cpu().numpy()


def rel(got, want):
    return np.linalg.norm(f64(got).ravel() - want.ravel()) / np.linalg.norm(want)


class Net:
    """One shard of a vocabulary, a norm, a square linear, a second norm; the linear's weight in a buffer of its own, as
    parameters of a layer-wise optimizer have."""

    def __init__(self, T=256, H=256, V=97, seed=0):
        self.T, self.H, self.V = T, H, V
        g = torch.Generator(device=DEV).manual_seed(seed)
        randn = lambda *s: torch.randn(*s, generator=g, device=DEV)
        # flat buffer: the table, both norms' weights; elements after each other
        self.n = V * H + 2 * H
        self.at_w1, self.at_w2 = V * H, V * H + H
        self.master = torch.cat([0.02 * randn(V * H), 1 + 0.1 * randn(2 * H)])
        self.m, self.v, self.grad = (torch.zeros(self.n, device=DEV) for _ in range(3))
        self.param = self.master.to(B)
        self.table = self.param[:V * H].view(V, H)
        self.w1, self.w2 = self.param[self.at_w1:self.at_w2], self.param[self.at_w2:]
        self.lin = dict(master=0.06 * randn(H * H), momentum=torch.zeros(H * H, device=DEV), grad=torch.zeros(H * H, device=DEV))
        self.lin["param"] = self.lin["master"].to(B)
        self.ids = torch.randint(V - 20, 2 * V + 20, (T,), generator=g, device=DEV)
        self.dout = randn(T, H)
        e = lambda *s, dt=F: torch.empty(*s, dtype=dt, device=DEV)
        view = lambda r, c: (e(r, c, dt=U8), e(r, c // 32, dt=U8))
        self.h0, self.h1, self.y2, self.dh1, self.dh0 = (e(T, H) for _ in range(5))
        self.y1, self.dy1, self.dn1 = (e(T, H, dt=B) for _ in range(3))
        self.r1, self.r2 = e(T), e(T)
        self.x_row, self.x_col = view(T, H), view(H, T)
        self.d_row, self.d_col = view(T, H), view(H, T)
        self.w_row, self.w_col = view(H, H), view(H, H)
        self.ws_e = e(gtp.gtp_embedding_grad_workspace_bytes(T, V, H), dt=U8)
        self.ws_n = e(gtp.gtp_rmsnorm_grad_workspace_bytes(T, H), dt=U8)
        self.ws_o = e(gtp.gtp_orthogonalize_workspace_bytes(1, H, H), dt=U8)
        self.hp = gtp.AdamHparams(lr=1e-2, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.0)
        self.muon = gtp.MuonHparams(lr=0.02, momentum=0.9, weight_decay=0.1, scale=0.2 * H ** 0.5)
        self.bucket = [dict(offset=0, numel=self.n)]
        self.quantize_weight()

    def quantize_weight(self):
        w = self.lin["param"].view(self.H, self.H)
        gtp.gtp_mxfp8_quantize_rowwise(w, *self.w_row)
        gtp.gtp_mxfp8_quantize_columnwise(w, *self.w_col)

    def forward_backward(self):
        gtp.gtp_embedding(self.ids, self.table, self.h0, first_row=self.V, scale=SCALE)
        gtp.gtp_rmsnorm(self.h0, self.w1, EPS, rstd=self.r1, row=self.x_row, col=self.x_col)
        gtp.gtp_linear_fprop_mxfp8(*self.x_row, *self.w_row, self.y1)
        gtp.gtp_rmsnorm(self.y1, self.w2, EPS, residual=self.h0, sum=self.h1, y=self.y2, rstd=self.r2)
        gtp.gtp_rmsnorm_grad(self.dout, self.h1, self.r2, self.w2, self.dh1, self.grad, self.at_w2, self.ws_n)
        self.dy1.copy_(self.dh1)
        gtp.gtp_mxfp8_quantize_rowwise(self.dy1, *self.d_row)
        gtp.gtp_mxfp8_quantize_columnwise(self.dy1, *self.d_col)
        gtp.gtp_linear_dgrad_mxfp8(*self.d_row, *self.w_col, self.dn1)
        gtp.gtp_linear_wgrad_accum_mxfp8(*self.d_col, *self.x_col, self.lin["grad"], 0)
        gtp.gtp_rmsnorm_grad(self.dn1, self.h0, self.r1, self.w1, self.dh0, self.grad, self.at_w1, self.ws_n, dsum=self.dh1)
        gtp.gtp_embedding_grad_accum(self.dh0, self.ids, self.grad, 0, self.V, self.ws_e, first_row=self.V, scale=SCALE)

    def update(self, step):
        gtp.gtp_muon_step(self.lin["grad"], self.lin["momentum"], self.lin["master"], self.lin["param"], [0], self.H, self.H,
                          self.muon, self.ws_o)
        gtp.gtp_adam_step_flat(self.grad, self.master, self.m, self.v, self.param, self.bucket, [1.0], self.hp, step=step)
        self.quantize_weight()

    def state(self):
        return [self.master, self.m, self.v, self.param, self.grad, *self.lin.values(), self.y2, *self.x_row, *self.w_col]


def value(view):
    return MX.dequantize_rowwise(*(t.cpu().numpy() for t in view))


def test_a_step_against_float64():
    n = Net()
    n.forward_backward()
    T, H, V, ids = n.T, n.H, n.V, n.ids.tolist()
    h0 = E.lookup(ids, f64(n.table), V, SCALE)
    r1, y = N.forward(h0, f64(n.w1), EPS)
    assert rel(n.h0, h0) <= 1e-6 and rel(n.r1, r1) <= 1e-5
    # the views hold the norm: a code is off by at most 2^-4 of its value, 2^-3 where it saturates (512 to 448 of the block's
    # scale), or half the smallest step of its block
    for got, want in ((value(n.x_row), y), (value(n.x_col), y.T)):
        assert np.linalg.norm(got - want) <= 2.0 ** -3 * np.linalg.norm(want)
    X, W = value(n.x_row), value(n.w_row)
    h1 = X @ W.T + h0
    r2, y2 = N.forward(h1, f64(n.w2), EPS)
    assert rel(n.h1, h1) <= 2e-2 and rel(n.y2, y2) <= 2e-2
    dh1, dw2 = N.gradient(f64(n.dout), h1, r2, f64(n.w2))
    assert rel(n.dh1, dh1) <= 2e-2 and rel(n.grad[n.at_w2:], dw2) <= 2e-2
    dn1 = value(n.d_row) @ value(n.w_col).T
    dh0, dw1 = N.gradient(dn1, h0, r1, f64(n.w1), f64(n.dh1))
    assert rel(n.dh0, dh0) <= 2e-2 and rel(n.grad[n.at_w1:n.at_w2], dw1) <= 2e-2
    dW = value(n.d_col) @ value(n.x_col).T
    assert rel(n.lin["grad"], dW) <= 1e-4
    table, _, hits = E.gradient(ids, f64(n.dh0), V, V, SCALE)
    assert rel(n.grad[:V * H], table) <= 1e-4
    assert not n.grad[:V * H].view(V, H)[torch.from_numpy(hits == 0).to(DEV)].any()
    # the update, from the gradients that the GPU summed
    grad, master, dw, w0 = f64(n.grad), f64(n.master), f64(n.lin["grad"]).reshape(H, H), f64(n.lin["master"]).reshape(H, H)
    n.update(1)
    h = A.AdamWHparams(lr=1e-2, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.0)
    P, M, S = A.adamw(master, grad, np.zeros_like(master), np.zeros_like(master), 1, h)
    assert rel(n.master, P) <= 1e-6 and rel(n.m, M) <= 1e-6 and rel(n.v, S) <= 1e-6
    _, w = O.step(dw, np.zeros((H, H)), w0, float(np.float32(0.9)), 0.02, 0.1, 0.2 * H ** 0.5)
    assert np.linalg.norm(f64(n.lin["master"]).reshape(H, H) - w) <= 4e-3 * np.linalg.norm(w - w0 * (1 - 0.002)) + 1e-6
    assert torch.equal(n.lin["param"], n.lin["master"].to(B)) and not n.lin["grad"].any() and not n.grad.any()
    assert gtp.gtp_wait_timeouts() == 0


def capture(net, stream):
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        net.forward_backward()
        net.update(1)
    return graph


def test_two_captured_steps_side_by_side_and_sharing():
    """Replays of two networks' graphs on two streams at once give the eager steps' bits, and so do replays of two graphs
    of one network, one after the other, which share its workspaces."""
    eager = [Net(seed=k) for k in range(2)]
    for _ in range(3):
        for n in eager:
            n.forward_backward()
            n.update(1)
    nets, streams = [Net(seed=k) for k in range(2)], [torch.cuda.Stream() for _ in range(2)]
    graphs = [capture(n, s) for n, s in zip(nets, streams)]
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for a, b in zip(eager, nets):
        assert all(torch.equal(x, y) for x, y in zip(a.state(), b.state()))
    one = Net(seed=0)
    pair = [capture(one, streams[0]), capture(one, streams[1])]
    for k in (0, 1, 0):
        pair[k].replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(eager[0].state(), one.state()))
    assert gtp.gtp_wait_timeouts() == 0


def test_on_a_stream_that_is_not_current():
    """The stream argument alone decides where the kernels run: a step passed a side stream, behind that stream's work."""
    want, n = Net(seed=5), Net(seed=5)
    want.forward_backward()
    out = torch.empty(n.H, n.H, device=DEV)
    src = want.lin["grad"].view(n.H, n.H)
    gtp.gtp_orthogonalize(src, out, want.ws_o)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    h0, h1 = torch.empty_like(n.h0), torch.empty_like(n.h0)
    y, r, got = torch.empty_like(n.y2), torch.empty_like(n.r1), torch.empty_like(out)
    late = torch.zeros_like(n.ids)
    with torch.cuda.stream(s):
        torch.cuda._sleep(2_000_000)
        late.copy_(n.ids)
    gtp.gtp_embedding(late, n.table, h0, first_row=n.V, scale=SCALE, stream=s)
    gtp.gtp_rmsnorm(want.y1, n.w2, EPS, residual=h0, sum=h1, y=y, rstd=r, stream=s)
    gtp.gtp_rmsnorm_grad(n.dout, h1, r, n.w2, n.dh1, n.grad, n.at_w2, n.ws_n, stream=s)
    gtp.gtp_embedding_grad_accum(want.dh0, late, n.grad, 0, n.V, n.ws_e, first_row=n.V, scale=SCALE, stream=s)
    gtp.gtp_orthogonalize(src, got, n.ws_o, stream=s)
    s.synchronize()
    assert torch.equal(h0, want.h0) and torch.equal(y, want.y2) and torch.equal(n.dh1, want.dh1) and torch.equal(got, out)
    assert torch.equal(n.grad[:n.V * n.H], want.grad[:n.V * n.H]) and torch.equal(n.grad[n.at_w2:], want.grad[n.at_w2:])


@pytest.mark.parametrize("R,C", [(100, 90), (600, 513)])
def test_orthogonalize_on_two_streams_at_once(R, C):
    """Each with a workspace of its own; the larger ones each take the whole machine, one after the other."""
    src = [1e-3 * torch.randn(R, C, device=DEV) for _ in range(2)]
    ws = [torch.empty(gtp.gtp_orthogonalize_workspace_bytes(1, R, C), dtype=U8, device=DEV) for _ in range(2)]
    want = [torch.empty(R, C, device=DEV) for _ in range(2)]
    for x, w, o in zip(src, ws, want):
        gtp.gtp_orthogonalize(x, o, w)
    got = [torch.empty(R, C, device=DEV) for _ in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(10):
        for x, w, o, s in zip(src, ws, got, streams):
            gtp.gtp_orthogonalize(x, o, w, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert gtp.gtp_wait_timeouts() == 0
