"""The cases by which the operators around a layer's linears are measured, and their plain forms.

Three operators and their gradients: the token embedding of a vocabulary shard (its gradient accumulates into
the flat gradient buffer), the root-mean-square norm with the residual's addition (its output in bf16 or as
the two MXFP8 views that the linears read), and the orthogonalised update of the layer-wise optimizer
(Newton-Schulz products, and the whole step on weights of the flat buffers).  ``run`` computes a pass in
elementary torch operations (32-bit arithmetic, rounded once at the end), or, where ``own`` is true, through
``param_buffers_gb300``.  ``exact`` computes the same outputs in 64 bits from the definitions.

Definitions that both forms follow:

* Embedding: out[t] = scale * table[ids[t] - first_row] for ids of the shard, 0 for others.  Gradient:
  grad[ids[t] - first_row] += scale * dout[t], the sum formed in 32 bits and rounded once to the buffer's type.
* Norm: s = x + residual, rounded to the residual's type (s = x where there is none); r = 1 / sqrt(mean s^2 +
  eps) of each row; y = s r w.  Gradient: with g = dy w and n = s r, dx = r (g - n mean(g n)) + dsum, and the
  weight's gradient buffer grows by the sum over rows of dy n.
* MXFP8 (OCP microscaling): blocks of 32 along a row, E4M3 elements under one E8M0 scale byte e + 127 with
  e = floor(log2 amax) - 8; ties to even, saturated at 448.  The columnwise view is the rowwise one of the
  transposed matrix.
* Orthogonalised update: X = G / |G|_F, then `steps` times X <- a X + (b A + c A^2) X with A = X X^T (the
  smaller Gram matrix: X^T X on the other side where there are more rows than columns).
* Step: m <- mu m + (1 - mu) g;  u = mu m + (1 - mu) g;  O = orthogonalised u;
  p <- p (1 - lr wd) - lr scale O;  param = bf16(p);  grad = 0.
"""
import math

import torch

own = False

DEVICE = torch.device("cuda" if torch.cuda.is_available() else "cpu")
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
DTYPES = {"bf16": BF16, "f32": F32}
COEFFICIENTS = (3.4445, -4.7750, 2.0315)
STEPS = 5
EPS = 1e-5
MU, LR, DECAY = 0.95, 3e-4, 0.1


# --------------------------------------------------------------------------- cases

def listed():
    return [
        # one new token of a decoding step
        dict(name="embedding 1 token", op="embedding", tokens=1, rows=64128, cols=2048, table="bf16", out="bf16",
             wide=True),
        # a whole microbatch into an fp32 residual stream
        dict(name="embedding microbatch", op="embedding", tokens=8192, rows=64128, cols=2048, table="bf16", out="f32",
             wide=True),
        # a short ragged sequence onto a small shard's bf16 gradient buffer, a quarter of it padding
        dict(name="embedding gradient ragged", op="embedding gradient", tokens=1111, rows=4001, cols=1000,
             dout="bf16", grad="bf16", padded=0.25, wide=False),
        # a microbatch onto the embedding half of a pipeline's first stage
        dict(name="embedding gradient", op="embedding gradient", tokens=8192, rows=64128, cols=2048, dout="bf16",
             grad="f32", padded=0.0, wide=True),
        # one token before the attention block
        dict(name="norm 1 token", op="norm", rows=1, cols=2048, x="bf16", residual="bf16", weight="bf16",
             views=False),
        # a ragged batch on an fp32 residual stream, rows that start anywhere
        dict(name="norm ragged", op="norm", rows=8001, cols=1535, x="bf16", residual="f32", weight="f32", views=False),
        # a microbatch before the MXFP8 QKV or fc1: both views, for the forward and for wgrad
        dict(name="norm MXFP8", op="norm", rows=8192, cols=2048, x="bf16", residual="bf16", weight="bf16", views=True),
        # the same microbatch's backward, with the residual stream's own gradient
        dict(name="norm gradient", op="norm gradient", rows=8192, cols=2048, dy="bf16", stream="bf16", weight="bf16",
             residual=True),
        # the smallest linear's momentum
        dict(name="orthogonalize small", op="orthogonalize", count=1, rows=512, cols=256, src="f32", out="bf16"),
        # fc1's momentum: the largest matrix of the layer, more rows than columns
        dict(name="orthogonalize fc1", op="orthogonalize", count=1, rows=8192, cols=2048, src="f32", out="bf16"),
        # a ragged matrix's step
        dict(name="step ragged", op="step", count=1, rows=777, cols=1111),
        # the QKV weights of a stage's eight layers in one call
        dict(name="step QKV x 8", op="step", count=8, rows=1536, cols=2048),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["embedding", "embedding gradient", "norm", "norm gradient", "orthogonalize", "step"])
    if op == "embedding":
        return dict(op=op, tokens=_log(rng, 1, 16384), rows=_log(rng, 128, 64128), cols=_log(rng, 16, 4096),
                    table=rng.choice(["bf16", "f32"]), out=rng.choice(["bf16", "f32"]), wide=rng.choice([False, True]))
    if op == "embedding gradient":
        return dict(op=op, tokens=_log(rng, 1, 16384), rows=_log(rng, 128, 32000), cols=_log(rng, 16, 2048),
                    dout=rng.choice(["bf16", "f32"]), grad=rng.choice(["bf16", "f32"]),
                    padded=rng.choice([0.0, 0.0, 0.25]), wide=rng.choice([False, True]))
    if op == "norm":
        views = rng.choice([False, True])
        rows, cols = _log(rng, 1, 8192), _log(rng, 32, 8192)
        if views:  # whole blocks in both directions
            rows, cols = 32 * max(1, rows // 32), 32 * max(1, cols // 32)
        return dict(op=op, rows=rows, cols=cols, x=rng.choice(["bf16", "f32"]),
                    residual=rng.choice(["none", "bf16", "f32"]), weight=rng.choice(["bf16", "f32"]), views=views)
    if op == "norm gradient":
        return dict(op=op, rows=_log(rng, 1, 8192), cols=_log(rng, 32, 8192), dy=rng.choice(["bf16", "f32"]),
                    stream=rng.choice(["bf16", "f32"]), weight=rng.choice(["bf16", "f32"]),
                    residual=rng.choice([False, True]))
    rows, cols = _log(rng, 16, 4096), _log(rng, 16, 4096)
    if op == "orthogonalize":
        return dict(op=op, count=rng.randint(1, 3), rows=rows, cols=cols, src=rng.choice(["bf16", "f32"]), out="bf16")
    return dict(op=op, count=rng.randint(1, 3), rows=rows, cols=cols)


def work(case):
    op = case["op"]
    size = {"bf16": 2, "f32": 4}
    if op in ("embedding", "embedding gradient"):
        T, V, C = case["tokens"], case["rows"], case["cols"]
        ids = T * (8 if case["wide"] else 4)
        padding = int(T * case.get("padded", 0.0))
        rank = torch.arange(1, 2 * V + 1, dtype=F64)  # by frequency, as _ids draws them
        rows = float((1 - (1 - torch.log1p(1 / rank) / math.log(2 * V + 1)) ** (T - padding)).sum()) / 2
        if op == "embedding":
            return {"bytes": ids + rows * C * size[case["table"]] + T * C * size[case["out"]], "flops": 0}
        tokens = (T - padding) / 2 + padding
        return {"bytes": ids + tokens * C * size[case["dout"]] + 2 * rows * C * size[case["grad"]], "flops": 0}
    if op == "norm":
        n, stream = case["rows"] * case["cols"], size[case["residual"]] if case["residual"] != "none" else 0
        # both views' values (bf16), or y
        return {"bytes": n * (size[case["x"]] + 2 * stream + (4 if case["views"] else 2)), "flops": 0}
    if op == "norm gradient":
        n, stream = case["rows"] * case["cols"], size[case["stream"]]
        return {"bytes": n * (size[case["dy"]] + stream * (3 if case["residual"] else 2)), "flops": 0}
    m, n = sorted((case["rows"], case["cols"]))
    flops = case["count"] * STEPS * (3 * m * m * n + m ** 3)  # a symmetric product is half of one
    if op == "orthogonalize":
        return {"bytes": case["count"] * m * n * (size[case["src"]] + size[case["out"]]), "flops": flops}
    return {"bytes": case["count"] * m * n * 26, "flops": flops}  # grad, momentum, master twice each, param once


# --------------------------------------------------------------------------- inputs

def _randn(shape, std, dtype, g):
    return (torch.randn(shape, generator=g, device=DEVICE, dtype=F32) * std).to(dtype)


def _ids(tokens, vocabulary, padded, wide, g):
    """Token ids of a text: a few frequent ones, many rare ones, spread over the vocabulary; the last of a padded
    batch are one and the same."""
    u = torch.rand(tokens, generator=g, device=DEVICE, dtype=F64)
    rank = torch.exp(u * math.log(vocabulary)).long().clamp(max=vocabulary) - 1
    ids = torch.randperm(vocabulary, generator=g, device=DEVICE)[rank]
    ids[tokens - int(tokens * padded):] = vocabulary // 2
    return ids if wide else ids.to(torch.int32)


def _gradient(shape, g):
    """A matrix as weight gradients are: a few strong directions, every row with a size of its own, noise."""
    count, rows, cols = shape
    k = min(64, rows, cols)
    strength = torch.arange(1, k + 1, device=DEVICE, dtype=F32) ** -0.7
    left, right = _randn((count, rows, k), 1.0, F32, g), _randn((count, k, cols), 1.0, F32, g)
    size = torch.exp(0.5 * _randn((count, rows, 1), 1.0, F32, g))
    return 1e-4 * size * ((left * strength) @ right + 0.5 * _randn(shape, 1.0, F32, g))


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    op = case["op"]
    s = {"case": dict(case)}
    if op in ("embedding", "embedding gradient"):
        T, V, C = case["tokens"], case["rows"], case["cols"]
        s["first_row"], s["scale"] = V, math.sqrt(C)  # the second of two shards
        s["ids"] = _ids(T, 2 * V, case.get("padded", 0.0), case["wide"], g)
        if op == "embedding":
            s["ids"][T // 2] = V + int(torch.randint(V, (1,), generator=g, device=DEVICE))  # of the shard, if only one
            s["table"] = _randn((V, C), 0.02, DTYPES[case["table"]], g)
            s["out"] = torch.empty(T, C, dtype=DTYPES[case["out"]], device=DEVICE)
        else:
            s["dout"] = _randn((T, C), 1e-3, DTYPES[case["dout"]], g)
            s["main_grad"] = _randn((V * C,), 1e-2, DTYPES[case["grad"]], g)
    elif op == "norm":
        R, C = case["rows"], case["cols"]
        # a few columns of the residual stream are far larger than the others
        wide = torch.where(torch.rand(C, generator=g, device=DEVICE) < 0.01, 20.0, 1.0)
        s["x"] = (_randn((R, C), 1.0, F32, g) * wide).to(DTYPES[case["x"]])
        s["weight"] = (1 + _randn((C,), 0.1, F32, g)).to(DTYPES[case["weight"]])
        s["rstd"] = torch.empty(R, dtype=F32, device=DEVICE)
        s["residual"] = s["sum"] = None
        if case["residual"] != "none":
            s["residual"] = (_randn((R, C), 3.0, F32, g) * wide).to(DTYPES[case["residual"]])
            s["sum"] = torch.empty_like(s["residual"])
        if case["views"]:
            u8 = dict(dtype=torch.uint8, device=DEVICE)
            s["row"] = torch.empty(R, C, **u8), torch.empty(R, C // 32, **u8)
            s["col"] = torch.empty(C, R, **u8), torch.empty(C, R // 32, **u8)
            s["out"] = torch.empty(R, C, dtype=BF16, device=DEVICE), torch.empty(C, R, dtype=BF16, device=DEVICE)
        else:
            s["y"] = torch.empty(R, C, dtype=BF16, device=DEVICE)
    elif op == "norm gradient":
        R, C = case["rows"], case["cols"]
        stream = DTYPES[case["stream"]]
        s["dy"] = (_randn((R, C), 1e-3, F32, g) * torch.exp(_randn((R, 1), 1.0, F32, g))).to(DTYPES[case["dy"]])
        s["sum"] = _randn((R, C), 3.0, stream, g)
        s["rstd"] = torch.rsqrt(s["sum"].float().square().mean(1) + EPS)
        s["weight"] = (1 + _randn((C,), 0.1, F32, g)).to(DTYPES[case["weight"]])
        s["dsum"] = _randn((R, C), 1e-3, stream, g) if case["residual"] else None
        s["dx"] = torch.empty(R, C, dtype=stream, device=DEVICE)
        s["main_grad"] = _randn((C,), 1e-2, F32, g)
    elif op == "orthogonalize":
        shape = case["count"], case["rows"], case["cols"]
        s["src"] = _gradient(shape, g).to(DTYPES[case["src"]])
        s["out"] = torch.empty(shape, dtype=DTYPES[case["out"]], device=DEVICE)
    else:
        count, R, C = case["count"], case["rows"], case["cols"]
        each = (R * C + 63) // 64 * 64  # weights start on multiples of 64 elements in the flat buffers
        s["offsets"], s["scale"] = [k * each for k in range(count)], 0.2 * math.sqrt(max(R, C))
        zeros = torch.zeros(count, each, dtype=F32, device=DEVICE)

        def flat(x):
            out = zeros.clone()
            out[:, :R * C] = x.reshape(count, -1)
            return out.reshape(-1)
        shape = count, R, C
        s["momentum"] = flat(_gradient(shape, g))
        s["grad"] = flat(_gradient(shape, g))
        s["master"] = flat(_randn(shape, 0.02, F32, g))
        s["param"] = s["master"].to(BF16)
    return s


# --------------------------------------------------------------------------- plain forms

def _local(s):
    """Rows of the shard and whether each token has one (row 0 where not)."""
    at = s["ids"].long() - s["first_row"]
    mine = (at >= 0) & (at < s["case"]["rows"])
    return torch.where(mine, at, 0), mine


def _mx_values(x):
    """The values of fp32 x's rowwise MXFP8 view."""
    R, C = x.shape
    x = x.view(R, C // 32, 32)
    byte = ((x.abs().amax(-1, keepdim=True).view(torch.int32) >> 23) - 8).clamp(min=0)
    y = x * ((254 - byte) << 23).view(F32)
    y = y.clamp(-448, 448).to(torch.float8_e4m3fn).float()
    scale = torch.where(byte == 0, 2.0 ** -127, (byte << 23).view(F32))
    return (y * scale).reshape(R, C)


def _orthogonal(X):
    """X [count, rows, cols] in fp32, orthogonalised."""
    a, b, c = COEFFICIENTS
    tall = X.shape[1] > X.shape[2]
    if tall:
        X = X.transpose(1, 2)
    norm = X.double().square().sum((1, 2), keepdim=True).sqrt()
    X = (X / torch.where(norm > 0, norm, 1.0)).float()
    for _ in range(STEPS):
        A = X @ X.transpose(1, 2)
        X = a * X + (b * A + c * (A @ A)) @ X
    return X.transpose(1, 2) if tall else X


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    if op == "embedding":
        at, mine = _local(s)
        return torch.where(mine[:, None], s["table"][at].float() * s["scale"], 0.0).to(s["out"].dtype)
    if op == "embedding gradient":
        at, mine = _local(s)
        d = torch.where(mine[:, None], s["dout"].float() * s["scale"], 0.0)
        grad = s["main_grad"].view(case["rows"], case["cols"])
        if grad.dtype == F32:
            grad.index_add_(0, at, d)
        else:
            grad.copy_(grad.float() + torch.zeros(grad.shape, device=grad.device).index_add_(0, at, d))
        return s["main_grad"]
    if op == "norm":
        out = {}
        h = s["x"].float()
        if s["residual"] is not None:
            out["sum"] = (h + s["residual"].float()).to(s["residual"].dtype)
            h = out["sum"].float()
        out["rstd"] = torch.rsqrt(h.square().mean(1) + EPS)
        y = h * out["rstd"][:, None] * s["weight"].float()
        if case["views"]:
            out["row"], out["col"] = _mx_values(y).to(BF16), _mx_values(y.t().contiguous()).to(BF16)
        else:
            out["y"] = y.to(BF16)
        return out
    if op == "norm gradient":
        dy, r = s["dy"].float(), s["rstd"][:, None]
        n = s["sum"].float() * r
        g = dy * s["weight"].float()
        dx = r * (g - n * (g * n).mean(1, keepdim=True))
        if s["dsum"] is not None:
            dx = dx + s["dsum"].float()
        s["main_grad"].add_((dy * n).sum(0))
        return {"dx": dx.to(s["dx"].dtype), "main_grad": s["main_grad"]}
    if op == "orthogonalize":
        return _orthogonal(s["src"].float()).to(s["out"].dtype)
    count, R, C = case["count"], case["rows"], case["cols"]
    view = lambda x: x.view(count, -1)[:, :R * C].reshape(count, R, C)
    grad = view(s["grad"])
    momentum = MU * view(s["momentum"]) + (1 - MU) * grad
    update = _orthogonal(MU * momentum + (1 - MU) * grad)
    master = view(s["master"]) * (1 - LR * DECAY) - (LR * s["scale"]) * update
    for name, x in (("momentum", momentum), ("master", master), ("param", master.to(BF16))):
        s[name].view(count, -1)[:, :R * C] = x.reshape(count, -1)
    s["grad"].zero_()
    return {k: s[k] for k in ("grad", "momentum", "master", "param")}


# --------------------------------------------------------------------------- the framework's calls

def _workspace(s, bytes_of, *sizes):
    """The workspace that a program keeps beside its buffers."""
    if "workspace" not in s:
        s["workspace"] = torch.empty(bytes_of(*sizes), dtype=torch.uint8, device=DEVICE)
    return s["workspace"]


def _run_own(s):
    import param_buffers_gb300 as gtp
    case = s["case"]
    op = case["op"]
    if op == "embedding":
        gtp.gtp_embedding(s["ids"], s["table"], s["out"], first_row=s["first_row"], scale=s["scale"])
        return s["out"]
    if op == "embedding gradient":
        ws = _workspace(s, gtp.gtp_embedding_grad_workspace_bytes, case["tokens"], case["rows"], case["cols"])
        gtp.gtp_embedding_grad_accum(s["dout"], s["ids"], s["main_grad"], 0, case["rows"], ws,
                                     first_row=s["first_row"], scale=s["scale"])
        return s["main_grad"]
    if op == "norm":
        views = dict(row=s["row"], col=s["col"]) if case["views"] else dict(y=s["y"])
        gtp.gtp_rmsnorm(s["x"], s["weight"], EPS, residual=s["residual"], sum=s["sum"], rstd=s["rstd"], **views)
        out = {"rstd": s["rstd"]}
        if s["sum"] is not None:
            out["sum"] = s["sum"]
        if not case["views"]:
            return out | {"y": s["y"]}
        gtp.gtp_mxfp8_dequantize(*s["row"], s["out"][0])
        gtp.gtp_mxfp8_dequantize(*s["col"], s["out"][1])
        return out | {"row": s["out"][0], "col": s["out"][1]}
    if op == "norm gradient":
        ws = _workspace(s, gtp.gtp_rmsnorm_grad_workspace_bytes, case["rows"], case["cols"])
        gtp.gtp_rmsnorm_grad(s["dy"], s["sum"], s["rstd"], s["weight"], s["dx"], s["main_grad"], 0, ws,
                             dsum=s["dsum"])
        return {"dx": s["dx"], "main_grad": s["main_grad"]}
    ws = _workspace(s, gtp.gtp_orthogonalize_workspace_bytes, case["count"], case["rows"], case["cols"])
    if op == "orthogonalize":
        gtp.gtp_orthogonalize(s["src"], s["out"], ws, steps=STEPS, coefficients=COEFFICIENTS)
        return s["out"]
    h = gtp.MuonHparams(lr=LR, momentum=MU, weight_decay=DECAY, scale=s["scale"], nesterov=True, steps=STEPS,
                        coefficients=COEFFICIENTS, zero_grad_after=True)
    gtp.gtp_muon_step(s["grad"], s["momentum"], s["master"], s["param"], s["offsets"], case["rows"], case["cols"], h, ws)
    return {k: s[k] for k in ("grad", "momentum", "master", "param")}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# --------------------------------------------------------------------------- 64 bits

def _exact_mx(x):
    """The rowwise MXFP8 view's values of a float64 matrix, rounded at the elements' own spacing."""
    R, C = x.shape
    x = x.view(R, C // 32, 32)
    _, exponent = torch.frexp(x.abs().amax(-1, keepdim=True))  # amax = mantissa * 2^exponent, mantissa in [0.5, 1)
    e = torch.where(x.abs().amax(-1, keepdim=True) > 0, exponent - 9, -127).clamp(min=-127)
    y = torch.ldexp(x, -e)
    _, own_exponent = torch.frexp(y)
    spacing = (own_exponent - 4).clamp(min=-9)  # three fractional bits of a normal number, subnormal below 2^-6
    y = torch.ldexp(torch.round(torch.ldexp(y, -spacing)), spacing).clamp(-448, 448)  # ties to even
    return torch.ldexp(y, e).reshape(R, C)


def _exact_orthogonal(X):
    """Through the Gram matrix's eigenvalues: every product is a function of them, l <- l f(l)^2 with
    f(l) = a + b l + c l^2, and X becomes Q (product of the f) Q^T X."""
    a, b, c = COEFFICIENTS
    out = []
    for G in X:
        tall = G.shape[0] > G.shape[1]
        G = G.t() if tall else G
        total = torch.linalg.vector_norm(G)
        G = G / total if total > 0 else G
        value, Q = torch.linalg.eigh(G @ G.t())
        factor = torch.ones_like(value)
        for _ in range(STEPS):
            f = a + value * (b + c * value)
            factor, value = factor * f, value * f * f
        G = (Q * factor) @ (Q.t() @ G)
        out.append(G.t() if tall else G)
    return torch.stack(out)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "embedding":
        out = torch.zeros(case["tokens"], case["cols"], dtype=F64, device=DEVICE)
        at = s["ids"].long() - s["first_row"]
        mine = torch.nonzero((at >= 0) & (at < case["rows"]))[:, 0]
        out[mine] = s["table"][at[mine]].double() * s["scale"]
        return out
    if op == "embedding gradient":
        # tokens in the order of their rows; a row's sum is the difference of two running sums
        grad = s["main_grad"].double().view(case["rows"], case["cols"])
        at = s["ids"].long() - s["first_row"]
        order = torch.argsort(at, stable=True)
        running = torch.cumsum(s["dout"][order].double() * s["scale"], 0)
        running = torch.cat((torch.zeros_like(running[:1]), running))
        edges = torch.searchsorted(at[order], torch.arange(case["rows"] + 1, device=DEVICE))
        grad += running[edges[1:]] - running[edges[:-1]]
        return grad.reshape(-1)
    if op == "norm":
        out = {}
        h = s["x"].double()
        if s["residual"] is not None:
            h = (h + s["residual"].double()).to(s["residual"].dtype).double()
            out["sum"] = h
        out["rstd"] = 1 / torch.sqrt((h * h).sum(1) / case["cols"] + EPS)
        y = torch.einsum("rc,r,c->rc", h, out["rstd"], s["weight"].double())
        if case["views"]:
            return out | {"row": _exact_mx(y), "col": _exact_mx(y.t().contiguous())}
        return out | {"y": y}
    if op == "norm gradient":
        dy, h, r, w = (s[k].double() for k in ("dy", "sum", "rstd", "weight"))
        dot = torch.einsum("rc,rc,c->r", dy, h, w)
        dx = torch.einsum("rc,r,c->rc", dy, r, w) - h * (r ** 3 * dot / case["cols"])[:, None]
        if s["dsum"] is not None:
            dx += s["dsum"].double()
        return {"dx": dx, "main_grad": s["main_grad"].double() + torch.einsum("rc,rc,r->c", dy, h, r)}
    if op == "orthogonalize":
        return _exact_orthogonal(s["src"].double())
    count, R, C = case["count"], case["rows"], case["cols"]
    each = s["grad"].numel() // count
    out = {k: s[k].double().view(count, each) for k in ("momentum", "master")}
    g = s["grad"].double().view(count, each)[:, :R * C]
    m = out["momentum"][:, :R * C]
    m += (g - m) * (1 - MU)
    O = _exact_orthogonal((g + (m - g) * MU).view(count, R, C))
    p = out["master"][:, :R * C]
    p -= LR * (DECAY * p + s["scale"] * O.reshape(count, -1))
    return {"grad": torch.zeros_like(s["grad"], dtype=F64), "momentum": out["momentum"].reshape(-1),
            "master": out["master"].reshape(-1), "param": out["master"].reshape(-1)}
