"""The cases by which the 4-bit training operators are measured, and their plain forms.

Four operators: MXFP4 quantisation, the MXFP4 products of a linear (forward, and the backward's
dgrad and wgrad accumulate), rotary positions, and dropout with the residual add.  ``run`` computes a
pass in elementary torch operations (32-bit arithmetic, rounded once at the end), or, where ``own`` is
true, through ``param_buffers_gb300``.  ``exact`` computes the same outputs in 64 bits from the
definitions.

Definitions that both forms follow:

* MXFP4 (OCP microscaling): a row is cut into blocks of 32, the last one zero-padded; an element is
  E2M1, packed two to a byte (the even element in the low nibble), a block has one E8M0 scale byte
  e + 127.  Nearest: e = floor(log2 amax) - 2, ties to even, saturated at 6.  Stochastic: e is the least
  with amax <= 6 * 2^e; y = |x| / 2^e, taken to 23 fractional bits below 1, lies between two grid points
  one step apart and goes up where its fraction of the step + (2 r + 1) / 512 reaches 1, r being its
  random byte.  The columnwise view is the rowwise one of the transposed matrix.
* Scale bytes [rows, blocks] are held in 512-byte atoms of 128 rows x 4 bytes, the word of row
  128 t + 32 c + l at byte 16 l + 4 c of atom (t, word); padding is zero.
* Random numbers: Philox4x32-10 with the 64-bit seed as key and the counter (group | stream << 30, row,
  offset low, offset high).  Stream 0, dropout: 8 columns a group, 16 bits each.  Streams 1 and 2, rounding
  of the rowwise and of the columnwise view: 16 elements of a view's row a group, 8 bits each.
* Rotary: pair i of a head turns by position * turns[i] / 2^64 of a full turn, an integer product taken
  modulo 2^64.
"""
import math

import numpy as np
import torch

own = False

DEVICE = torch.device("cuda" if torch.cuda.is_available() else "cpu")
BF16, F32 = torch.bfloat16, torch.float32
DTYPES = {"bf16": BF16, "f32": F32}


# --------------------------------------------------------------------------- cases

def listed():
    return [
        # the optimizer step's write of the QKV shard's 4-bit weight: fp32 master, both views
        dict(name="quantize QKV weight", op="quantize", rows=1536, cols=2048, dtype="f32", rounding="nearest"),
        # a ragged last microbatch's gradient of fc1, rounded stochastically, both views
        dict(name="quantize fc1 gradient", op="quantize", rows=8001, cols=8192, dtype="bf16",
             rounding="stochastic"),
        # one token through the fc1 shard: latency and the weight's bytes
        dict(name="forward 1 token", op="forward", M=1, N=8192, K=2048),
        # the layer's largest forward: quantise X, then the product
        dict(name="forward fc1", op="forward", M=8192, N=8192, K=2048),
        # a short packed sequence through the QKV shard's backward, tokens not a multiple of anything
        dict(name="backward QKV ragged", op="backward", M=1111, N=1536, K=2048),
        # the layer's largest backward: quantise dY in both views and X columnwise, dgrad and wgrad accumulate
        dict(name="backward fc1", op="backward", M=8192, N=8192, K=2048),
        # one new token's queries and keys far into a long context
        dict(name="rotary 1 token", op="rotary", tokens=1, groups=4, heads=5, packed=6, head_dim=64, rot_dim=64,
             layout="half", dtype="bf16", inverse=False, start=131000),
        # the QKV shard's packed output of a whole microbatch (4 groups of 4 queries, a key and a value)
        dict(name="rotary QKV", op="rotary", tokens=8192, groups=4, heads=5, packed=6, head_dim=64, rot_dim=64,
             layout="half", dtype="bf16", inverse=False, start=0),
        # the gradient of a long packed batch in fp32, half of each head rotated, neighbours paired
        dict(name="rotary gradient long", op="rotary", tokens=32769, groups=1, heads=20, packed=24, head_dim=128,
             rot_dim=64, layout="interleaved", dtype="f32", inverse=True, start=500000),
        # a few tokens of the projection's output
        dict(name="dropout 37 tokens", op="dropout", rows=37, cols=2048, dtype="bf16", residual="bf16", p=0.1,
             direction="forward"),
        # the projection's output of a whole microbatch onto an fp32 residual stream
        dict(name="dropout fp32 residual", op="dropout", rows=8192, cols=2048, dtype="bf16", residual="f32", p=0.1,
             direction="forward"),
        # the gradient of four microbatches
        dict(name="dropout gradient", op="dropout", rows=32768, cols=2048, dtype="bf16", residual="bf16", p=0.1,
             direction="backward"),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["quantize", "forward", "backward", "rotary", "dropout"])
    if op == "quantize":
        return dict(op=op, rows=_log(rng, 1, 8192), cols=_log(rng, 32, 8192), dtype=rng.choice(["bf16", "f32"]),
                    rounding=rng.choice(["nearest", "stochastic"]))
    if op in ("forward", "backward"):  # output rows are multiples of 16 bytes
        return dict(op=op, M=_log(rng, 1, 8192), N=8 * _log(rng, 16, 1024), K=8 * _log(rng, 16, 256))
    if op == "rotary":
        half = rng.choice([16, 32, 64])
        head_dim = 2 * half * rng.choice([1, 1, 2]) if half < 64 else 128
        heads = rng.randint(1, 8)
        return dict(op=op, tokens=_log(rng, 1, 16384), groups=rng.randint(1, 4), heads=heads,
                    packed=heads + rng.randint(0, 2), head_dim=head_dim, rot_dim=2 * half,
                    layout=rng.choice(["half", "interleaved"]), dtype=rng.choice(["bf16", "f32"]),
                    inverse=rng.choice([False, True]), start=rng.randint(0, 1000000))
    dtype = rng.choice(["bf16", "f32"])
    return dict(op=op, rows=_log(rng, 1, 16384), cols=_log(rng, 16, 4096), dtype=dtype,
                residual="f32" if dtype == "f32" else rng.choice(["bf16", "f32"]),
                p=rng.choice([0.05, 0.1, 0.25, 0.5]), direction=rng.choice(["forward", "backward"]))


def work(case):
    op = case["op"]
    size = {"bf16": 2, "f32": 4}
    if op == "quantize":  # the source once, both views' values (bf16) out
        n = case["rows"] * case["cols"]
        return {"bytes": n * (size[case["dtype"]] + 4), "flops": 0}
    if op in ("forward", "backward"):
        M, N, K = case["M"], case["N"], case["K"]
        four = 17 / 32
        if op == "forward":  # X in bf16, W in 4 bits, Y in bf16
            return {"bytes": 2 * M * K + four * N * K + 2 * M * N, "flops": 2 * M * N * K}
        # dY and X in bf16, W's columnwise view in 4 bits, dX in bf16, main_grad read and written
        return {"bytes": 2 * M * N + four * N * K + 4 * M * K + 8 * N * K, "flops": 4 * M * N * K}
    if op == "rotary":
        n = case["tokens"] * case["groups"] * case["heads"] * case["head_dim"]
        return {"bytes": 2 * n * size[case["dtype"]] + 4 * case["tokens"], "flops": 0}
    n = case["rows"] * case["cols"]
    if case["direction"] == "backward":
        return {"bytes": 2 * n * size[case["dtype"]], "flops": 0}
    return {"bytes": n * (size[case["dtype"]] + 2 * size[case["residual"]]), "flops": 0}


# --------------------------------------------------------------------------- inputs

def _randn(shape, std, dtype, g):
    return (torch.randn(shape, generator=g, device=DEVICE, dtype=F32) * std).to(dtype)


def _blocks(n):
    return (n + 31) // 32


def _view_buffers(rows, cols):
    """Packed codes and tiled scales of the rowwise view of a [rows, cols] matrix."""
    tiles, words = (rows + 127) // 128, (_blocks(cols) + 3) // 4
    return (torch.empty(rows, 16 * _blocks(cols), dtype=torch.uint8, device=DEVICE),
            torch.empty(tiles * words * 512, dtype=torch.uint8, device=DEVICE))


def _pack(x):
    """x's rowwise MXFP4 view (rounded to nearest) as a user's program keeps a weight: codes and scales."""
    rows, cols = x.shape
    code, byte = _quantize(x.float(), None, None)
    packed = (code[:, 0::2] | (code[:, 1::2] << 4)).to(torch.uint8)
    tiles, words = (rows + 127) // 128, (byte.shape[1] + 3) // 4
    full = torch.zeros(tiles * 128, words * 4, dtype=torch.uint8, device=x.device)
    full[:rows, :byte.shape[1]] = byte.to(torch.uint8)
    tiled = full.view(tiles, 4, 32, words, 4).permute(0, 3, 2, 1, 4).reshape(-1)
    return packed.contiguous(), tiled.contiguous()


def _heavy(shape, std, dtype, g):
    """A gradient: most of it small, every token with a size of its own."""
    size = torch.exp(torch.randn(shape[0], 1, generator=g, device=DEVICE))
    return (torch.randn(shape, generator=g, device=DEVICE, dtype=F32) * (std * size)).to(dtype)


def _turns(rot_dim, base=500000.0, factor=32.0, low=1.0, high=4.0, context=8192):
    """Turns per position of each pair, as 64-bit fractions: frequencies base^(-2 i / rot_dim), the slow ones
    stretched by `factor` and those between `low` and `high` turns per trained context blended."""
    out = []
    for i in range(rot_dim // 2):
        f = base ** (-2.0 * i / rot_dim)
        turns = context * f / (2 * math.pi)
        blend = min(1.0, max(0.0, (turns - low) / (high - low)))
        f = (1 - blend) * f / factor + blend * f
        out.append(int(round(f / (2 * math.pi) * 2.0 ** 64)))
    return out


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    op = case["op"]
    s = {"case": dict(case), "rng": (0x9E3779B97F4A7C15 * (seed + 1) % 2 ** 64, 1000 + seed)}
    if op == "quantize":
        rows, cols = case["rows"], case["cols"]
        if case["rounding"] == "nearest":
            s["src"] = _randn((rows, cols), 0.02, DTYPES[case["dtype"]], g)
        else:
            s["src"] = _heavy((rows, cols), 1e-3, DTYPES[case["dtype"]], g)
        s["row"], s["col"] = _view_buffers(rows, cols), _view_buffers(cols, rows)
        s["out"] = (torch.empty(rows, cols, dtype=BF16, device=DEVICE),
                    torch.empty(cols, rows, dtype=BF16, device=DEVICE))
    elif op == "forward":
        M, N, K = case["M"], case["N"], case["K"]
        s["X"] = _randn((M, K), 1.0, BF16, g)
        s["W"] = _pack(_randn((N, K), 0.02, F32, g))
        s["row"] = _view_buffers(M, K)
        s["Y"] = torch.empty(M, N, dtype=BF16, device=DEVICE)
    elif op == "backward":
        M, N, K = case["M"], case["N"], case["K"]
        s["dY"] = _heavy((M, N), 1e-3, BF16, g)
        s["Wt"] = _pack(_randn((K, N), 0.02, F32, g))
        s["X"] = _randn((M, K), 1.0, BF16, g)
        s["row"], s["col"], s["X col"] = _view_buffers(M, N), _view_buffers(N, M), _view_buffers(K, M)
        s["dX"] = torch.empty(M, K, dtype=BF16, device=DEVICE)
        s["main_grad"] = _randn((N * K,), 1e-3, F32, g)
    elif op == "rotary":
        T, G, H, P, D = (case[k] for k in ("tokens", "groups", "heads", "packed", "head_dim"))
        dtype = DTYPES[case["dtype"]]
        s["src"] = _randn((T, G, P, D), 1.0, dtype, g)[:, :, :H]
        s["dst"] = torch.empty(T, G, H, D, dtype=dtype, device=DEVICE)
        # packed sequences: positions count up and start again
        length = max(1, T // 3 + 1)
        s["positions"] = (case["start"] + torch.arange(T, device=DEVICE) % length).to(torch.int32)
        s["turns"] = _turns(case["rot_dim"])
    else:
        rows, cols = case["rows"], case["cols"]
        s["x"] = _randn((rows, cols), 1.0, DTYPES[case["dtype"]], g)
        if case["direction"] == "forward":
            s["residual"] = _randn((rows, cols), 1.0, DTYPES[case["residual"]], g)
            s["out"] = torch.empty_like(s["residual"])
        else:
            s["out"] = torch.empty_like(s["x"])
    return s


# --------------------------------------------------------------------------- plain forms

def _philox(seed, c0, c1, offset):
    """Philox4x32-10 words (int64 tensors holding 32-bit values) of counters (c0, c1, offset) under `seed`."""
    low = 0xFFFFFFFF

    def product(m, c):  # high and low 32 bits of m * c, in 16-bit halves so that no product passes 63 bits
        a, b = m * (c & 0xFFFF), m * (c >> 16)
        b = b + (a >> 16)
        return (b >> 16) & low, ((b << 16) | (a & 0xFFFF)) & low

    c0, c1 = torch.broadcast_tensors(c0, c1)
    c2, c3 = torch.full_like(c0, offset & low), torch.full_like(c0, offset >> 32)
    k0, k1 = seed & low, seed >> 32
    for _ in range(10):
        h0, l0 = product(0xD2511F53, c0)
        h1, l1 = product(0xCD9E8D57, c2)
        c0, c1, c2, c3 = h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    return c0, c1, c2, c3


def _draws(rng, rows, cols, bits, stream):
    """[rows, cols] random integers of `bits` bits (int32), 128 / bits columns to a generator call."""
    per = 128 // bits
    groups = torch.arange((cols + per - 1) // per, device=DEVICE) | (stream << 30)
    words = torch.stack(_philox(rng[0], groups[None, :], torch.arange(rows, device=DEVICE)[:, None], rng[1]), -1)
    shifts = torch.arange(0, 32, bits, device=DEVICE)
    return ((words[..., None] >> shifts) & ((1 << bits) - 1)).to(torch.int32).reshape(rows, -1)[:, :cols]


def _quantize(x, rng, stream):
    """E2M1 codes [rows, 32 blocks] and E8M0 bytes [rows, blocks] of fp32 x; rng None rounds to nearest."""
    rows, cols = x.shape
    x = torch.nn.functional.pad(x, (0, 32 * _blocks(cols) - cols)).view(rows, -1, 32)
    amax = x.abs().amax(-1, keepdim=True)
    bits = amax.view(torch.int32)
    byte = (bits >> 23) - 2
    if rng is not None:
        byte = byte + ((bits & 0x7FFFFF) > 0x400000)
    byte = byte.clamp(min=0)
    y = x.abs() * ((254 - byte) << 23).view(F32)
    if rng is None:
        code = (y > 0.25).int() + (y >= 0.75) + (y > 1.25) + (y >= 1.75) + (y > 2.5) + (y >= 3.5) + (y > 5)
    else:
        r = _draws(rng, rows, x.shape[1] * 32, 8, stream).view_as(x)
        y = torch.where(y < 1, (y * 2.0 ** 23).round() * 2.0 ** -23, y)
        step = torch.where(y < 2, 0.5, torch.where(y < 4, 1.0, 2.0))
        low = (y / step).floor()
        up = (y / step - low) + (2 * r + 1) / 512 >= 1
        code = (low + torch.where(y < 2, 0.0, torch.where(y < 4, 2.0, 4.0))).int() + up
    bad = ~torch.isfinite(amax)
    code = torch.where(bad, 0, code + 8 * torch.signbit(x))
    return code.reshape(rows, -1), torch.where(bad, 255, byte)[..., 0]


def _values(code, byte):
    """fp32 values of codes [rows, 32 blocks] under scale bytes [rows, blocks]."""
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0] + [-0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0],
                         device=code.device)
    v = table[code.long()].view(code.shape[0], -1, 32)
    scale = torch.where(byte == 255, torch.nan, torch.exp2((byte - 127).float()))
    return (v * scale[..., None]).reshape(code.shape[0], -1)


def _unpack(view, rows, cols):
    """fp32 values [rows, cols] of a packed view (codes, tiled scales)."""
    packed, tiled = view
    code = torch.stack((packed & 15, packed >> 4), -1).reshape(rows, -1)
    words = (_blocks(cols) + 3) // 4
    byte = tiled.view(-1, words, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(-1, words * 4)[:rows, :_blocks(cols)]
    return _values(code, byte.int())[:, :cols]


def _quantized(x, rng, stream):
    """fp32 values of x's rowwise view."""
    return _values(*_quantize(x, rng, stream))[:, :x.shape[1]]


def _rotate(s):
    case, x = s["case"], s["src"].float()
    half = case["rot_dim"] // 2
    turns = torch.tensor(s["turns"], device=x.device)
    turn = s["positions"].long()[:, None] * turns[None, :]  # modulo 2^64
    angle = (turn >> 32).float() * (2 * math.pi * 2.0 ** -32)
    cos, sin = angle.cos()[:, None, None], angle.sin()[:, None, None]
    if case["inverse"]:
        sin = -sin
    if case["layout"] == "half":
        a, b = x[..., :half], x[..., half:2 * half]
    else:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
    c, d = a * cos - b * sin, a * sin + b * cos
    turned = torch.cat((c, d), -1) if case["layout"] == "half" else torch.stack((c, d), -1).flatten(-2)
    return torch.cat((turned, x[..., 2 * half:]), -1).to(s["src"].dtype)


def _dropped(s):
    case, x = s["case"], s["x"]
    threshold = int(round(case["p"] * 65536))
    keep = _draws(s["rng"], case["rows"], case["cols"], 16, 0) >= threshold
    kept = torch.where(keep, x.float() * (65536 / (65536 - threshold)), 0.0)
    if case["direction"] == "backward":
        return kept.to(x.dtype)
    return (s["residual"].float() + kept).to(s["residual"].dtype)


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    if op == "quantize":
        rng = s["rng"] if case["rounding"] == "stochastic" else None
        x = s["src"].float()
        return {"row": _quantized(x, rng, 1).to(BF16), "col": _quantized(x.t().contiguous(), rng, 2).to(BF16)}
    if op == "forward":
        return {"Y": (_quantized(s["X"].float(), None, 1) @ _unpack(s["W"], case["N"], case["K"]).t()).to(BF16)}
    if op == "backward":
        M, N, K = case["M"], case["N"], case["K"]
        dy = s["dY"].float()
        dx = _quantized(dy, s["rng"], 1) @ _unpack(s["Wt"], K, N).t()
        dw = _quantized(dy.t().contiguous(), s["rng"], 2) @ _quantized(s["X"].float().t().contiguous(), None, 2).t()
        s["main_grad"].view(N, K).add_(dw)
        return {"dX": dx.to(BF16), "main_grad": s["main_grad"]}
    return _rotate(s) if op == "rotary" else _dropped(s)


# --------------------------------------------------------------------------- the framework's calls

def _run_own(s):
    import param_buffers_gb300 as gtp
    case = s["case"]
    op = case["op"]
    if op == "quantize":
        rng = s["rng"] if case["rounding"] == "stochastic" else None
        gtp.gtp_mxfp4_quantize(s["src"], row=s["row"], col=s["col"], rng=rng)
        gtp.gtp_mxfp4_dequantize(*s["row"], s["out"][0])
        gtp.gtp_mxfp4_dequantize(*s["col"], s["out"][1])
        return {"row": s["out"][0], "col": s["out"][1]}
    if op == "forward":
        gtp.gtp_mxfp4_quantize(s["X"], row=s["row"])
        gtp.gtp_linear_fprop_mxfp4(*s["row"], *s["W"], s["Y"])
        return {"Y": s["Y"]}
    if op == "backward":
        gtp.gtp_mxfp4_quantize(s["dY"], row=s["row"], col=s["col"], rng=s["rng"])
        gtp.gtp_mxfp4_quantize(s["X"], col=s["X col"])
        gtp.gtp_linear_dgrad_mxfp4(*s["row"], *s["Wt"], s["dX"])
        gtp.gtp_linear_wgrad_accum_mxfp4(*s["col"], *s["X col"], s["main_grad"], 0)
        return {"dX": s["dX"], "main_grad": s["main_grad"]}
    if op == "rotary":
        gtp.gtp_rotary(s["src"], s["dst"], s["turns"], positions=s["positions"], layout=case["layout"],
                       inverse=case["inverse"])
        return s["dst"]
    if case["direction"] == "backward":
        gtp.gtp_dropout_grad(s["x"], s["out"], case["p"], s["rng"])
    else:
        gtp.gtp_dropout_add(s["x"], s["residual"], s["out"], case["p"], s["rng"])
    return s["out"]


def run(state):
    return _run_own(state) if own else _run_plain(state)


# --------------------------------------------------------------------------- 64 bits

_GRID = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _exact_bytes(rng, rows, cols, stream):
    """[rows, 16 groups] generator bytes, by unsigned 64-bit products on the host."""
    groups = (cols + 127) // 128 * 8 if stream == 0 else (cols + 15) // 16
    c = [np.broadcast_to(np.arange(groups, dtype=np.uint64)[None, :] | np.uint64(stream << 30), (rows, groups)),
         np.broadcast_to(np.arange(rows, dtype=np.uint64)[:, None], (rows, groups)),
         np.full((rows, groups), rng[1] % 2 ** 32, np.uint64), np.full((rows, groups), rng[1] // 2 ** 32, np.uint64)]
    key = [rng[0] % 2 ** 32, rng[0] // 2 ** 32]
    s32, low = np.uint64(32), np.uint64(2 ** 32 - 1)
    for n in range(10):
        p, q = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        k = [np.uint64((key[0] + n * 0x9E3779B9) % 2 ** 32), np.uint64((key[1] + n * 0xBB67AE85) % 2 ** 32)]
        c = [(q >> s32) ^ c[1] ^ k[0], q & low, (p >> s32) ^ c[3] ^ k[1], p & low]
    words = np.stack([v.astype("<u4") for v in c], -1)
    return torch.from_numpy(words.view(np.uint8).reshape(rows, groups * 16)).to(DEVICE)


def _exact_view(x, rng, stream):
    """The rowwise view's values of a float64 matrix, row by block, from the distance to the grid's points."""
    rows, cols = x.shape
    width = 32 * _blocks(cols)
    x = torch.nn.functional.pad(x, (0, width - cols)).view(rows, -1, 32)
    amax = x.abs().max(-1, keepdim=True).values
    mantissa, exponent = torch.frexp(amax)  # amax = mantissa * 2^exponent, mantissa in [0.5, 1)
    e = exponent - 3
    if rng is not None:
        e = e + (mantissa > 0.75).int()
    e = torch.where(amax == 0, -127, e).clamp(min=-127)
    y = torch.ldexp(x.abs(), -e)
    grid = torch.tensor(_GRID, dtype=torch.float64, device=x.device)
    if rng is None:
        middle = (grid[1:] + grid[:-1]) / 2
        below = torch.searchsorted(middle, y)  # the middles less than y
        tie = y == middle[below.clamp(max=6)]  # on a middle: the point whose index is even
        index = torch.where(tie & (below < 7) & (below % 2 == 1), below + 1, below)
    else:
        y = torch.where(y < 1, torch.ldexp(torch.round(torch.ldexp(y, torch.tensor(23))), torch.tensor(-23)), y)
        index = (torch.searchsorted(grid, y, right=True) - 1).clamp(0, 7)
        above = grid[(index + 1).clamp(max=7)]
        span = torch.where(index < 7, above - grid[index], 2.0)
        r = _exact_bytes(rng, rows, width, stream)[:, :width].view(x.shape).double()
        index = index + ((y - grid[index]) / span + (r + 0.5) / 256 >= 1)
    v = torch.ldexp(grid[index.clamp(max=7)], e) * torch.where(x < 0, -1.0, 1.0)
    return v.reshape(rows, width)[:, :cols]


def _exact_stored(view, rows, cols):
    """Values of a packed view, byte by byte from the layout's formula."""
    packed, tiled = view
    r = torch.arange(rows, device=DEVICE)[:, None]
    b = torch.arange(_blocks(cols), device=DEVICE)[None, :]
    words = (_blocks(cols) + 3) // 4
    at = ((r // 128) * words + b // 4) * 512 + (r % 32) * 16 + (r // 32 % 4) * 4 + b % 4
    e = tiled[at].int() - 127
    k = torch.arange(cols, device=DEVICE)
    code = (packed[:, k // 2].int() >> (4 * (k % 2)).int()) & 15
    v = torch.tensor(_GRID, dtype=torch.float64, device=DEVICE)[(code & 7).long()] * (1.0 - 2.0 * (code >> 3))
    return torch.ldexp(v, e.repeat_interleave(32, 1)[:, :cols])


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        rng = s["rng"] if case["rounding"] == "stochastic" else None
        x = s["src"].double()
        return {"row": _exact_view(x, rng, 1), "col": _exact_view(x.t().contiguous(), rng, 2)}
    if op == "forward":
        return {"Y": _exact_view(s["X"].double(), None, 1) @ _exact_stored(s["W"], case["N"], case["K"]).t()}
    if op == "backward":
        M, N, K = case["M"], case["N"], case["K"]
        dy, x = s["dY"].double(), s["X"].double()
        dx = _exact_view(dy, s["rng"], 1) @ _exact_stored(s["Wt"], K, N).t()
        dw = _exact_view(dy.t().contiguous(), s["rng"], 2) @ _exact_view(x.t().contiguous(), None, 2).t()
        return {"dX": dx, "main_grad": s["main_grad"].double() + dw.reshape(-1)}
    if op == "rotary":
        rot = case["rot_dim"]
        # whole turns drop out in Python's integers; what is left is below one turn
        spot = s["positions"].tolist()
        angle = np.array([[(p * f) % 2 ** 64 / 2.0 ** 64 for f in s["turns"]] for p in sorted(set(spot))])
        where = {p: i for i, p in enumerate(sorted(set(spot)))}
        angle = torch.from_numpy(angle[[where[p] for p in spot]] * (2 * math.pi)).to(DEVICE)
        z = torch.polar(torch.ones_like(angle), -angle if case["inverse"] else angle)[:, None, None]
        x = s["src"].double()
        if case["layout"] == "half":
            w = torch.complex(x[..., :rot // 2], x[..., rot // 2:rot].contiguous()) * z
            return torch.cat((w.real, w.imag, x[..., rot:]), -1)
        w = torch.view_as_complex(x[..., :rot].reshape(*x.shape[:3], rot // 2, 2)) * z
        return torch.cat((torch.view_as_real(w).flatten(-2), x[..., rot:]), -1)
    rows, cols = case["rows"], case["cols"]
    b = _exact_bytes(s["rng"], rows, 16 * cols, 0)[:, :2 * cols].view(rows, cols, 2).int()
    cut = int(round(case["p"] * 65536))
    kept = s["x"].double() * ((b[..., 0] + 256 * b[..., 1]) >= cut) / (1 - cut / 65536)
    return kept if case["direction"] == "backward" else s["residual"].double() + kept
