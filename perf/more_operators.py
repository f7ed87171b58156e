"""Measured cases of the operators between a layer's products: the gated activation with its inputs kept as 8-bit
codes, its backward pass from those codes, the restoring of coded matrices, and the norm of queries and keys for each
head with the position rotation, forward and backward.

``listed()`` and ``draw()`` give the cases, ``prepare()`` the tensors a program holds before the call, and
``run()`` one pass: with ``own`` false in elementary torch operations, with ``own`` true by the library's
entry points.  ``exact()`` gives the same outputs from the definitions in 64 bits, and ``work()`` the bytes
and operations a pass cannot do without.

A block-coded matrix is a pair (codes, scales): E4M3 codes [rows, cols rounded up to 16] with zero codes past
the last column, and one power-of-two scale X = 2^(byte - 127) for each row and each 128 columns, stored
[ceil(cols / 128), rows rounded up to 4].  X is the smallest power of two with absmax <= 448 X.
"""
import math

import torch

own = False

BLOCK = 128
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
DEVICE = "cuda"
EPS = 1e-6
GELU_SCALE, GELU_CUBE = 2 * math.sqrt(2 / math.pi), 0.044715     # s(x) = x sigmoid(scale (x + cube x^3))
TABLE_ROWS = 65536


def up(n, m):
    return (n + m - 1) // m * m


# ---------------------------------------------------------------------------------------------------------
# the cases


def listed():
    return [
        # serving or the last token of a batch: one row to codes for the product that follows; latency
        dict(name="gate-token", op="gate", rows=1, cols=11008, dtype="bf16", act="silu", out="codes", keep=False, halves=True),
        # a training pass: 8192 tokens to codes, both inputs kept as codes for the backward pass
        dict(name="gate-tokens", op="gate", rows=8192, cols=11008, dtype="bf16", act="silu", out="codes", keep=True, halves=True),
        # a result in 32 bits from two matrices, odd sizes, the other activation
        dict(name="gate-odd", op="gate", rows=1023, cols=4099, dtype="f32", act="gelu", out="y", keep=False, halves=False),
        # the backward pass of the training pass, from the codes: gradients in both layouts, the activation again, transposed
        dict(name="gate-gradient", op="gate_grad", rows=8192, cols=11008, dtype="bf16", act="silu", source="codes", out="codes",
             halves=True),
        # the backward pass of inputs kept in 16 bits, gradients in 16 bits, an odd number of rows
        dict(name="gate-gradient-matrix", op="gate_grad", rows=2047, cols=4096, dtype="f16", act="gelu", source="matrix", out="matrix",
             halves=True),
        # a product's own input, restored as the transposed codes of the weight gradient
        dict(name="restore-transposed", op="restore", rows=8192, cols=4096, dtype="bf16", out="codes"),
        # a short odd checkpoint back to 16 bits
        dict(name="restore-odd", op="restore", rows=517, cols=4099, dtype="bf16", out="matrix"),
        # serving: one token far into its sequence
        dict(name="heads-token", op="heads", tokens=1, heads=32, kv=8, dim=128, rot=128, dtype="bf16", pairs="halves", keep=False,
             layout="token"),
        # a training pass over packed sequences, the raw heads kept as codes
        dict(name="heads-tokens", op="heads", tokens=8192, heads=32, kv=8, dim=128, rot=128, dtype="bf16", pairs="halves", keep=True,
             layout="token"),
        # short heads, part of each rotated, neighbouring pairs, heads outermost in the results
        dict(name="heads-odd", op="heads", tokens=1537, heads=12, kv=3, dim=80, rot=32, dtype="f16", pairs="neighbours", keep=False,
             layout="head"),
        # the backward pass from the codes, with the gradients of both weights
        dict(name="heads-gradient", op="heads_grad", tokens=8192, heads=32, kv=8, dim=128, rot=128, dtype="bf16", pairs="halves",
             source="codes", layout="token"),
        # the backward pass in 32 bits from the matrix, wide heads
        dict(name="heads-gradient-odd", op="heads_grad", tokens=1001, heads=7, kv=7, dim=192, rot=64, dtype="f32", pairs="halves",
             source="matrix", layout="head"),
    ]


def spread(rng, lo, hi, odd=0.5):
    """A size over the logarithm of [lo, hi]; half of them as they fall, the others a multiple of 16."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return v if rng.random() < odd else min(hi, max(lo, up(v, 16)))


def drawn(rng):
    op = rng.choice(["gate", "gate", "gate_grad", "gate_grad", "restore", "heads", "heads", "heads_grad"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op in ("heads", "heads_grad"):
        heads = rng.choice([1, 2, 4, 7, 8, 12, 16, 32, 40, 64])
        dim = rng.choice([32, 64, 72, 80, 96, 100, 128, 128, 192, 256])
        case = dict(op=op, tokens=spread(rng, 1, 32768), heads=heads, kv=rng.choice([0, 1, 2, 4, 8, heads]), dim=dim,
                    rot=rng.choice([dim, dim, dim // 2 // 2 * 2, 16, 20, 0]), dtype=dtype,
                    pairs=rng.choice(["halves", "halves", "neighbours"]), layout=rng.choice(["token", "head"]))
        if op == "heads":
            return dict(case, keep=rng.random() < 0.5)
        return dict(case, source=rng.choice(["codes", "matrix"]))
    case = dict(op=op, rows=spread(rng, 1, 32768), cols=spread(rng, 64, 16384), dtype=dtype)
    if op == "restore":
        return dict(case, out=rng.choice(["codes", "matrix", "both"]))
    case = dict(case, act=rng.choice(["silu", "silu", "gelu"]), halves=rng.random() < 0.6)
    if op == "gate":
        return dict(case, out=rng.choice(["codes", "y", "both"]), keep=rng.random() < 0.5)
    return dict(case, source=rng.choice(["codes", "matrix"]), out=rng.choice(["codes", "codes", "matrix"]))


def draw(rng):
    case = drawn(rng)
    most, side = max(work(c)["bytes"] for c in listed()), "tokens" if "tokens" in case else "rows"
    while work(case)["bytes"] > most:
        case[side] = max(1, case[side] // 2)
    return case


# ---------------------------------------------------------------------------------------------------------
# inputs


def coded_buffers(rows, cols):
    return (torch.zeros(rows, up(cols, 16), dtype=torch.uint8, device=DEVICE),
            torch.zeros(up(cols, BLOCK) // BLOCK, up(rows, 4), dtype=torch.uint8, device=DEVICE))


def two_buffers(rows, cols, down):
    """Buffers of two coded matrices of one size; where the blocks allow it the halves of one matrix, side by side or (down) one
    below the other, as one product reads them."""
    if down and cols and rows % 4 == 0:
        q, s = coded_buffers(2 * rows, cols)
        return (q[:rows], s[:, :rows]), (q[rows:], s[:, rows:2 * rows])
    if not down and cols % BLOCK == 0:
        q, s = coded_buffers(rows, 2 * cols)
        n = cols // BLOCK
        return (q[:, :cols], s[:n]), (q[:, cols:], s[n:])
    return coded_buffers(rows, cols), coded_buffers(rows, cols)


def coded(x):
    """A block-coded copy of a matrix, as a program has it from the forward pass."""
    rows, cols = x.shape
    q, e = encode(x.float())
    buf = coded_buffers(rows, cols)
    buf[0][:, :cols] = q.view(torch.uint8)
    buf[1][:, :rows] = e.to(torch.uint8)
    return buf


def values(pair, rows, cols):
    """What a pair's bytes stand for: E4M3 values and power-of-two scales."""
    q, s = pair
    return {"codes": q[:, :cols].view(torch.float8_e4m3fn), "scales": s[:, :rows].view(torch.float8_e8m0fnu)}


def normal(g, shape, dtype, std=1.0):
    return (torch.randn(*shape, generator=g, device=DEVICE) * std).to(DTYPES[dtype])


def projected(g, rows, cols, dtype):
    """Results of a layer's product: rows of different sizes and a few loud channels."""
    loud = 1 + 3 * (torch.rand(cols, generator=g, device=DEVICE) < 0.02).float()
    size = 0.5 + torch.rand(rows, 1, generator=g, device=DEVICE)
    return (torch.randn(rows, cols, generator=g, device=DEVICE) * loud * size).to(DTYPES[dtype])


def table(rot):
    """cos and sin of every position's angles, formed in 64 bits."""
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEVICE) / rot)
    a = torch.arange(TABLE_ROWS, dtype=torch.float64, device=DEVICE)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float()


def prepare_heads(case, g, s):
    t, n, kv, dim = case["tokens"], case["heads"], case["kv"], case["dim"]
    # the product's result [tokens, queries | keys | values], of which the heads are views
    wide = projected(g, t, (n + 2 * kv) * dim, case["dtype"])
    s["q"] = wide[:, :n * dim].view(t, n, dim)
    s["k"] = wide[:, n * dim:(n + kv) * dim].view(t, kv, dim) if kv else None
    s["wq"] = 1 + normal(g, (dim,), case["dtype"], 0.2)
    s["wk"] = 1 + normal(g, (dim,), case["dtype"], 0.2) if kv else None
    s["table"] = table(case["rot"]) if case["rot"] else None
    # packed sequences: each starts somewhere and runs on; one token is far into its own
    run = max(1, t // 4 + 1)
    start = torch.randint(0, TABLE_ROWS - run + 1, (4,), generator=g, device=DEVICE)
    at = torch.arange(t, device=DEVICE)
    s["pos"] = start[at // run] + at % run

    def heads_like(h):
        if case["layout"] == "head":
            return torch.empty(h, t, dim, dtype=DTYPES[case["dtype"]], device=DEVICE).transpose(0, 1)
        return torch.empty(t, h, dim, dtype=DTYPES[case["dtype"]], device=DEVICE)

    sides = [("q", n)] + ([("k", kv)] if kv else [])
    for name, h in sides:
        if case["op"] == "heads":
            s[name + "_out"] = heads_like(h)
            s[name + "_codes"] = coded_buffers(t * h, dim) if case["keep"] else None
            s[name + "_values"] = values(s[name + "_codes"], t * h, dim) if case["keep"] else None
        else:
            s["d" + name + "_out"] = heads_like(h).copy_(normal(g, (t, h, dim), case["dtype"], 0.01))
            s["dw" + name] = torch.empty(dim, dtype=torch.float32, device=DEVICE)
            if case["source"] == "codes":
                s[name + "_codes"] = coded(s[name].reshape(t * h, dim))
    if case["op"] == "heads_grad":
        wide = torch.empty_like(wide)
        s["dq"] = wide[:, :n * dim].view(t, n, dim)
        s["dk"] = wide[:, n * dim:(n + kv) * dim].view(t, kv, dim) if kv else None
    return s


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    s = dict(case)
    if case["op"] in ("heads", "heads_grad"):
        return prepare_heads(case, g, s)
    rows, cols, dt = case["rows"], case["cols"], DTYPES[case["dtype"]]
    if case["op"] == "restore":
        s["q"] = coded(projected(g, rows, cols, case["dtype"]))
        s["x"] = torch.empty(rows, cols, dtype=dt, device=DEVICE) if case["out"] != "codes" else None
        s["qt"] = coded_buffers(cols, rows) if case["out"] != "matrix" else None
        s["qt_values"] = values(s["qt"], cols, rows) if s["qt"] else None
        return s
    if case["halves"]:      # one product's result holds both
        z = projected(g, rows, 2 * cols, case["dtype"])
        s["gate"], s["up"] = z[:, :cols], z[:, cols:]
    else:
        s["gate"], s["up"] = projected(g, rows, cols, case["dtype"]), projected(g, rows, cols, case["dtype"])
    if case["op"] == "gate":
        s["y"] = torch.empty(rows, cols, dtype=dt, device=DEVICE) if case["out"] != "codes" else None
        for name, there in (("q", case["out"] != "y"), ("gate_q", case["keep"]), ("up_q", case["keep"])):
            s[name] = coded_buffers(rows, cols) if there else None
            s[name + "_values"] = values(s[name], rows, cols) if there else None
        return s
    s["dy"] = normal(g, (rows, cols), case["dtype"], 0.01)
    if case["source"] == "codes":
        s["gate_q"], s["up_q"] = coded(s["gate"]), coded(s["up"])
        del s["gate"], s["up"]
    if case["out"] == "matrix":
        if case["halves"]:
            dz = torch.empty(rows, 2 * cols, dtype=dt, device=DEVICE)
            s["dgate"], s["dup"] = dz[:, :cols], dz[:, cols:]
        else:
            s["dgate"], s["dup"] = (torch.empty(rows, cols, dtype=dt, device=DEVICE) for _ in range(2))
        return s
    if case["halves"]:
        (s["dgate_q"], s["dup_q"]), (s["dgate_t"], s["dup_t"]) = two_buffers(rows, cols, False), two_buffers(cols, rows, True)
    else:
        s["dgate_q"], s["dup_q"], s["dgate_t"], s["dup_t"] = (coded_buffers(*v) for v in ((rows, cols),) * 2 + ((cols, rows),) * 2)
    s["y_t"] = coded_buffers(cols, rows)
    s["all_values"] = {k: values(s[k], rows, cols) for k in ("dgate_q", "dup_q")}
    s["all_values"].update({k: values(s[k], cols, rows) for k in ("dgate_t", "dup_t", "y_t")})
    return s


# ---------------------------------------------------------------------------------------------------------
# the plain form


def power(e):
    """2^e as binary32, -127 <= e <= 127."""
    return torch.where(e < -126, torch.full_like(e, 0x00400000), (e + 127) << 23).to(torch.int32).view(torch.float32)


def encode(x):
    """(E4M3 values, scale bytes) of fp32 x, a scale for each row and 128 columns."""
    rows, cols = x.shape
    a = torch.nn.functional.pad(x.abs(), (0, -cols % BLOCK)).view(rows, -1, BLOCK).amax(2).t()
    m, e = torch.frexp(a)                                          # a = m 2^e with m in [0.5, 1)
    e = torch.where(a > 0, e.long() - 9 + (m > 0.875), -127).clamp(min=-127)   # 448 = 0.875 * 2^9
    shift = power(-e).t().repeat_interleave(BLOCK, 1)[:, :cols]
    return (x * shift).to(torch.float8_e4m3fn), e + 127


def encoded(x):
    q, e = encode(x)
    return {"codes": q, "scales": e.to(torch.uint8).view(torch.float8_e8m0fnu)}


def decode(pair, rows, cols):
    q, s = pair
    scale = power(s[:, :rows].long() - 127).t().repeat_interleave(BLOCK, 1)[:, :cols]
    return q[:, :cols].view(torch.float8_e4m3fn).to(torch.float32) * scale


def activation(x, act, slope=False):
    """s(x) = x sigmoid(p(x)), and its derivative."""
    if act == "silu":
        h = torch.sigmoid(x)
        return (x * h, h * (1 + x * torch.sigmoid(-x))) if slope else x * h
    p = GELU_SCALE * (x + GELU_CUBE * x * x * x)
    h = torch.sigmoid(p)
    if not slope:
        return x * h
    return x * h, h * (1 + x * torch.sigmoid(-p) * (GELU_SCALE * (1 + 3 * GELU_CUBE * x * x)))


def root(x):
    """1 / sqrt(mean x^2 + eps) of each head, the sum in 64 bits, as binary32."""
    return (1 / torch.sqrt(x.double().square().mean(-1, keepdim=True) + EPS)).float()


def rotated(x, s, back=False):
    """The first rot columns of heads [tokens, heads, dim] turned by their positions' angles, or back by them."""
    rot = s["rot"]
    if not rot:
        return x
    row = s["table"][s["pos"]][:, None, :]
    c, d = row[..., :rot // 2], row[..., rot // 2:]
    d = -d if back else d
    a, b = (x[..., :rot // 2], x[..., rot // 2:rot]) if s["pairs"] == "halves" else (x[..., 0:rot:2], x[..., 1:rot:2])
    u, v = a * c - b * d, b * c + a * d
    turned = torch.cat([u, v], -1) if s["pairs"] == "halves" else torch.stack([u, v], -1).flatten(-2)
    return torch.cat([turned, x[..., rot:]], -1)


def run(state):
    s = state
    op = s["op"]
    if own:
        return run_own(s)
    dt = DTYPES[s["dtype"]]
    if op == "gate":
        gate, upper = s["gate"].float(), s["up"].float()
        y = activation(gate, s["act"]) * upper
        out = {}
        if s["y"] is not None:
            out["y"] = y.to(dt)
        if s["q"] is not None:
            out["q"] = encoded(y)
        if s["keep"]:
            out["gate_q"], out["up_q"] = encoded(gate), encoded(upper)
        return out
    if op == "gate_grad":
        if s["source"] == "codes":
            gate, upper = decode(s["gate_q"], s["rows"], s["cols"]), decode(s["up_q"], s["rows"], s["cols"])
        else:
            gate, upper = s["gate"].float(), s["up"].float()
        dy = s["dy"].float()
        y, slope = activation(gate, s["act"], True)
        dgate, dup, y = dy * upper * slope, dy * y, y * upper
        if s["out"] == "matrix":
            return {"dgate": dgate.to(dt), "dup": dup.to(dt)}
        return {"dgate_q": encoded(dgate), "dup_q": encoded(dup), "dgate_t": encoded(dgate.t().contiguous()),
                "dup_t": encoded(dup.t().contiguous()), "y_t": encoded(y.t().contiguous())}
    if op == "restore":
        x = decode(s["q"], s["rows"], s["cols"])
        out = {}
        if s["x"] is not None:
            out["x"] = x.to(dt)
        if s["qt"] is not None:
            out["qt"] = encoded(x.t().contiguous())
        return out
    out = {}
    for name in ("q", "k") if s["kv"] else ("q",):
        x, w = s[name].float(), s["w" + name].float()
        t, h, dim = x.shape
        if op == "heads":
            out[name] = rotated(x * root(x) * w, s).to(dt)
            if s["keep"]:
                out[name + "_codes"] = encoded(x.reshape(t * h, dim))
            continue
        if s["source"] == "codes":
            x = decode(s[name + "_codes"], t * h, dim).view(t, h, dim)
        r = root(x)
        dn = rotated(s["d" + name + "_out"].float(), s, back=True)
        g = dn * w
        mean = (g.double() * x.double()).mean(-1, keepdim=True)
        out["d" + name] = (r * (g - x * (r.double() * r.double() * mean).float())).to(dt)
        out["dw" + name] = (dn * (x * r)).sum((0, 1), dtype=torch.float64).float()
    return out


# ---------------------------------------------------------------------------------------------------------
# the library's operators


def run_own(s):
    import optimizer_step_amd as osa
    op = s["op"]
    if op == "gate":
        osa.opt_gated_act(s["gate"], s["up"], s["act"], y=s["y"], codes=s["q"], gate_codes=s["gate_q"], up_codes=s["up_q"])
        out = {k: s[k + "_values"] for k in ("q", "gate_q", "up_q") if s[k] is not None}
        if s["y"] is not None:
            out["y"] = s["y"]
        return out
    if op == "gate_grad":
        gate, upper = (s["gate_q"], s["up_q"]) if s["source"] == "codes" else (s["gate"], s["up"])
        if s["out"] == "matrix":
            osa.opt_gated_act_backward(s["dy"], gate, upper, s["act"], dgate=s["dgate"], dup=s["dup"])
            return {"dgate": s["dgate"], "dup": s["dup"]}
        osa.opt_gated_act_backward(s["dy"], gate, upper, s["act"], dgate_codes=s["dgate_q"], dup_codes=s["dup_q"],
                                   dgate_codes_t=s["dgate_t"], dup_codes_t=s["dup_t"], y_codes_t=s["y_t"])
        return s["all_values"]
    if op == "restore":
        osa.opt_block_restore(s["q"], out=s["x"], codes_t=s["qt"])
        out = {}
        if s["x"] is not None:
            out["x"] = s["x"]
        if s["qt"] is not None:
            out["qt"] = s["qt_values"]
        return out
    near = s["pairs"] == "neighbours"
    if op == "heads":
        osa.opt_head_norm(s["q"], s["k"], s["wq"], s["wk"], table=s["table"], positions=s["pos"], eps=EPS, interleaved=near,
                          q_out=s["q_out"], k_out=s.get("k_out"), q_codes=s["q_codes"], k_codes=s.get("k_codes"))
        out = {"q": s["q_out"]}
        if s["kv"]:
            out["k"] = s["k_out"]
        if s["keep"]:
            out["q_codes"] = s["q_values"]
            if s["kv"]:
                out["k_codes"] = s["k_values"]
        return out
    q, k = (s["q_codes"], s.get("k_codes")) if s["source"] == "codes" else (s["q"], s["k"])
    osa.opt_head_norm_backward(s["dq_out"], s.get("dk_out"), q, k, s["wq"], s["wk"], table=s["table"], positions=s["pos"], eps=EPS,
                               interleaved=near, dq=s["dq"], dk=s["dk"], dweight_q=s["dwq"], dweight_k=s.get("dwk"))
    out = {"dq": s["dq"], "dwq": s["dwq"]}
    if s["kv"]:
        out["dk"], out["dwk"] = s["dk"], s["dwk"]
    return out


# ---------------------------------------------------------------------------------------------------------
# what a pass cannot do without


def coded_bytes(rows, cols):
    return rows * cols + rows * ((cols + BLOCK - 1) // BLOCK)


def work(case):
    if case["op"] in ("heads", "heads_grad"):
        t, h, dim, size = case["tokens"], case["heads"] + case["kv"], case["dim"], BYTES[case["dtype"]]
        n, codes = t * h * dim, coded_bytes(t * h, dim)
        small = t * (case["rot"] * 4 + 8) + (2 if case["kv"] else 1) * dim * size
        if case["op"] == "heads":
            return {"bytes": 2 * n * size + (codes if case["keep"] else 0) + small, "flops": 9 * n}
        return {"bytes": 2 * n * size + (codes if case["source"] == "codes" else n * size) + small + (2 if case["kv"] else 1) * dim * 4,
                "flops": 16 * n}
    rows, cols = case["rows"], case["cols"]
    n, size, codes, codes_t = rows * cols, BYTES[case["dtype"]], coded_bytes(rows, cols), coded_bytes(cols, rows)
    if case["op"] == "restore":
        return {"bytes": codes + (n * size if case["out"] != "codes" else 0) + (codes_t if case["out"] != "matrix" else 0), "flops": 2 * n}
    if case["op"] == "gate":
        moved = 2 * n * size + (n * size if case["out"] != "codes" else 0) + (codes if case["out"] != "y" else 0)
        return {"bytes": moved + (2 * codes if case["keep"] else 0), "flops": 6 * n}
    moved = n * size + (2 * codes if case["source"] == "codes" else 2 * n * size)
    return {"bytes": moved + (2 * n * size if case["out"] == "matrix" else 2 * codes + 3 * codes_t), "flops": 14 * n}


# ---------------------------------------------------------------------------------------------------------
# the definitions in 64 bits


def grid(x):
    """E4M3 values and scales of a 64-bit matrix: the scale is the smallest 2^e with absmax <= 448 2^e."""
    rows, cols = x.shape
    big = torch.zeros(rows, up(cols, BLOCK), dtype=torch.float64, device=x.device)
    big[:, :cols] = x.abs()
    top = big.unfold(1, BLOCK, BLOCK).amax(2)
    e = torch.ceil(torch.log2(top.clamp(min=1e-300) / 448))
    e = e + (top > 448 * torch.exp2(e)).double()
    e = (e - (top <= 448 * torch.exp2(e - 1)).double()).clamp(min=-127)
    scale = torch.exp2(e)
    y = x / scale.repeat_interleave(BLOCK, 1)[:, :cols]
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0**-6))) - 3)
    return {"codes": torch.round(y / step) * step, "scales": scale.t().contiguous()}


def meaning(pair, rows, cols):
    q, s = pair
    scale = torch.exp2(s[:, :rows].double() - 127).t()
    return q[:, :cols].view(torch.float8_e4m3fn).to(torch.float64) * scale.repeat_interleave(BLOCK, 1)[:, :cols]


def exact_gate(x, act):
    """(s, s') of the activation: the logistic function by exp, the other by tanh."""
    if act == "silu":
        h = 1 / (1 + torch.exp(-x))
        return x * h, h + x * h * (1 - h)
    t = torch.tanh(math.sqrt(2 / math.pi) * (x + 0.044715 * x**3))
    return 0.5 * x * (1 + t), 0.5 * (1 + t) + 0.5 * x * (1 - t * t) * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * x * x)


def exact_turn(x, s, sign):
    """Heads [tokens, heads, dim] turned pair by pair, as products with complex numbers."""
    rot = s["rot"]
    if not rot:
        return x
    row = s["table"].double()[s["pos"]]
    unit = torch.complex(row[:, :rot // 2], sign * row[:, rot // 2:])[:, None, :]
    y = x.clone()
    if s["pairs"] == "halves":
        z = torch.complex(x[..., :rot // 2].contiguous(), x[..., rot // 2:rot].contiguous()) * unit
        y[..., :rot // 2], y[..., rot // 2:rot] = z.real, z.imag
    else:
        z = torch.complex(x[..., 0:rot:2].contiguous(), x[..., 1:rot:2].contiguous()) * unit
        y[..., 0:rot:2], y[..., 1:rot:2] = z.real, z.imag
    return y


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("gate", "gate_grad"):
        rows, cols = case["rows"], case["cols"]
        if case.get("source") == "codes":
            gate, upper = meaning(s["gate_q"], rows, cols), meaning(s["up_q"], rows, cols)
        else:
            gate, upper = s["gate"].double(), s["up"].double()
        y, slope = exact_gate(gate, case["act"])
        if op == "gate":
            out = {"y": y * upper} if case["out"] != "codes" else {}
            if case["out"] != "y":
                out["q"] = grid(y * upper)
            if case["keep"]:
                out["gate_q"], out["up_q"] = grid(gate), grid(upper)
            return out
        dy = s["dy"].double()
        dgate, dup = dy * upper * slope, dy * y
        if case["out"] == "matrix":
            return {"dgate": dgate, "dup": dup}
        out = {"dgate_q": grid(dgate), "dup_q": grid(dup)}
        for name, v in (("dgate_t", dgate), ("dup_t", dup), ("y_t", y * upper)):
            out[name] = grid(v.t().contiguous())
        return out
    if op == "restore":
        x = meaning(s["q"], case["rows"], case["cols"])
        out = {"x": x} if case["out"] != "codes" else {}
        if case["out"] != "matrix":
            out["qt"] = grid(x.t().contiguous())
        return out
    out = {}
    for name in ("q", "k") if case["kv"] else ("q",):
        x, w = s[name].double(), s["w" + name].double()
        t, h, dim = x.shape
        if op == "heads":
            n = x / torch.sqrt((x * x).sum(-1, keepdim=True) / dim + EPS) * w
            out[name] = exact_turn(n, s, 1.0)
            if case["keep"]:
                out[name + "_codes"] = grid(x.reshape(t * h, dim))
            continue
        if case["source"] == "codes":
            x = meaning(s[name + "_codes"], t * h, dim).view(t, h, dim)
        v = (x * x).sum(-1, keepdim=True) / dim + EPS
        dn = exact_turn(s["d" + name + "_out"].double(), s, -1.0)
        g = dn * w
        out["d" + name] = g / v.sqrt() - x * ((g * x).sum(-1, keepdim=True) / dim) / v**1.5
        out["dw" + name] = (dn * x / v.sqrt()).sum((0, 1))
    return out
