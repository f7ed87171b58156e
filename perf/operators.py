"""Measured cases of the training-pass operators beside the optimizer step: dropout, the RMS norm with the
residual's addition, the cast to block-scaled 8-bit codes, and the product of two such matrices.

``listed()`` and ``draw()`` give the cases, ``prepare()`` the tensors a program holds before the call, and
``run()`` one pass: with ``own`` false in elementary torch operations, with ``own`` true by the library's
entry points.  ``exact()`` gives the same outputs from the definitions in 64 bits, and ``work()`` the bytes
and operations a pass cannot do without.

A block-coded matrix is a pair (codes, scales): E4M3 codes [rows, cols rounded up to 16] with zero codes past
the last column, and one power-of-two scale X = 2^(byte - 127) for each row and each 128 columns, stored
[ceil(cols / 128), rows rounded up to 4].  X is the smallest power of two with absmax <= 448 X.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 128
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
DEVICE = "cuda"


def up(n, m):
    return (n + m - 1) // m * m


# ---------------------------------------------------------------------------------------------------------
# the cases


def listed():
    return [
        # one token's activations on their way into the residual stream: latency
        dict(name="dropout-token", op="dropout", rows=1, cols=4096, dtype="bf16", p=0.1, residual=True),
        # the branch of a block joins the residual stream, 8192 tokens
        dict(name="dropout-residual", op="dropout", rows=8192, cols=4096, dtype="bf16", p=0.1, residual=True),
        # the gradient goes back through the same mask, in 32 bits, an odd size
        dict(name="dropout-gradient-odd", op="dropout", rows=1023, cols=4099, dtype="f32", p=0.35, residual=False),
        # serving: one token, the residual's addition, codes for the product that follows
        dict(name="norm-token", op="norm", rows=1, cols=4096, dtype="bf16", residual=True, out="codes", pad=0),
        # a training or prompt pass: 8192 tokens into 8-bit codes
        dict(name="norm-tokens", op="norm", rows=8192, cols=4096, dtype="bf16", residual=True, out="codes", pad=0),
        # heads' norms in 16 bits, short rows out of a wider tensor
        dict(name="norm-heads", op="norm", rows=30001, cols=128, dtype="f16", residual=False, out="y", pad=256),
        # its backward pass with the residual's gradient
        dict(name="norm-gradient", op="norm_grad", rows=8192, cols=4096, dtype="bf16", residual=True, pad=0),
        # activations to codes in both layouts: the forward product's and the weight gradient's
        dict(name="cast-activations", op="cast", rows=8192, cols=4096, dtype="bf16", block_rows=1, both=True),
        # a fp32 weight after the step, one scale per 128 x 128, both layouts
        dict(name="cast-weight", op="cast", rows=11008, cols=4096, dtype="f32", block_rows=128, both=True),
        # serving: one token through the widest layer
        dict(name="product-token", op="product", m=1, n=11008, k=4096, out="bf16", accumulate=False),
        # a batch of tokens, odd
        dict(name="product-batch-odd", op="product", m=77, n=4100, k=4112, out="f16", accumulate=False),
        # the weight gradient of 8192 tokens, added to the fp32 gradient the step reads
        dict(name="product-weight-gradient", op="product", m=11008, n=4096, k=8192, out="f32", accumulate=True),
    ]


def spread(rng, lo, hi, odd=0.5):
    """A size over the logarithm of [lo, hi]; half of them as they fall, the others a multiple of 16."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return v if rng.random() < odd else min(hi, max(lo, up(v, 16)))


def draw(rng):
    op = rng.choice(["dropout", "norm", "norm_grad", "cast", "product", "product"])
    if op == "product":
        m, n, k = spread(rng, 1, 8192), spread(rng, 16, 16384), spread(rng, 64, 16384)
        while m * n * k > 11008 * 4096 * 8192:
            m, n, k = max(1, m // 2), n // 2 + 8, k // 2 + 32
        out = rng.choice(["bf16", "bf16", "f16", "f32"])
        return dict(op=op, m=m, n=n, k=k, out=out, accumulate=out == "f32" and rng.random() < 0.5)
    rows, cols = spread(rng, 1, 32768), spread(rng, 64, 16384)
    while rows * cols > 8192 * 4096:
        rows = max(1, rows // 2)
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "dropout":
        return dict(op=op, rows=rows, cols=cols, dtype=dtype, p=round(rng.uniform(0.02, 0.6), 3), residual=rng.random() < 0.5)
    if op == "norm":
        return dict(op=op, rows=rows, cols=cols, dtype=dtype, residual=rng.random() < 0.6, out=rng.choice(["codes", "y", "both"]),
                    pad=rng.choice([0, 0, 8, 51]))
    if op == "norm_grad":
        return dict(op=op, rows=rows, cols=cols, dtype=dtype, residual=rng.random() < 0.6, pad=rng.choice([0, 0, 8, 51]))
    return dict(op=op, rows=rows, cols=cols, dtype=dtype, block_rows=rng.choice([1, 128]), both=rng.random() < 0.6)


# ---------------------------------------------------------------------------------------------------------
# inputs


def coded_buffers(rows, cols):
    return (torch.zeros(rows, up(cols, 16), dtype=torch.uint8, device=DEVICE),
            torch.zeros(up(cols, BLOCK) // BLOCK, up(rows, 4), dtype=torch.uint8, device=DEVICE))


def values(q, s, rows, cols):
    """What a pair's bytes stand for: E4M3 values and power-of-two scales."""
    return {"codes": q[:, :cols].view(torch.float8_e4m3fn), "scales": s[:, :rows].view(torch.float8_e8m0fnu)}


def normal(g, rows, cols, dtype, std=1.0, pad=0):
    return (torch.randn(rows, cols + pad, generator=g, device=DEVICE) * std).to(DTYPES[dtype])[:, :cols]


def activations(g, rows, cols, dtype, pad=0):
    """Rows of different sizes and a few loud channels, as a residual stream has them."""
    loud = 1 + 9 * (torch.rand(cols + pad, generator=g, device=DEVICE) < 0.01).float()
    size = 0.5 + torch.rand(rows, 1, generator=g, device=DEVICE)
    return (torch.randn(rows, cols + pad, generator=g, device=DEVICE) * loud * size).to(DTYPES[dtype])[:, :cols]


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    s = dict(case)
    if case["op"] == "product":
        m, n, k = case["m"], case["n"], case["k"]
        for name, rows, block_rows, x in (("a", m, 1, activations(g, m, k, "f32")), ("b", n, 128, normal(g, n, k, "f32", 0.02))):
            q, e = encode(x, block_rows)
            buf = coded_buffers(rows, k)
            buf[0][:, :k] = q.view(torch.uint8)
            buf[1][:, :rows] = e.to(torch.uint8)
            s[name] = buf
        s["out_t"] = normal(g, m, n, "f32", 0.1) if case["accumulate"] else torch.empty(m, n, dtype=DTYPES[case["out"]], device=DEVICE)
        return s
    rows, cols, dt = case["rows"], case["cols"], DTYPES[case["dtype"]]
    pad = case.get("pad", 0)

    def empty():
        return torch.empty(rows, cols, dtype=dt, device=DEVICE)

    if case["op"] == "dropout":
        s["x"] = activations(g, rows, cols, case["dtype"])
        s["res"] = activations(g, rows, cols, case["dtype"]) if case["residual"] else None
        s["seed"], s["offset"] = seed * 0x9E3779B97F4A7C15 % 2**64, 2 * seed + 1
        s["out_t"] = empty()
    elif case["op"] == "norm":
        s["x"] = activations(g, rows, cols, case["dtype"], pad)
        s["res"] = activations(g, rows, cols, case["dtype"]) if case["residual"] else None
        s["w"] = 1 + normal(g, 1, cols, case["dtype"], 0.2)[0]
        s["h"] = empty() if case["residual"] else None
        s["y"] = empty() if case["out"] != "codes" else None
        s["q"] = coded_buffers(rows, cols) if case["out"] != "y" else None
        s["q_values"] = values(*s["q"], rows, cols) if s["q"] else None
    elif case["op"] == "norm_grad":
        s["dy"] = normal(g, rows, cols, case["dtype"], 0.01, pad)
        s["h"] = activations(g, rows, cols, case["dtype"])
        s["w"] = 1 + normal(g, 1, cols, case["dtype"], 0.2)[0]
        s["dres"] = normal(g, rows, cols, case["dtype"], 0.01) if case["residual"] else None
        s["dx"] = empty()
        s["dw"] = torch.empty(cols, dtype=torch.float32, device=DEVICE)
    else:
        s["x"] = normal(g, rows, cols, case["dtype"], 0.02) if case["block_rows"] == BLOCK else activations(g, rows, cols, case["dtype"])
        s["q"] = coded_buffers(rows, cols)
        s["qt"] = coded_buffers(cols, rows) if case["both"] else None
        s["q_values"] = values(*s["q"], rows, cols)
        s["qt_values"] = values(*s["qt"], cols, rows) if case["both"] else None
    return s


# ---------------------------------------------------------------------------------------------------------
# the plain form


def philox(c0, c1, c2, c3, k0, k1):
    """Philox4x32-10 over int64 tensors that hold 32-bit words (Salmon, Moraes, Dror, Shaw, SC'11)."""
    mask = 0xFFFFFFFF

    def product(a, b):   # the high and the low word of a 32 x 32 bit product, in 63 bits
        t = (a >> 16) * b + (((a & 0xFFFF) * b) >> 16)
        return t >> 16, (a * (b & 0xFFFF) + (((a * (b >> 16)) & 0xFFFF) << 16)) & mask

    for r in range(10):
        h0, l0 = product(c0, 0xD2511F53)
        h1, l1 = product(c2, 0xCD9E8D57)
        c0, c1, c2, c3 = h1 ^ c1 ^ ((k0 + r * 0x9E3779B9) & mask), l1, h0 ^ c3 ^ ((k1 + r * 0xBB67AE85) & mask), l0
    return c0, c1, c2, c3


def kept(n, p, seed, offset):
    """Which of n elements stay: element j takes the j%8-th 16 bits of block j>>3 of its stream."""
    q = torch.arange((n + 7) // 8, dtype=torch.int64, device=DEVICE)
    c = [torch.full_like(q, v) for v in (offset & 0xFFFFFFFF, offset >> 32)]
    w = philox(q & 0xFFFFFFFF, (q >> 32) | 0x80000000, c[0], c[1], seed & 0xFFFFFFFF, seed >> 32)
    bits = torch.stack([h for v in w for h in (v & 0xFFFF, v >> 16)], 1).reshape(-1)[:n]
    return bits >= math.floor(p * 65536 + 0.5)


def power(e):
    """2^e as binary32, -127 <= e <= 127."""
    return torch.where(e < -126, torch.full_like(e, 0x00400000), (e + 127) << 23).to(torch.int32).view(torch.float32)


def block_max(x, block_rows):
    """Largest magnitude for each row (or 128 rows) and 128 columns, as [ceil(cols / 128), rows]."""
    rows, cols = x.shape
    a = torch.nn.functional.pad(x.abs(), (0, -cols % BLOCK, 0, -rows % block_rows))
    a = a.reshape(a.shape[0] // block_rows, block_rows, -1, BLOCK).amax((1, 3))
    return a.repeat_interleave(block_rows, 0)[:rows].t().contiguous()


def encode(x, block_rows):
    """(E4M3 values, scale bytes) of fp32 x."""
    a = block_max(x, block_rows)
    m, e = torch.frexp(a)                                          # a = m 2^e with m in [0.5, 1)
    e = torch.where(a > 0, e.long() - 9 + (m > 0.875), -127).clamp(min=-127)   # 448 = 0.875 * 2^9
    shift = power(-e).t().repeat_interleave(BLOCK, 1)[:, :x.shape[1]]
    return (x * shift).to(torch.float8_e4m3fn), e + 127


def decode(q, s, rows, cols):
    scale = power(s[:, :rows].long() - 127).t().repeat_interleave(BLOCK, 1)[:, :cols]
    return q[:, :cols].view(torch.float8_e4m3fn).to(torch.float32) * scale


def root(h, eps):
    """1 / sqrt(mean h^2 + eps) of each row, the sum in 64 bits, as binary32."""
    return (1 / torch.sqrt(h.double().square().mean(1, keepdim=True) + eps)).float()


EPS = 1e-6


def run(state):
    s = state
    op = s["op"]
    if own:
        return run_own(s)
    if op == "dropout":
        t = math.floor(s["p"] * 65536 + 0.5)
        y = s["x"].float() * float(np.float32(1 / (1 - t / 65536)))
        keep = kept(y.numel(), s["p"], s["seed"], s["offset"]).view_as(y)
        y = torch.where(keep, y, torch.zeros_like(y))
        return (y if s["res"] is None else y + s["res"].float()).to(s["x"].dtype)
    if op == "norm":
        h = s["x"].float()
        out = {}
        if s["res"] is not None:
            out["h"] = (h + s["res"].float()).to(s["x"].dtype)
            h = out["h"].float()
        y = h * root(h, EPS) * s["w"].float()
        if s["y"] is not None:
            out["y"] = y.to(s["x"].dtype)
        if s["q"] is not None:
            q, e = encode(y, 1)
            out["q"] = {"codes": q, "scales": e.to(torch.uint8).view(torch.float8_e8m0fnu)}
        return out
    if op == "norm_grad":
        h, dy = s["h"].float(), s["dy"].float()
        r = root(h, EPS)
        dn = dy * s["w"].float()
        mean = (dn.double() * h.double()).mean(1, keepdim=True)
        dx = r * (dn - h * (r.double() * r.double() * mean).float())
        if s["dres"] is not None:
            dx = dx + s["dres"].float()
        return {"dx": dx.to(s["dy"].dtype), "dw": (dy * (h * r)).sum(0)}
    if op == "cast":
        x = s["x"].float()
        q, e = encode(x, s["block_rows"])
        out = {"q": {"codes": q, "scales": e.to(torch.uint8).view(torch.float8_e8m0fnu)}}
        if s["qt"] is not None:
            q, e = encode(x.t().contiguous(), s["block_rows"])
            out["qt"] = {"codes": q, "scales": e.to(torch.uint8).view(torch.float8_e8m0fnu)}
        return out
    a, b = (decode(*s[v], rows, s["k"]) for v, rows in (("a", s["m"]), ("b", s["n"])))
    c = a @ b.t()
    return s["out_t"].add_(c) if s["accumulate"] else c.to(s["out_t"].dtype)


# ---------------------------------------------------------------------------------------------------------
# the library's operators


def run_own(s):
    import optimizer_step_amd as osa
    op = s["op"]
    if op == "dropout":
        osa.opt_dropout(s["x"], s["out_t"], s["p"], seed=s["seed"], offset=s["offset"], residual=s["res"])
        return s["out_t"]
    if op == "norm":
        osa.opt_rms_norm(s["x"], s["w"], eps=EPS, residual=s["res"], h=s["h"], y=s["y"], codes=s["q"])
        out = {}
        if s["h"] is not None:
            out["h"] = s["h"]
        if s["y"] is not None:
            out["y"] = s["y"]
        if s["q"] is not None:
            out["q"] = s["q_values"]
        return out
    if op == "norm_grad":
        osa.opt_rms_norm_backward(s["dy"], s["h"], s["w"], s["dx"], s["dw"], eps=EPS, dh=s["dres"])
        return {"dx": s["dx"], "dw": s["dw"]}
    if op == "cast":
        osa.opt_block_cast(s["x"], codes=s["q"], codes_t=s["qt"], block_rows=s["block_rows"])
        out = {"q": s["q_values"]}
        if s["qt"] is not None:
            out["qt"] = s["qt_values"]
        return out
    osa.opt_block_matmul(s["a"], s["b"], s["out_t"], accumulate=s["accumulate"])
    return s["out_t"]


# ---------------------------------------------------------------------------------------------------------
# what a pass cannot do without


def coded_bytes(rows, cols):
    return rows * cols + rows * ((cols + BLOCK - 1) // BLOCK)


def work(case):
    if case["op"] == "product":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": coded_bytes(m, k) + coded_bytes(n, k) + m * n * BYTES[case["out"]] * (2 if case["accumulate"] else 1),
                "flops": 2 * m * n * k}
    rows, cols = case["rows"], case["cols"]
    n, size = rows * cols, BYTES[case["dtype"]]
    if case["op"] == "dropout":
        return {"bytes": n * size * (3 if case["residual"] else 2), "flops": 2 * n}
    if case["op"] == "norm":
        moved = n * size * (3 if case["residual"] else 1) + cols * size
        moved += n * size if case["out"] != "codes" else 0
        moved += coded_bytes(rows, cols) if case["out"] != "y" else 0
        return {"bytes": moved, "flops": 5 * n}
    if case["op"] == "norm_grad":
        return {"bytes": n * size * (4 if case["residual"] else 3) + cols * (size + 4), "flops": 11 * n}
    return {"bytes": n * size + coded_bytes(rows, cols) + (coded_bytes(cols, rows) if case["both"] else 0), "flops": 3 * n}


# ---------------------------------------------------------------------------------------------------------
# the definitions in 64 bits


def words(n, seed, offset):
    """The 16-bit random integers of n elements, from the generator's definition on 64-bit unsigned integers."""
    u = np.uint64
    low = u(0xFFFFFFFF)
    q = np.arange((n + 7) // 8, dtype=np.uint64)
    x = [q & low, (q >> u(32)) | u(1 << 31), np.full_like(q, offset & 0xFFFFFFFF), np.full_like(q, offset >> 32)]
    key = [seed & 0xFFFFFFFF, seed >> 32]
    for _ in range(10):
        a, b = x[0] * u(0xD2511F53), x[2] * u(0xCD9E8D57)
        x = [(b >> u(32)) ^ x[1] ^ u(key[0]), b & low, (a >> u(32)) ^ x[3] ^ u(key[1]), a & low]
        key = [(key[0] + 0x9E3779B9) % 2**32, (key[1] + 0xBB67AE85) % 2**32]
    return np.stack(x, 1).astype(np.uint32).view(np.uint16).reshape(-1)[:n]


def grid(x, block_rows):
    """E4M3 values and scales of a 64-bit matrix: the scale is the smallest 2^e with absmax <= 448 2^e."""
    rows, cols = x.shape
    big = torch.zeros(up(rows, block_rows), up(cols, BLOCK), dtype=torch.float64, device=x.device)
    big[:rows, :cols] = x.abs()
    top = big.unfold(0, block_rows, block_rows).unfold(1, BLOCK, BLOCK).amax((2, 3))
    e = torch.ceil(torch.log2(top.clamp(min=1e-300) / 448))
    e = e + (top > 448 * torch.exp2(e)).double()
    e = (e - (top <= 448 * torch.exp2(e - 1)).double()).clamp(min=-127)
    scale = torch.exp2(e)
    each = scale.repeat_interleave(block_rows, 0)[:rows]
    y = x / each.repeat_interleave(BLOCK, 1)[:, :cols]
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0**-6))) - 3)
    return {"codes": torch.round(y / step) * step, "scales": each.t().contiguous()}


def meaning(q, s, rows, cols):
    scale = torch.exp2(s[:, :rows].double() - 127).t()
    return q[:, :cols].view(torch.float8_e4m3fn).to(torch.float64) * scale.repeat_interleave(BLOCK, 1)[:, :cols]


def exact(case, seed):
    s = prepare(case, seed)
    wide = {k: v.double() for k, v in s.items() if torch.is_tensor(v)}
    op = case["op"]
    if op == "dropout":
        t = math.floor(case["p"] * 65536 + 0.5)
        stay = torch.from_numpy((words(case["rows"] * case["cols"], s["seed"], s["offset"]) >= t)).to(DEVICE).view_as(wide["x"])
        y = wide["x"] / (1 - t / 65536) * stay
        return y + wide["res"] if "res" in wide else y
    if op == "norm":
        out, h = {}, wide["x"]
        if "res" in wide:
            out["h"] = h + wide["res"]
            h = out["h"].to(DTYPES[case["dtype"]]).double()        # the norm is that of the stored sum
        y = h * torch.rsqrt((h * h).sum(1, keepdim=True) / case["cols"] + EPS) * wide["w"]
        if case["out"] != "codes":
            out["y"] = y
        if case["out"] != "y":
            out["q"] = grid(y, 1)
        return out
    if op == "norm_grad":
        h, dy = wide["h"], wide["dy"]
        v = (h * h).sum(1, keepdim=True) / case["cols"] + EPS
        g = dy * wide["w"]
        dx = g / v.sqrt() - h * ((g * h).sum(1, keepdim=True) / case["cols"]) / v**1.5
        return {"dx": dx + wide["dres"] if "dres" in wide else dx, "dw": (dy * h / v.sqrt()).sum(0)}
    if op == "cast":
        out = {"q": grid(wide["x"], case["block_rows"])}
        if case["both"]:
            out["qt"] = grid(wide["x"].t().contiguous(), case["block_rows"])
        return out
    c = meaning(*s["a"], case["m"], case["k"]) @ meaning(*s["b"], case["n"], case["k"]).t()
    return wide["out_t"] + c if case["accumulate"] else c
