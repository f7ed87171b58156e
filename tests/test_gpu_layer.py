"""GPU parity of the operators between a layer's products (gated activation,
restored codes, heads' norm with rotation, and their backward passes) against
their plain forms in binary64."""
import numpy as np
import pytest

from tests import layer_plain as G
from tests import pass_plain as P
from tests.test_gpu_pass import check_coded, data, dev, empty, host, marked_codes, untouched

pytestmark = pytest.mark.gpu

DTYPES = ["f32", "bf16", "f16"]


@pytest.fixture(scope="module", autouse=True)
def gpu():
    import torch
    import optimizer_step_amd as osa
    assert torch.cuda.is_available()
    osa.lib()


def coded(x, block_rows=1):
    """(a pair on the device, the values it holds) of a host array."""
    import torch
    import optimizer_step_amd as osa
    codes, scales = P.encode(x, block_rows)
    q, s = osa.block_buffers(*x.shape)
    q[:, :x.shape[1]] = torch.from_numpy(codes).cuda()
    s[:, :x.shape[0]] = torch.from_numpy(scales).cuda()
    return (q, s), P.decode(codes, scales, x.shape[1])


def same_codes(a, b, rows, cols):
    import torch
    n = (cols + 127) // 128
    return torch.equal(a[0][:rows, :cols], b[0][:rows, :cols]) and torch.equal(a[1][:n, :rows], b[1][:n, :rows])


def kept(pair, rows):
    """The mark beside a marked_codes pair's rows still stands."""
    return bool((pair[0][rows:] == 0x5A).all()) and bool((pair[1][:, P.up(rows, 4):] == 0x5A).all())


def part(pair, rows):
    return pair[0][:rows], pair[1]


# ---- the gated activation ---------------------------------------------------

SIZES = [(1, 1), (1, 8), (3, 5), (17, 127), (5, 128), (130, 129), (128, 256), (33, 250), (257, 1000), (2, 2049), (1, 11008)]


def gate_inputs(rows, cols, dtype, seed=0):
    return (P.rounded(4 * data(seed + cols, rows, cols, "f32"), dtype), data(seed + cols + 1, rows, cols, dtype),
            data(seed + cols + 2, rows, cols, dtype, 0.1))


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gated_act(rows, cols, dtype, act):
    import torch
    import optimizer_step_amd as osa
    x, u, _ = gate_inputs(rows, cols, dtype)
    y, q, gq, uq = empty(rows, cols, dtype, 3), marked_codes(rows, cols), marked_codes(rows, cols), marked_codes(rows, cols)
    dx, du = dev(x, dtype, 5), dev(u, dtype, 2)
    osa.opt_gated_act(dx, du, act, y=y, codes=part(q, rows), gate_codes=part(gq, rows), up_codes=part(uq, rows))
    want, bound = G.gate(x, u, act, dtype)
    G.check_values(host(y), want, G.stored(want, bound, dtype))
    assert untouched(y) and kept(q, rows)
    G.check_codes(part(q, rows), want, bound, rows, cols)
    check_coded(gq, *P.encode(x), rows, cols)
    check_coded(uq, *P.encode(u), rows, cols)
    # each output alone has the same bits; the halves of one matrix too
    z = torch.cat([dx, du], 1)
    y2, q2, g2 = empty(rows, cols, dtype), osa.block_buffers(rows, cols), osa.block_buffers(rows, cols)
    osa.opt_gated_act(z[:, :cols], z[:, cols:], act, y=y2)
    osa.opt_gated_act(z[:, :cols], z[:, cols:], act, codes=q2)
    osa.opt_gated_act(z[:, :cols], z[:, cols:], act, gate_codes=g2)
    assert torch.equal(y, y2) and same_codes(q, q2, rows, cols) and same_codes(gq, g2, rows, cols)
    for out in (dx, du):                            # in place
        a, b = dx.contiguous().clone(), du.contiguous().clone()
        osa.opt_gated_act(a, b, act, y=a if out is dx else b)
        assert torch.equal(a if out is dx else b, y2)


EDGES = np.array([0.0, -0.0, 1e-30, -1e-30, 88.0, -88.0, 104.0, -104.0, 1e4, -1e4, 3e38, -3e38, np.inf, -np.inf, np.nan, 16.0, -16.0, 15.9])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gated_act_edge_values(dtype, act):
    """The formula's values at its ends, forward and backward: a saturated gate
    passes up or nothing, infinities and NaNs as the formula in binary64 gives
    them, and only their own block's codes are lost."""
    import torch
    import optimizer_step_amd as osa
    cols = 256
    x = np.zeros((EDGES.size, cols), np.float32)
    x[:, 130] = P.rounded(EDGES.astype(np.float32), dtype)
    x[:, 3] = 1.0
    u, dy = np.full_like(x, 0.5), np.full_like(x, 0.25)
    y, dg, du = (empty(EDGES.size, cols, dtype) for _ in range(3))
    q = osa.block_buffers(EDGES.size, cols)
    osa.opt_gated_act(dev(x, dtype), dev(u, dtype), act, y=y, codes=q)
    osa.opt_gated_act_backward(dev(dy, dtype), dev(x, dtype), dev(u, dtype), act, dgate=dg, dup=du)
    with np.errstate(invalid="ignore", over="ignore"):
        want, bound = G.gate(x, u, act, dtype)
        (wg, bg), (wu, bu), _ = G.gate_gradients(dy, x, u, act, dtype)
    for got, w, b in ((y, want, bound), (dg, wg, bg), (du, wu, bu)):
        w = np.where(np.abs(w) > 65520 if dtype == "f16" else False, np.copysign(np.inf, w), w)   # past the type's range
        with np.errstate(invalid="ignore"):
            lim = G.stored(w, np.where(np.isfinite(b), b, 2.0 ** -100), dtype)
        G.check_values(host(got), w, lim)
    s = q[1].cpu().numpy()[:, :EDGES.size]
    with np.errstate(invalid="ignore"):
        lost = ~np.isfinite(want[:, 128:]).all(1)
    assert np.array_equal(s[1] == 255, lost) and not (s[0] == 255).any()


def grad_outputs(rows, cols, dtype):
    return dict(dgate=empty(rows, cols, dtype, 3), dup=empty(rows, cols, dtype, 1)), {
        "dgate_codes": marked_codes(rows, cols), "dup_codes": marked_codes(rows, cols), "dgate_codes_t": marked_codes(cols, rows),
        "dup_codes_t": marked_codes(cols, rows), "y_codes_t": marked_codes(cols, rows)}


@pytest.mark.parametrize("rows,cols", SIZES + [(129, 5), (300, 130)])
@pytest.mark.parametrize("dtype,act,from_codes", [("f32", "silu", False), ("f32", "gelu", True), ("bf16", "silu", True), ("bf16", "gelu", False),
                                                  ("f16", "gelu", True), ("f16", "silu", False)])
def test_gated_act_backward(rows, cols, dtype, act, from_codes):
    import torch
    import optimizer_step_amd as osa
    x, u, dy = gate_inputs(rows, cols, dtype)
    if from_codes:
        (gx, x), (gu, u) = coded(x), coded(u)
    else:
        gx, gu = dev(x, dtype, 5), dev(u, dtype, 2)
    mats, pairs = grad_outputs(rows, cols, dtype)
    sides = {k: (cols, rows) if k.endswith("_t") else (rows, cols) for k in pairs}
    osa.opt_gated_act_backward(dev(dy, dtype, 9), gx, gu, act, **mats, **{k: part(v, sides[k][0]) for k, v in pairs.items()})
    want = G.gate_gradients(dy, x, u, act, dtype)
    for (w, b), k in zip(want, ("dgate", "dup", "y")):
        if k != "y":
            G.check_values(host(mats[k]), w, G.stored(w, b, dtype))
            assert untouched(mats[k])
            G.check_codes(part(pairs[k + "_codes"], rows), w, b, rows, cols)
        G.check_codes(part(pairs[k + "_codes_t"], cols), w.T.copy(), b.T.copy(), cols, rows)
    for k, (r, c) in sides.items():
        assert kept(pairs[k], r)
    # each output alone has the same bits
    for k, v in mats.items():
        alone = empty(rows, cols, dtype)
        osa.opt_gated_act_backward(dev(dy, dtype), gx, gu, act, **{k: alone})
        assert torch.equal(alone, v)
    for k, v in pairs.items():
        alone = osa.block_buffers(*sides[k])
        osa.opt_gated_act_backward(dev(dy, dtype), gx, gu, act, **{k: alone})
        assert same_codes(alone, v, *sides[k])


def test_gated_act_backward_in_place_and_halves():
    """dgate over dy or gate, dup over dy or up; both halves of one matrix and of one coded matrix in both layouts."""
    import torch
    import optimizer_step_amd as osa
    rows, cols = 200, 384
    x, u, dy = (dev(v, "bf16") for v in gate_inputs(rows, cols, "bf16"))
    dg, du = torch.empty_like(x), torch.empty_like(x)
    osa.opt_gated_act_backward(dy, x, u, dgate=dg, dup=du)
    for over in range(4):
        a, b, d = x.clone(), u.clone(), dy.clone()
        og, ou = ((a, b), (d, b), (a, d), (b, a))[over]
        osa.opt_gated_act_backward(d, a, b, dgate=og, dup=ou)
        assert torch.equal(og, dg) and torch.equal(ou, du)
    dz = torch.empty(rows, 2 * cols, dtype=torch.bfloat16, device="cuda")
    zq, zt = osa.block_buffers(rows, 2 * cols), osa.block_buffers(2 * cols, rows)
    n = cols // 128
    osa.opt_gated_act_backward(dy, x, u, dgate=dz[:, :cols], dup=dz[:, cols:], dgate_codes=(zq[0][:, :cols], zq[1][:n]),
                               dup_codes=(zq[0][:, cols:], zq[1][n:]), dgate_codes_t=(zt[0][:cols], zt[1][:, :cols]),
                               dup_codes_t=(zt[0][cols:], zt[1][:, cols:]))
    assert torch.equal(dz, torch.cat([dg, du], 1))
    each = {k: osa.block_buffers(*((cols, rows) if k.endswith("t") else (rows, cols)))
            for k in ("dgate_codes", "dup_codes", "dgate_codes_t", "dup_codes_t")}
    osa.opt_gated_act_backward(dy, x, u, **each)
    assert torch.equal(zq[0], torch.cat([each["dgate_codes"][0], each["dup_codes"][0]], 1))
    assert torch.equal(zq[1], torch.cat([each["dgate_codes"][1], each["dup_codes"][1]], 0))
    assert torch.equal(zt[0], torch.cat([each["dgate_codes_t"][0], each["dup_codes_t"][0]], 0))
    assert torch.equal(zt[1], torch.cat([each["dgate_codes_t"][1], each["dup_codes_t"][1]], 1))


def test_gated_act_backward_lost_block():
    """A block of the checkpoint that says NaN makes NaNs of its own elements and of the blocks that hold them."""
    import optimizer_step_amd as osa
    rows, cols = 140, 300
    x, u, dy = gate_inputs(rows, cols, "f32")
    x[7, 200] = np.inf
    u[133, 299] = np.nan
    (gx, vx), (gu, vu) = coded(x), coded(u)
    dg, du, tq, yt = empty(rows, cols, "f32"), empty(rows, cols, "f32"), osa.block_buffers(cols, rows), osa.block_buffers(cols, rows)
    osa.opt_gated_act_backward(dev(dy, "f32"), gx, gu, dgate=dg, dup=du, dup_codes_t=tq, y_codes_t=yt)
    with np.errstate(invalid="ignore"):
        (wg, bg), (wu, bu), (wy, _) = G.gate_gradients(dy, vx, vu, "silu", "f32")
    assert np.isnan(vx[7, 128:256]).all() and np.isnan(vu[133, 256:]).all()
    G.check_values(host(dg), wg, G.stored(wg, bg, "f32"))
    G.check_values(host(du), wu, G.stored(wu, bu, "f32"))
    for pair, w in ((tq, wu), (yt, wy)):
        s, q = pair[1].cpu().numpy()[:, :cols], pair[0].cpu().numpy()
        bad = np.isnan(np.pad(w, ((0, 116), (0, 0)))).reshape(2, 128, cols).any(1)
        assert np.array_equal(s == 255, bad)
        assert not q[np.repeat(bad.T, 128, 1)[:, :q.shape[1]]].any()


@pytest.mark.parametrize("rows,cols", [(1, 8), (5, 128), (129, 256), (130, 300), (131, 1000)])
def test_nobodys_scales(rows, cols):
    """Scale bytes past the last row, up to the multiple of four, may hold anything (NaN's here)."""
    import torch
    import optimizer_step_amd as osa
    x, u, dy = gate_inputs(rows, cols, "bf16")
    (gx, _), (gu, _) = coded(x), coded(u)
    dyd, outs = dev(dy, "bf16"), []
    for fill in (0, 255):
        for pair in (gx, gu):
            pair[1][:, rows:] = fill
        keys = ("dgate_codes", "dup_codes", "dgate_codes_t", "dup_codes_t", "y_codes_t")
        pairs = {k: osa.block_buffers(*((cols, rows) if k.endswith("_t") else (rows, cols))) for k in keys}
        dg, qt, back = empty(rows, cols, "bf16"), osa.block_buffers(cols, rows), empty(rows, cols, "bf16")
        osa.opt_gated_act_backward(dyd, gx, gu, dgate=dg, **pairs)
        osa.opt_block_restore(gx, out=back, codes_t=qt)
        heads, hq = dev(dy, "bf16").view(rows, 1, cols), gx
        dx, dw = torch.zeros_like(heads), torch.zeros(cols, device="cuda")
        if cols <= 512:
            osa.opt_head_norm_backward(heads, None, hq, None, dq=dx, dweight_q=dw)
        outs.append([dg, back, dx, dw, *qt, *(t for v in pairs.values() for t in v)])
    assert all(torch.equal(a, b) for a, b in zip(*outs))


# ---- restored codes ---------------------------------------------------------


@pytest.mark.parametrize("rows,cols", SIZES + [(129, 5), (300, 130), (512, 384)])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("block_rows", [1, 128])
def test_block_restore(rows, cols, dtype, block_rows):
    import torch
    import optimizer_step_amd as osa
    x = data(cols, rows, cols, "f32") * np.exp2(np.random.RandomState(rows).randint(-9, 4, (1, cols))).astype(np.float32)
    pair, held = coded(x, block_rows)
    out, qt = empty(rows, cols, dtype, 5), marked_codes(cols, rows)
    osa.opt_block_restore(pair, out=out, codes_t=part(qt, cols))
    assert np.array_equal(host(out), P.rounded(held, dtype)) and untouched(out)
    check_coded(qt, *P.encode(held.T.copy()), cols, rows)
    o2, q2 = empty(rows, cols, dtype), osa.block_buffers(cols, rows)
    osa.opt_block_restore(pair, out=o2)
    osa.opt_block_restore(pair, codes_t=q2)
    assert torch.equal(o2, out) and same_codes(q2, qt, cols, rows)
    # what opt_block_cast makes of the restored matrix
    wide, q3 = torch.empty(rows, cols, device="cuda"), osa.block_buffers(cols, rows)
    osa.opt_block_restore(pair, out=wide)
    osa.opt_block_cast(wide, codes_t=q3)
    assert same_codes(q3, qt, cols, rows)


def test_block_restore_scales():
    """Every scale byte: the smallest, the largest (past the type's range: infinities), and NaN."""
    import torch
    import optimizer_step_amd as osa
    q, s = osa.block_buffers(256, 128)
    q[:, :] = torch.arange(128, dtype=torch.uint8, device="cuda") * 2      # both signs, no NaN but 0x7F's neighbours
    s[0, :256] = torch.arange(256, device="cuda").to(torch.uint8)
    codes, scales = q.cpu().numpy(), s.cpu().numpy()[:, :256]
    with np.errstate(over="ignore", invalid="ignore"):
        held = P.decode(codes, scales, 128).astype(np.float32)
    for dtype in DTYPES:
        out = empty(256, 128, dtype)
        osa.opt_block_restore((q, s), out=out)
        assert np.array_equal(host(out), P.rounded(held, dtype), equal_nan=True)
    qt = osa.block_buffers(128, 256)
    osa.opt_block_restore((q, s), codes_t=qt)
    st = qt[1].cpu().numpy()[:, :128]
    assert (st[1] == 255).all()                     # rows 128 to 255 hold a NaN block
    want = P.encode(held[:128].T.copy())
    assert np.array_equal(st[0], want[1][0]) and np.array_equal(qt[0].cpu().numpy()[:, :128], want[0])


# ---- heads ------------------------------------------------------------------


def head_data(seed, tokens, heads, dim, dtype, std=1.0):
    return data(seed, tokens, heads * dim, dtype, std).reshape(tokens, heads, dim)


def laid(a, dtype, how):
    """Heads on the device: apart in a wider matrix, heads outermost, or packed."""
    import torch
    t = torch.from_numpy(np.ascontiguousarray(a)).to(P.TYPES[dtype]).cuda()
    if how == "head":
        return t.transpose(0, 1).contiguous().transpose(0, 1)
    if how == "wide":
        w = torch.full((a.shape[0], a.shape[1] + 1, a.shape[2] + 3), float("nan"), dtype=t.dtype, device="cuda")
        w[:, :a.shape[1], :a.shape[2]] = t
        return w[:, :a.shape[1], :a.shape[2]]
    return t


def head_out(tokens, heads, dim, dtype, how):
    return laid(np.full((tokens, heads, dim), -77.0, np.float32), dtype, how)


HEADS = [(1, 1, 0, 1, 0, False), (1, 32, 8, 128, 128, False), (3, 2, 1, 2, 2, False), (3, 2, 1, 2, 2, True), (5, 3, 1, 7, 6, False), (5, 3, 3, 7, 4, True),
         (9, 5, 2, 64, 64, False), (9, 4, 4, 64, 32, True), (33, 12, 3, 80, 32, True), (17, 7, 2, 80, 80, False), (11, 3, 1, 96, 24, False),
         (130, 2, 1, 128, 64, False), (8, 9, 4, 128, 128, True), (6, 3, 2, 100, 100, False), (6, 3, 2, 129, 128, False), (4, 5, 1, 192, 64, False),
         (4, 2, 1, 256, 256, False), (4, 2, 2, 255, 200, False), (3, 2, 1, 512, 512, False), (3, 2, 1, 512, 256, True), (7, 3, 2, 128, 0, False),
         (1200, 4, 2, 40, 32, False)]


def positions_of(tokens, rows, seed=0):
    p = np.random.RandomState(seed).randint(0, rows, tokens)
    p[-1] = rows - 1
    return p


@pytest.mark.parametrize("tokens,nq,nk,dim,rot,near", HEADS)
@pytest.mark.parametrize("dtype,w_dtype", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16")])
@pytest.mark.parametrize("how", ["packed", "wide", "head"])
def test_head_norm(tokens, nq, nk, dim, rot, near, dtype, w_dtype, how):
    import torch
    import optimizer_step_amd as osa
    eps, rows = 1e-5, 5000
    xs = [head_data(dim + i, tokens, n, dim, dtype) for i, n in enumerate((nq, nk))]
    ws = [P.rounded(0.5 + np.random.RandomState(dim + i).rand(dim), w_dtype) for i in range(2)]
    tab, pos = G.table(rows, max(rot, 2)), positions_of(tokens, rows)
    xd = [laid(x, dtype, how) for x in xs]
    outs = [head_out(tokens, n, dim, dtype, how) for n in (nq, nk)]
    qs = [marked_codes(tokens * n, dim) for n in (nq, nk)]
    wd = [dev(w, w_dtype) for w in ws]
    table = torch.from_numpy(tab).cuda() if rot else None
    bits = torch.int64 if dim % 2 else torch.int32
    kw = dict(table=table, positions=torch.from_numpy(pos).to(bits).cuda(), eps=eps, interleaved=near)
    osa.opt_head_norm(xd[0], xd[1] if nk else None, wd[0], wd[1], q_out=outs[0], k_out=outs[1] if nk else None,
                      q_codes=part(qs[0], tokens * nq), k_codes=part(qs[1], tokens * nk) if nk else None, **kw)
    for x, w, y, q, n in zip(xs, ws, outs, qs, (nq, nk)):
        if n:
            want, bound = G.heads(x, w, tab, pos, eps, rot, near)
            G.check_values(host(y), want, G.stored(want, bound, dtype))
            check_coded(q, *P.encode(x.reshape(tokens * n, dim)), tokens * n, dim)
            if how == "wide":
                assert bool(torch.isnan(y._base[:, n:]).all()) and bool(torch.isnan(y._base[:, :, dim:]).all())
    # in place, and without codes
    osa.opt_head_norm(xd[0], xd[1] if nk else None, wd[0], wd[1], q_out=xd[0], k_out=xd[1] if nk else None, **kw)
    assert torch.equal(xd[0], outs[0]) and (not nk or torch.equal(xd[1], outs[1]))


def sums_bound(tokens, heads, dim):
    """Additions of binary32 a lane's sum takes at most: every head of one in
    2048 waves' tokens, the lanes of a wave and its workgroup's waves."""
    lanes = 8 if dim <= 64 else 16 if dim <= 128 else 32 if dim <= 256 else 64
    return -(-tokens // min(2048, 4 * -(-tokens // 4))) * -(-heads * lanes // 64) + 8


@pytest.mark.parametrize("tokens,nq,nk,dim,rot,near", HEADS + [(2500, 2, 1, 64, 64, False), (700, 20, 1, 128, 96, False)])
@pytest.mark.parametrize("dtype,w_dtype,how,from_codes", [("f32", "f32", "wide", False), ("bf16", "bf16", "packed", True), ("bf16", "f32", "head", False),
                                                          ("f16", "f16", "head", True), ("f32", "bf16", "packed", True)])
def test_head_norm_backward(tokens, nq, nk, dim, rot, near, dtype, w_dtype, how, from_codes):
    import torch
    import optimizer_step_amd as osa
    eps, rows, more = 1e-5, 3000, how == "head"
    xs = [head_data(dim + i, tokens, n, dim, dtype) for i, n in enumerate((nq, nk))]
    dys = [head_data(dim + 7 + i, tokens, n, dim, dtype, 0.1) for i, n in enumerate((nq, nk))]
    ws = [P.rounded(0.5 + np.random.RandomState(dim + i).rand(dim), w_dtype) for i in range(2)]
    tab, pos = G.table(rows, max(rot, 2)), positions_of(tokens, rows)
    if from_codes:
        both = [coded(x.reshape(-1, dim)) if n else (None, x) for x, n in zip(xs, (nq, nk))]
        xin, xs = [b[0] for b in both], [b[1].reshape(x.shape) for b, x in zip(both, xs)]
    else:
        xin = [laid(x, dtype, how) for x in xs]
    dyd = [laid(d, dtype, how) for d in dys]
    dxs = [head_out(tokens, n, dim, dtype, how) for n in (nq, nk)]
    start = np.random.RandomState(dim).randn(2, dim).astype(np.float32) if more else np.zeros((2, dim), np.float32)
    dws = [torch.from_numpy(start[i].copy()).cuda() if more else torch.full((dim,), -5.0, device="cuda") for i in range(2)]
    table = torch.from_numpy(tab).cuda() if rot else None
    kw = dict(table=table, positions=torch.from_numpy(pos).cuda(), eps=eps, interleaved=near)
    wd = [dev(w, w_dtype) for w in ws]
    k = dict(dk=dxs[1], dweight_k=dws[1]) if nk else {}
    args = (dyd[0], dyd[1] if nk else None, xin[0], xin[1] if nk else None, wd[0], wd[1])
    osa.opt_head_norm_backward(*args, dq=dxs[0], dweight_q=dws[0], accumulate=more, **k, **kw)
    for i, n in enumerate((nq, nk)):
        if n:
            (want, bound), (want_w, terms) = G.head_gradients(dys[i], xs[i], ws[i], tab, pos, eps, rot, near)
            G.check_values(host(dxs[i]), want, G.stored(want, bound, dtype))
            lim = (5 + sums_bound(tokens, n, dim)) * P.U32 * terms * 1.05 + 2 * P.U32 * np.abs(want_w + start[i])
            G.check_values(host(dws[i]), want_w + start[i], lim)
    # without the weights' gradients; dx over dy
    alone = torch.empty_like(dxs[0])
    osa.opt_head_norm_backward(args[0], None, args[2], None, wd[0], dq=alone, **kw)
    assert torch.equal(alone, dxs[0])
    osa.opt_head_norm_backward(*args, dq=dyd[0], dk=dyd[1] if nk else None, **kw)
    assert torch.equal(dyd[0], dxs[0]) and (not nk or torch.equal(dyd[1], dxs[1]))


def test_head_positions():
    """Positions the table does not hold give NaNs to their tokens alone; none
    given, token t stands at row t; a table's rows may be apart."""
    import torch
    import optimizer_step_amd as osa
    x = head_data(1, 6, 2, 64, "bf16")
    tab = G.table(40, 64)
    wide = torch.full((40, 70), float("nan"), device="cuda")
    wide[:, :64] = torch.from_numpy(tab).cuda()
    pos = np.array([39, 40, -1, 0, 1 << 40, 7])
    ones = np.ones(64, np.float32)
    for bits in (torch.int64, torch.int32):
        p = torch.from_numpy(np.where(pos > 1000, 1000, pos) if bits == torch.int32 else pos).to(bits).cuda()
        y, dx, dw = head_out(6, 2, 64, "bf16", "packed"), head_out(6, 2, 64, "bf16", "packed"), torch.zeros(64, device="cuda")
        osa.opt_head_norm(laid(x, "bf16", "packed"), None, table=wide[:, :64], positions=p, q_out=y)
        want, bound = G.heads(x, ones, tab, pos, 1e-6, 64, False)
        assert np.isnan(want[[1, 2, 4]]).all() and np.isfinite(want[[0, 3, 5]]).all()
        G.check_values(host(y), want, G.stored(want, bound, "bf16"))
        osa.opt_head_norm_backward(laid(x, "bf16", "packed"), None, laid(x, "bf16", "packed"), None, table=wide[:, :64], positions=p, dq=dx,
                                   dweight_q=dw)
        (want, bound), _ = G.head_gradients(x, x, ones, tab, pos, 1e-6, 64, False)
        G.check_values(host(dx), want, G.stored(want, bound, "bf16"))
        assert torch.isnan(dw).all()
    y = head_out(6, 2, 64, "bf16", "packed")
    osa.opt_head_norm(laid(x, "bf16", "packed"), None, table=wide[:, :64], q_out=y)
    want, bound = G.heads(x, ones, tab, np.arange(6), 1e-6, 64, False)
    G.check_values(host(y), want, G.stored(want, bound, "bf16"))


@pytest.mark.parametrize("dtype", DTYPES)
def test_head_edge_rows(dtype):
    """Heads of zeros, tiny, large, with an infinity or a NaN: each keeps to itself."""
    import optimizer_step_amd as osa
    x = head_data(3, 2, 6, 96, dtype)
    x[0, 1] = 0
    x[0, 2] = P.rounded(np.full(96, 1e-4, np.float32), dtype)
    x[0, 3] = P.rounded(np.full(96, 6e4, np.float32), dtype)
    x[0, 4, 5] = np.inf
    x[0, 5, 90] = np.nan
    w = np.linspace(0.5, 1.5, 96).astype(np.float32)
    tab, pos = G.table(9, 64), np.array([8, 3])
    import torch
    kw = dict(table=torch.from_numpy(tab).cuda(), positions=torch.from_numpy(pos).cuda())
    y, dx = head_out(2, 6, 96, dtype, "packed"), head_out(2, 6, 96, dtype, "packed")
    osa.opt_head_norm(laid(x, dtype, "packed"), None, dev(w, "f32"), q_out=y, **kw)
    dy = head_data(4, 2, 6, 96, dtype, 0.1)
    osa.opt_head_norm_backward(laid(dy, dtype, "packed"), None, laid(x, dtype, "packed"), None, dev(w, "f32"), dq=dx, **kw)
    with np.errstate(invalid="ignore"):
        want, bound = G.heads(x, w, tab, pos, 1e-6, 64, False)
        (wg, bg), _ = G.head_gradients(dy, x, w, tab, pos, 1e-6, 64, False)
    sound = np.ones((2, 6), bool)
    sound[0, 4:] = False
    for got, v, b in ((host(y), want, bound), (host(dx), wg, bg)):
        G.check_values(got[sound], v[sound], G.stored(v, b, dtype)[sound])
    assert np.isnan(host(y)[0, 5]).all() and np.isnan(host(dx)[0, 4:]).all()
    got = host(y)[0, 4]                             # r = 0: zeros beside an infinity that becomes NaN, with its partner
    assert np.isnan(got[[5, 37]]).all() and not np.delete(got, [5, 37]).any()


def test_head_broadcast_gradient():
    """A gradient that is one token's or one head's, broadcast (strides of zero), is read as it stands."""
    import torch
    import optimizer_step_amd as osa
    x = laid(head_data(5, 20, 3, 64, "bf16"), "bf16", "packed")
    one = laid(head_data(6, 1, 1, 64, "bf16"), "bf16", "packed")
    outs = []
    for dy in (one.expand(20, 3, 64), one.expand(20, 3, 64).contiguous()):
        dx, dw = torch.empty_like(x), torch.empty(64, device="cuda")
        osa.opt_head_norm_backward(dy, None, x, None, dq=dx, dweight_q=dw)
        outs.append((dx, dw))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])


def test_keys_alone():
    """A set of no heads beside one of some: what the other set gives alone."""
    import torch
    import optimizer_step_amd as osa
    x, dy = (laid(head_data(s, 9, 3, 64, "bf16"), "bf16", "packed") for s in (7, 8))
    w = dev(1 + 0.1 * data(9, 1, 64, "f32")[0], "f32")
    none = torch.empty(9, 0, 64, dtype=torch.bfloat16, device="cuda")
    table = osa.rotation_table(9, 64)
    outs = []
    for alone in (True, False):
        y, dx, dw, q = torch.empty_like(x), torch.empty_like(x), torch.empty(64, device="cuda"), osa.block_buffers(27, 64)
        other = torch.full((64,), 5.0, device="cuda")
        if alone:
            osa.opt_head_norm(x, None, w, table=table, q_out=y, q_codes=q)
            osa.opt_head_norm_backward(dy, None, x, None, w, table=table, dq=dx, dweight_q=dw)
        else:
            osa.opt_head_norm(none, x, None, w, table=table, q_out=none, k_out=y, k_codes=q)
            osa.opt_head_norm_backward(dy[:, :0], dy, none, x, None, w, table=table, dq=none, dk=dx, dweight_q=other, dweight_k=dw)
            assert not other.any()
        outs.append((y, dx, dw, *q))
    assert all(torch.equal(a, b) for a, b in zip(*outs))


def test_readme_block_runs():
    """The block example of README.md runs as written; its results in 8 bits
    against the same block in binary32 from the tensors it holds."""
    import os
    import re
    import torch
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")).read()
    code = re.findall(r"```python\n(.*?)```", text, re.S)[2]
    torch.manual_seed(0)
    env = {}
    exec(compile("import torch, optimizer_step_amd as osa\n" + code, "README.md", "exec"), env)
    torch.cuda.synchronize()
    b, inner = env["b"].float(), env["inner"]
    gate, up = b[:, :inner].cpu().numpy(), b[:, inner:].cpu().numpy()
    want, bound = G.gate(gate, up, "silu", "bf16")
    G.check_codes(env["aq"], want, bound, *want.shape)
    held = [P.decode(q[0].cpu().numpy(), q[1].cpu().numpy()[:, :want.shape[0]], inner) for q in (env["gq"], env["uq"])]
    (dg, bg), _, _ = G.gate_gradients(env["da"].float().cpu().numpy(), held[0], held[1], "silu", "bf16")
    G.check_codes((env["bq"][0][:, :inner], env["bq"][1][:inner // 128]), dg, bg, *dg.shape)
    tokens, heads, dim = env["tokens"], env["heads"], env["dim"]
    x = env["z"].float().cpu().numpy()[:, :heads * dim].reshape(tokens, heads, dim)
    want, bound = G.heads(x, np.ones(dim), env["table"].cpu().numpy(), np.arange(tokens), 1e-6, dim, False)
    G.check_values(host(env["q"]), want, G.stored(want, bound, "bf16"))


def test_head_backward_empty():
    import torch
    import optimizer_step_amd as osa
    for tokens, heads in ((0, 4), (4, 0)):
        e = torch.empty(tokens, heads, 64, device="cuda")
        dw = torch.full((64,), 3.0, device="cuda")
        osa.opt_head_norm(e, None, q_out=e)
        osa.opt_head_norm_backward(e, None, e, None, dq=e, dweight_q=dw, accumulate=True)
        assert bool((dw == 3.0).all())
        osa.opt_head_norm_backward(e, None, e, None, dq=e, dweight_q=dw)
        assert not dw.any()


# ---- a run of them together -------------------------------------------------


def block_tensors(osa, tokens, heads, kv, dim, inner, seed=1):
    """A layer's attention inputs and feed-forward part: width heads * dim, feed-forward width inner."""
    import torch
    width, wide = heads * dim, (heads + 2 * kv) * dim
    t = {"h": dev(data(seed, tokens, width, "bf16"), "bf16"), "w": dev(1 + 0.1 * data(seed + 1, 1, width, "f32")[0], "f32"),
         "wq": dev(1 + 0.1 * data(seed + 2, 1, dim, "f32")[0], "f32"), "wk": dev(1 + 0.1 * data(seed + 3, 1, dim, "f32")[0], "f32"),
         "Wa": dev(data(seed + 4, wide, width, "f32", 0.1), "f32"), "Wb": dev(data(seed + 5, 2 * inner, width, "f32", 0.1), "f32"),
         "Wc": dev(data(seed + 6, width, inner, "f32", 0.05), "f32"), "dout": dev(data(seed + 7, tokens, width, "bf16", 0.01), "bf16"),
         "dqo": laid(head_data(seed + 8, tokens, heads, dim, "bf16", 0.01), "bf16", "head"),
         "dko": laid(head_data(seed + 9, tokens, kv, dim, "bf16", 0.01), "bf16", "head"),
         "table": osa.rotation_table(tokens + 50, dim), "pos": torch.arange(50, tokens + 50, device="cuda")}
    for name, shape, dt in (("y", (tokens, width), "bf16"), ("z", (tokens, wide), "bf16"), ("qo", (heads, tokens, dim), "bf16"),
                            ("ko", (kv, tokens, dim), "bf16"), ("dz", (tokens, wide), "bf16"), ("dwq", (dim,), "f32"), ("dwk", (dim,), "f32"),
                            ("dWa", (wide, width), "f32"), ("b", (tokens, 2 * inner), "bf16"), ("out", (tokens, width), "bf16"),
                            ("da", (tokens, inner), "bf16"), ("dWc", (width, inner), "f32"), ("dWb", (2 * inner, width), "f32"),
                            ("dy", (tokens, width), "bf16")):
        t[name] = torch.zeros(shape, dtype=P.TYPES[dt], device="cuda")
    for name, rows, cols in (("yq", tokens, width), ("Waq", wide, width), ("Wbq", 2 * inner, width), ("Wbt", width, 2 * inner),
                             ("Wcq", width, inner), ("Wct", inner, width), ("qq", tokens * heads, dim), ("kq", tokens * kv, dim),
                             ("gq", tokens, inner), ("uq", tokens, inner), ("aq", tokens, inner), ("yt", width, tokens),
                             ("dzt", wide, tokens), ("doq", tokens, width), ("dot", width, tokens), ("dbq", tokens, 2 * inner),
                             ("dbt", 2 * inner, tokens), ("at", inner, tokens)):
        t[name] = osa.block_buffers(rows, cols)
    return t


def block_pass(osa, t, heads, kv, dim, inner, stream=None):
    """Forward and backward of both parts over preallocated tensors; nothing in 16 bits is kept for the backward pass but h."""
    kw = dict(stream=stream)
    tokens = t["h"].shape[0]
    split = lambda z: (z[:, :heads * dim].view(tokens, heads, dim), z[:, heads * dim:(heads + kv) * dim].view(tokens, kv, dim))  # noqa: E731
    turn = dict(table=t["table"], positions=t["pos"], **kw)
    for w, q, wt in (("Wa", "Waq", None), ("Wb", "Wbq", "Wbt"), ("Wc", "Wcq", "Wct")):
        osa.opt_block_cast(t[w], codes=t[q], codes_t=t[wt] if wt else None, block_rows=128, **kw)
    osa.opt_rms_norm(t["h"], t["w"], y=t["y"], codes=t["yq"], **kw)
    osa.opt_block_matmul(t["yq"], t["Waq"], t["z"], **kw)
    osa.opt_head_norm(*split(t["z"]), t["wq"], t["wk"], q_out=t["qo"].transpose(0, 1), k_out=t["ko"].transpose(0, 1), q_codes=t["qq"],
                      k_codes=t["kq"], **turn)
    osa.opt_block_matmul(t["yq"], t["Wbq"], t["b"], **kw)
    osa.opt_gated_act(t["b"][:, :inner], t["b"][:, inner:], codes=t["aq"], gate_codes=t["gq"], up_codes=t["uq"], **kw)
    osa.opt_block_matmul(t["aq"], t["Wcq"], t["out"], **kw)
    osa.opt_block_cast(t["dout"], codes=t["doq"], codes_t=t["dot"], **kw)
    osa.opt_block_matmul(t["doq"], t["Wct"], t["da"], **kw)
    n = inner // 128
    osa.opt_gated_act_backward(t["da"], t["gq"], t["uq"], dgate_codes=(t["dbq"][0][:, :inner], t["dbq"][1][:n]),
                               dup_codes=(t["dbq"][0][:, inner:], t["dbq"][1][n:]), dgate_codes_t=(t["dbt"][0][:inner], t["dbt"][1][:, :inner]),
                               dup_codes_t=(t["dbt"][0][inner:], t["dbt"][1][:, inner:]), y_codes_t=t["at"], **kw)
    osa.opt_block_matmul(t["dot"], t["at"], t["dWc"], **kw)
    osa.opt_block_restore(t["yq"], codes_t=t["yt"], **kw)
    osa.opt_block_matmul(t["dbt"], t["yt"], t["dWb"], **kw)
    osa.opt_block_matmul(t["dbq"], t["Wbt"], t["dy"], **kw)
    dq, dk = split(t["dz"])
    osa.opt_head_norm_backward(t["dqo"], t["dko"], t["qq"], t["kq"], t["wq"], t["wk"], dq=dq, dk=dk, dweight_q=t["dwq"], dweight_k=t["dwk"], **turn)
    osa.opt_block_cast(t["dz"], codes_t=t["dzt"], **kw)
    osa.opt_block_matmul(t["dzt"], t["yt"], t["dWa"], **kw)


BLOCK_OUT = ("y", "z", "qo", "ko", "b", "out", "da", "dWc", "dWb", "dy", "dz", "dwq", "dwk", "dWa")


@pytest.mark.parametrize("tokens,heads,kv,dim,inner", [(1, 4, 1, 64, 128), (77, 4, 2, 80, 384), (300, 3, 3, 128, 640)])
def test_block_then_step(tokens, heads, kv, dim, inner):
    """Both parts of a layer as a program runs them, each operator against its
    plain form on what the one before it wrote, and the step on a gradient."""
    import torch
    import optimizer_step_amd as osa
    t = block_tensors(osa, tokens, heads, kv, dim, inner)
    block_pass(osa, t, heads, kv, dim, inner)
    H = {k: host(v) for k, v in t.items() if torch.is_tensor(v)}
    C = {k: (v[0].cpu().numpy(), v[1].cpu().numpy()) for k, v in t.items() if not torch.is_tensor(v)}
    val = lambda k, rows, cols: P.decode(C[k][0][:rows], C[k][1][:, :rows], cols)  # noqa: E731
    width, wide = heads * dim, (heads + 2 * kv) * dim
    # the heads, forward and from the codes
    z, pos = H["z"], np.arange(50, tokens + 50)
    parts = {"q": (z[:, :width].reshape(tokens, heads, dim), H["wq"], heads, slice(0, width)),
             "k": (z[:, width:width + kv * dim].reshape(tokens, kv, dim), H["wk"], kv, slice(width, width + kv * dim))}
    for k, (x, w, n, cols) in parts.items():
        want, bound = G.heads(x, w, H["table"], pos, 1e-6, dim, False)
        G.check_values(H[k + "o"].transpose(1, 0, 2), want, G.stored(want, bound, "bf16"))
        codes, scales = P.encode(x.reshape(-1, dim))
        assert np.array_equal(C[k + "q"][0][:, :dim], codes) and np.array_equal(C[k + "q"][1][:, :tokens * n], scales)
        (want, bound), (want_w, terms) = G.head_gradients(H["d" + k + "o"], val(k + "q", tokens * n, dim).reshape(x.shape), w, H["table"], pos, 1e-6, dim, False)
        G.check_values(H["dz"][:, cols].reshape(x.shape), want, G.stored(want, bound, "bf16"))
        G.check_values(H["dw" + k], want_w, (5 + sums_bound(tokens, n, dim)) * P.U32 * terms * 1.05 + 2 * P.U32 * np.abs(want_w))
    # the gated activation, forward and from the codes
    x, u = H["b"][:, :inner], H["b"][:, inner:]
    want, bound = G.gate(x, u, "silu", "bf16")
    G.check_codes(t["aq"], want, bound, tokens, inner)
    for k, v in (("gq", x), ("uq", u)):
        codes, scales = P.encode(v)
        assert np.array_equal(C[k][0][:, :inner], codes) and np.array_equal(C[k][1][:, :tokens], scales)
    grads = G.gate_gradients(H["da"], val("gq", tokens, inner), val("uq", tokens, inner), "silu", "bf16")
    n = inner // 128
    for i, (w, b) in enumerate(grads[:2]):
        cut = slice(i * inner, (i + 1) * inner)
        G.check_codes((t["dbq"][0][:, cut], t["dbq"][1][i * n:(i + 1) * n]), w, b, tokens, inner)
        G.check_codes((t["dbt"][0][cut], t["dbt"][1][:, cut]), w.T.copy(), b.T.copy(), inner, tokens)
    G.check_codes(t["at"], grads[2][0].T.copy(), grads[2][1].T.copy(), inner, tokens)
    codes, scales = P.encode(val("yq", tokens, width).T.copy())
    assert np.array_equal(C["yt"][0][:, :tokens], codes) and np.array_equal(C["yt"][1][:, :width], scales)
    # the products between them
    for out, a, b, m, n, k, dt in (("z", "yq", "Waq", tokens, wide, width, "bf16"), ("out", "aq", "Wcq", tokens, width, inner, "bf16"),
                                   ("da", "doq", "Wct", tokens, inner, width, "bf16"), ("dWc", "dot", "at", width, inner, tokens, "f32"),
                                   ("dWb", "dbt", "yt", 2 * inner, width, tokens, "f32"), ("dy", "dbq", "Wbt", tokens, width, 2 * inner, "bf16"),
                                   ("dWa", "dzt", "yt", wide, width, tokens, "f32")):
        av, bv = val(a, m, k), val(b, n, k)
        want, size = av @ bv.T, np.abs(av) @ np.abs(bv).T
        G.check_values(H[out], want, P.HALF[dt] * np.abs(want) * 1.001 + (k + 8) * 2.0 ** -23 * size + P.TINY[dt])
    # the gradients go where the step reads them
    from tests.gpu_common import fp32_close
    import oracle
    for p, g in ((t["wq"], t["dwq"]), (t["Wc"], t["dWc"])):
        before, grad = host(p).reshape(-1).copy(), host(g).reshape(-1)
        d = dict(p=p.view(-1), g=g.view(-1), **osa.state_buffers("f32", p.numel()))
        osa.opt_step_adamw([d], "f32", osa.hparams(lr=1e-2, weight_decay=0.1, step=1))
        st = oracle.state_zeros("f32", before.size)
        oracle.step("adamw", "f32", oracle.make_hp(lr=1e-2, weight_decay=0.1, step=1), before, grad, **st)
        assert fp32_close(host(d["p"]), before)


SHAPE = (4, 2, 64, 256)


def test_block_on_another_stream():
    import torch
    import optimizer_step_amd as osa
    a, b = block_tensors(osa, 130, *SHAPE), block_tensors(osa, 130, *SHAPE)
    block_pass(osa, a, *SHAPE)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream):
        for k in BLOCK_OUT:
            b[k].zero_()
        torch.cuda.synchronize()
        block_pass(osa, b, *SHAPE, stream)
        s.synchronize()
        assert all(torch.equal(a[k], b[k]) for k in BLOCK_OUT)


def test_blocks_on_two_streams_at_once():
    import torch
    import optimizer_step_amd as osa
    want = [block_tensors(osa, 200, *SHAPE, seed) for seed in (1, 50)]
    got = [block_tensors(osa, 200, *SHAPE, seed) for seed in (1, 50)]
    for t in want:
        block_pass(osa, t, *SHAPE)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for t, s in zip(got, streams):
            block_pass(osa, t, *SHAPE, s)
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(a[k], b[k]) for k in BLOCK_OUT)


def test_captured_blocks():
    """Two captured passes, replayed in turn and at once with eager work
    between, give the eager bits every time."""
    import torch
    import optimizer_step_amd as osa
    want = [block_tensors(osa, 130, *SHAPE, seed) for seed in (1, 50)]
    got = [block_tensors(osa, 130, *SHAPE, seed) for seed in (1, 50)]
    for t in want:
        block_pass(osa, t, *SHAPE)
    torch.cuda.synchronize()
    graphs = []
    for t in got:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            block_pass(osa, t, *SHAPE)
        graphs.append(g)
    other = block_tensors(osa, 64, *SHAPE, 9)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for turn in range(4):
        for t in got:
            for k in BLOCK_OUT:
                t[k].zero_()
        torch.cuda.synchronize()
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s if turn % 2 else torch.cuda.current_stream()):
                g.replay()
        block_pass(osa, other, *SHAPE)
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert all(torch.equal(a[k], b[k]) for k in BLOCK_OUT)
