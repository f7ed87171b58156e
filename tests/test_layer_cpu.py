"""Host-side checks of the operators between a layer's products that need no
GPU: refusals of the C entry points (made-up addresses: every refused call ends
before any device work) and of the binding, workspace sizes, and the plain forms
the GPU tests compare with."""
import ctypes
import os

import numpy as np
import pytest
import torch

from tests import layer_plain as G
from tests import pass_plain as P

EINVAL, EUNSUP, EALIGN = -1, -2, -3


@pytest.fixture(scope="module")
def L():
    import optimizer_step_amd as osa
    if not os.path.exists(osa.LIB_PATH):
        from optimizer_step_amd import build
        build.build()
    return osa


def codes(L, codes=1 << 20, ld=128, scales=1 << 21, lds=64):
    return L.OptCodes(codes or None, ld, scales or None, lds)


BAD_CODES = [(dict(codes=(1 << 20) + 8), EALIGN), (dict(ld=120), EALIGN), (dict(ld=96), EINVAL), (dict(scales=0), EINVAL),
             (dict(scales=(1 << 21) + 2), EALIGN), (dict(lds=6), EALIGN), (dict(lds=0), EINVAL)]


def gate(L, **kw):
    a = dict(rows=4, cols=100, dtype=1, act=0, gate=4096, ldg=100, up=8192, ldu=100, y=1 << 17, ldy=100, q=L.OptCodes(),
             gate_q=L.OptCodes(), up_q=L.OptCodes())
    a.update(kw)
    return L.lib().opt_gated_act(ctypes.byref(L.OptGate(**a)), None)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), EINVAL), (dict(cols=1 << 31), EINVAL), (dict(dtype=3), EINVAL), (dict(act=2), EINVAL), (dict(act=-1), EINVAL),
    (dict(gate=None), EINVAL), (dict(up=None), EINVAL), (dict(y=None), EINVAL), (dict(ldg=99), EINVAL), (dict(ldu=0), EINVAL),
    (dict(ldy=50), EINVAL), (dict(gate=4097), EALIGN), (dict(up=8194, dtype=0), EALIGN), (dict(y=(1 << 17) + 1), EALIGN),
    (dict(ldg=1 << 45), EINVAL),
])
def test_gate_refusals(L, kw, status):
    assert gate(L, **kw) == status
    assert L.opt_last_error()


def gate_grad(L, coded=False, **kw):
    a = dict(rows=4, cols=100, dtype=1, act=0, dy=4096, lddy=100, gate=None if coded else 8192, ldg=100, up=None if coded else 12288,
             ldu=100, dgate=1 << 17, lddg=100, dup=1 << 18, lddu=100)
    for k in ("gate_q", "up_q", "dgate_q", "dup_q", "dgate_t", "dup_t", "y_t"):
        a[k] = codes(L, codes=1 << 22) if coded and k in ("gate_q", "up_q") else L.OptCodes()
    a.update(kw)
    return L.lib().opt_gated_act_backward(ctypes.byref(L.OptGateGrad(**a)), None)


@pytest.mark.parametrize("coded", [False, True])
@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), EINVAL), (dict(cols=-1), EINVAL), (dict(dtype=7), EINVAL), (dict(act=3), EINVAL), (dict(dy=None), EINVAL),
    (dict(dy=4097), EALIGN), (dict(lddy=99), EINVAL), (dict(dgate=None, dup=None), EINVAL), (dict(dgate=1 << 18), EINVAL),
    (dict(lddg=9), EINVAL), (dict(lddu=9), EINVAL), (dict(dup=(1 << 18) + 1), EALIGN),
])
def test_gate_backward_refusals(L, coded, kw, status):
    assert gate_grad(L, coded, **kw) == status
    assert L.opt_last_error()


def test_gate_backward_takes_one_kind_of_input(L):
    for kw in (dict(gate=None), dict(up=None), dict(gate_q=codes(L)), dict(up_q=codes(L)), dict(gate=None, up=None)):
        assert gate_grad(L, **kw) == EINVAL
    for kw in (dict(gate_q=L.OptCodes()), dict(up_q=L.OptCodes()), dict(gate=8192)):
        assert gate_grad(L, True, **kw) == EINVAL


@pytest.mark.parametrize("kw,status", BAD_CODES)
def test_code_buffer_refusals(L, kw, status):
    for k in ("q", "gate_q", "up_q"):
        assert gate(L, **{k: codes(L, **kw)}) == status
    for k in ("gate_q", "up_q", "dgate_q", "dup_q"):
        assert gate_grad(L, True, **{k: codes(L, **kw)}) == status
    assert restore(L, q=codes(L, **kw)) == status
    assert heads(L, q=dict(codes=codes(L, **kw)), tokens=2, q_heads=2, dim=100) == status
    assert heads_grad(L, True, q=dict(codes=codes(L, **kw)), tokens=2, q_heads=2, dim=100) == status


@pytest.mark.parametrize("kw,status", [
    (dict(codes=(1 << 20) + 8), EALIGN), (dict(ld=8), EALIGN), (dict(ld=0), EINVAL), (dict(scales=0), EINVAL), (dict(lds=96), EINVAL)])
def test_transposed_code_buffer_refusals(L, kw, status):
    good = dict(ld=16, lds=100)
    for k in ("dgate_t", "dup_t", "y_t"):
        assert gate_grad(L, **{k: codes(L, **{**good, **kw})}) == status
    assert restore(L, qt=codes(L, **{**good, **kw})) == status


def restore(L, **kw):
    a = dict(rows=4, cols=100, q=codes(L, codes=1 << 22), x=4096, ldx=100, dtype=1, reserved=0, qt=L.OptCodes())
    a.update(kw)
    return L.lib().opt_block_restore(ctypes.byref(L.OptRestore(**a)), None)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), EINVAL), (dict(cols=1 << 31), EINVAL), (dict(dtype=3), EINVAL), (dict(x=None), EINVAL), (dict(x=4097), EALIGN),
    (dict(ldx=99), EINVAL),
])
def test_restore_refusals(L, kw, status):
    assert restore(L, **kw) == status
    assert L.opt_last_error()


def test_restore_needs_two_matrices(L):
    assert restore(L, rows=100, q=codes(L, codes=1 << 22, lds=100), qt=codes(L, codes=1 << 22, lds=100)) == EINVAL
    assert restore(L, q=L.OptCodes()) == EINVAL


def table_of(L, **kw):
    a = dict(cos_sin=1 << 30, rows=50, ld=64, positions=1 << 31, position_bits=64, reserved=0)
    a.update(kw)
    return L.OptHeadTable(**a)


def heads(L, tokens=5, q_heads=3, dim=64, rot=64, q=None, k=None, table=None, **kw):
    def one(n, at, more):
        a = dict(heads=n, x=at, x_token=n * dim, x_head=dim, weight=at + (1 << 12), y=at + (1 << 13), y_token=n * dim, y_head=dim,
                 codes=L.OptCodes())
        a.update(more or {})
        return L.OptHeadSet(**a)

    a = dict(tokens=tokens, dim=dim, rot=rot, dtype=1, w_dtype=1, interleaved=0, reserved=0, eps=1e-6, table=table_of(L, **(table or {})),
             q=one(q_heads, 1 << 14, q), k=one(1, 1 << 16, k))
    a.update(kw)
    return L.lib().opt_head_norm(ctypes.byref(L.OptHeads(**a)), None)


HEADS = [
    (dict(tokens=-1), EINVAL), (dict(tokens=1 << 31), EINVAL), (dict(dim=0), EINVAL), (dict(dim=513, rot=64), EUNSUP), (dict(rot=63), EINVAL),
    (dict(rot=66), EINVAL), (dict(rot=-2), EINVAL), (dict(dtype=3), EINVAL), (dict(w_dtype=5), EINVAL), (dict(interleaved=2), EINVAL),
    (dict(eps=-1.0), EINVAL), (dict(eps=float("nan")), EINVAL), (dict(eps=float("inf")), EINVAL),
    (dict(table=dict(cos_sin=None)), EINVAL), (dict(table=dict(cos_sin=(1 << 30) + 2)), EALIGN), (dict(table=dict(rows=0)), EINVAL),
    (dict(table=dict(ld=63)), EINVAL), (dict(table=dict(position_bits=16)), EINVAL), (dict(table=dict(positions=(1 << 31) + 4)), EALIGN),
    (dict(table=dict(positions=None, rows=4)), EINVAL), (dict(table=dict(rows=1 << 31)), EINVAL),
    (dict(q=dict(heads=-1)), EINVAL), (dict(k=dict(heads=65536)), EINVAL), (dict(q=dict(x=None)), EINVAL), (dict(k=dict(x=4097)), EALIGN),
    (dict(q=dict(x_token=-64)), EINVAL), (dict(q=dict(x_head=-64)), EINVAL), (dict(q=dict(x_token=1 << 45)), EINVAL),
    (dict(q=dict(weight=4097)), EALIGN),
]


@pytest.mark.parametrize("kw,status", HEADS + [
    (dict(q=dict(y=None)), EINVAL), (dict(k=dict(y=4097)), EALIGN), (dict(q=dict(y_head=63)), EINVAL), (dict(q=dict(y_token=191)), EINVAL),
    (dict(q=dict(y_head=0)), EINVAL), (dict(k=dict(y_token=0)), EINVAL), (dict(q=dict(y_token=64, y_head=5 * 64 - 1)), EINVAL),
])
def test_head_refusals(L, kw, status):
    assert heads(L, **kw) == status
    assert L.opt_last_error()


def heads_grad(L, coded=False, tokens=5, q_heads=3, dim=64, rot=64, q=None, k=None, table=None, **kw):
    def one(n, at, more):
        a = dict(heads=n, dy=at, dy_token=n * dim, dy_head=dim, x=None if coded else at + (1 << 11), x_token=n * dim, x_head=dim,
                 codes=codes(L, codes=1 << 22) if coded else L.OptCodes(), weight=at + (1 << 12), dx=at + (1 << 13), dx_token=n * dim,
                 dx_head=dim, dweight=at + (3 << 12))
        a.update(more or {})
        return L.OptHeadGradSet(**a)

    a = dict(tokens=tokens, dim=dim, rot=rot, dtype=1, w_dtype=1, interleaved=0, accumulate=0, eps=1e-6, table=table_of(L, **(table or {})),
             q=one(q_heads, 1 << 14, q), k=one(1, 1 << 16, k), workspace=1 << 24, workspace_bytes=1 << 22)
    a.update(kw)
    return L.lib().opt_head_norm_backward(ctypes.byref(L.OptHeadsGrad(**a)), None)


@pytest.mark.parametrize("kw,status", HEADS + [
    (dict(accumulate=2), EINVAL), (dict(workspace=None), EINVAL), (dict(workspace=(1 << 24) + 8), EALIGN), (dict(workspace_bytes=100), EINVAL),
    (dict(q=dict(dy=None)), EINVAL), (dict(q=dict(dx=None)), EINVAL), (dict(k=dict(dx=4097)), EALIGN), (dict(q=dict(dx_head=63)), EINVAL),
    (dict(q=dict(dx_token=100)), EINVAL), (dict(q=dict(dy_token=-1)), EINVAL), (dict(q=dict(dweight=(1 << 20) + 2)), EALIGN),
    (dict(q=dict(dx=(1 << 14) + (1 << 11))), EINVAL), (dict(q=dict(dweight=1 << 20), k=dict(dweight=1 << 20)), EINVAL),
])
def test_head_backward_refusals(L, kw, status):
    assert heads_grad(L, **kw) == status
    assert L.opt_last_error()


def test_head_backward_takes_one_kind_of_input(L):
    assert heads_grad(L, q=dict(x=None)) == EINVAL
    assert heads_grad(L, q=dict(x=None, codes=codes(L, codes=1 << 22))) == EINVAL
    assert heads_grad(L, q=dict(codes=codes(L, codes=1 << 22))) == EINVAL
    assert heads_grad(L, True, k=dict(x=1 << 26)) == EINVAL


def test_null_records_and_empty_calls(L):
    for fn in ("opt_gated_act", "opt_gated_act_backward", "opt_block_restore", "opt_head_norm", "opt_head_norm_backward"):
        assert getattr(L.lib(), fn)(None, None) == EINVAL
    for kw in (dict(rows=0), dict(cols=0)):
        assert gate(L, gate=None, y=None, **kw) == 0
        assert gate_grad(L, dy=None, **kw) == 0
        assert restore(L, x=None, **kw) == 0
    assert heads(L, tokens=0, q=dict(x=None)) == 0
    assert heads(L, q=dict(heads=0, x=None), k=dict(heads=0)) == 0
    assert heads_grad(L, tokens=0, q=dict(dweight=None), k=dict(dweight=None)) == 0


def test_workspace_sizes(L):
    assert L.opt_head_norm_workspace(0, 4, 4, 64) == 0 and L.opt_head_norm_workspace(4, 0, 0, 64) == 0
    for a in ((1, 1, 0, 1), (7, 32, 8, 128), (100000, 7, 7, 512)):
        n = L.opt_head_norm_workspace(*a)
        assert n > 0 and n % (8 * a[3]) == 0
    for bad in ((-1, 1, 1, 64), (5, -1, 1, 64), (5, 1, 65536, 64), (5, 1, 1, 0), (5, 1, 1, 513)):
        with pytest.raises(L.OptError):
            L.opt_head_norm_workspace(*bad)


def test_binding_refusals(L, monkeypatch):
    """The binding refuses host tensors, and arguments of other shapes and types before it makes any call."""
    monkeypatch.setattr(L, "_device", lambda: -1)       # a host tensor's device number, so that the checks behind it are reached
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    q = L.block_buffers(4, 128, device="cpu")
    h, w, tab = torch.zeros(4, 2, 64, dtype=torch.bfloat16), torch.ones(64), torch.zeros(9, 64)
    for call, text in (
            (lambda: L.opt_gated_act(x[:, :128], x[:, :100], y=x[:, :128]), "elements"),
            (lambda: L.opt_gated_act(x[:, :128], None, y=x[:, :128]), "up"),
            (lambda: L.opt_gated_act(x[:, :128], x[:, 128:].float(), y=x[:, :128]), "float32"),
            (lambda: L.opt_gated_act(x[:, :128], x[:, 128:], act="relu"), "act"),
            (lambda: L.opt_gated_act(x[:, :128], x[:, 128:], codes=L.block_buffers(4, 256, device="cpu")), "codes"),
            (lambda: L.opt_gated_act_backward(x[:, :128], q, x[:, :128], dgate=x[:, :128]), "two pairs"),
            (lambda: L.opt_gated_act_backward(x[:, :128], None, None, dgate=x[:, :128]), "two pairs"),
            (lambda: L.opt_gated_act_backward(x[:, :128], q, q, dgate_codes_t=q), "codes"),
            (lambda: L.opt_block_restore(q), "neither"),
            (lambda: L.opt_block_restore(q, out=torch.zeros(5, 128)), "rows"),
            (lambda: L.opt_block_restore(q, out=torch.zeros(4, 100)), "codes"),
            (lambda: L.opt_head_norm(h[0], None, q_out=h[0]), "tokens"),
            (lambda: L.opt_head_norm(h, None), "q_out"),
            (lambda: L.opt_head_norm(h, h[:3], q_out=h, k_out=h[:3]), "k must"),
            (lambda: L.opt_head_norm(h, None, w[:60], q_out=h), "weight"),
            (lambda: L.opt_head_norm(h, h, w, w.bfloat16(), q_out=h, k_out=h), "one type"),
            (lambda: L.opt_head_norm(h, None, w, q_out=h.float()), "float32"),
            (lambda: L.opt_head_norm(h.transpose(1, 2), None, q_out=h.transpose(1, 2)), "contiguous"),
            (lambda: L.opt_head_norm(h, None, w, table=tab.double(), q_out=h), "table"),
            (lambda: L.opt_head_norm(h, None, w, table=tab, positions=torch.zeros(3, dtype=torch.int64), q_out=h), "positions"),
            (lambda: L.opt_head_norm(h, None, w, table=tab, positions=torch.zeros(4, dtype=torch.int16), q_out=h), "positions"),
            (lambda: L.opt_head_norm(h, None, w, q_out=h, q_codes=L.block_buffers(8, 32, device="cpu")), "q_codes"),
            (lambda: L.opt_head_norm_backward(h, None, h, None, w, dq=None), "dq"),
            (lambda: L.opt_head_norm_backward(h, None, h, None, w, dq=h, dk=h), "dk_out"),
            (lambda: L.opt_head_norm_backward(h, h[:, :1], h, h, w, w, dq=h, dk=h[:, :1]), "k must"),
            (lambda: L.opt_head_norm_backward(h, None, h, None, w, dq=h, dweight_q=w.double()), "dweight_q")):
        with pytest.raises(ValueError, match=text):
            call()
    monkeypatch.setattr(L, "_device", lambda: 0)
    for call in (lambda: L.opt_gated_act(x, x, y=x), lambda: L.opt_gated_act_backward(x, x, x, dgate=x), lambda: L.opt_block_restore(q, out=x),
                 lambda: L.opt_head_norm(h, None, q_out=h), lambda: L.opt_head_norm_backward(h, None, h, None, dq=h)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


# ---- the plain forms --------------------------------------------------------


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_activations_are_torchs(act):
    x = np.concatenate([np.random.RandomState(0).randn(500) * 4, [0.0, -0.0, 20.0, -20.0, 300.0, -300.0]])
    t = torch.from_numpy(x)
    want = torch.nn.functional.silu(t) if act == "silu" else torch.nn.functional.gelu(t, approximate="tanh")
    got, _ = G.gate(x, np.ones_like(x), act, "f32")
    assert np.allclose(got, want.numpy(), rtol=1e-12, atol=1e-13)


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gate_gradients_against_differences(act):
    rng = np.random.RandomState(1)
    x, u, t = rng.randn(40) * 3, rng.randn(40), rng.randn(40)
    (dg, _), (du, _), (y, _) = G.gate_gradients(t, x, u, act, "f32")
    d = 1e-6
    f = lambda x, u: G.gate(x, u, act, "f32")[0] * t  # noqa: E731
    assert np.allclose((f(x + d, u) - f(x - d, u)) / (2 * d), dg, atol=1e-8)
    assert np.allclose((f(x, u + d) - f(x, u - d)) / (2 * d), du, atol=1e-8)
    assert np.allclose(y * t, f(x, u), atol=1e-14)


@pytest.mark.parametrize("rot,interleaved", [(0, False), (6, False), (6, True), (10, False), (10, True)])
def test_head_gradients_against_differences(rot, interleaved):
    rng = np.random.RandomState(2)
    x, w, t = rng.randn(3, 2, 10), rng.rand(10) + 0.5, rng.randn(3, 2, 10)
    tab, pos = G.table(20, max(rot, 2)).astype(np.float64), np.array([19, 0, 7])
    (dx, _), (dw, _) = G.head_gradients(t, x, w, tab, pos, 1e-3, rot, interleaved)
    f = lambda x, w: float((G.heads(x, w, tab, pos, 1e-3, rot, interleaved)[0] * t).sum())  # noqa: E731
    d = 1e-6
    for at in ((0, 0, 0), (1, 1, 3), (2, 0, 9), (0, 1, 5)):
        e = np.zeros_like(x)
        e[at] = d
        assert abs((f(x + e, w) - f(x - e, w)) / (2 * d) - dx[at]) < 1e-8
    for j in range(10):
        e = np.zeros(10)
        e[j] = d
        assert abs((f(x, w + e) - f(x, w - e)) / (2 * d) - dw[j]) < 1e-7


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_keeps_lengths_and_distances(interleaved):
    """A turned pair keeps its length, and a query's product with a key depends on the distance alone."""
    rng = np.random.RandomState(3)
    q, k = rng.randn(1, 1, 16), rng.randn(1, 1, 16)
    a = np.arange(40)[:, None] * 10000.0 ** (-np.arange(0, 16, 2) / 16)
    tab = np.concatenate([np.cos(a), np.sin(a)], 1)
    at = lambda x, p: G.turn(x, tab, np.array([p]), 16, interleaved)[0]  # noqa: E731
    assert np.isclose((at(q, 11) ** 2).sum(), (q ** 2).sum())
    assert np.isclose((at(q, 11) * at(k, 4)).sum(), (at(q, 37) * at(k, 30)).sum())
    assert np.allclose(G.turn(at(q, 9), tab, np.array([9]), 16, interleaved, back=True)[0], q)


def test_rotation_table(L):
    t = L.rotation_table(300, 24, base=5000.0, device="cpu")
    assert t.shape == (300, 24) and t.dtype == torch.float32
    assert np.abs(t.numpy() - G.table(300, 24, 5000.0)).max() <= 2.0 ** -24


def test_code_check_catches_mistakes():
    """The GPU tests' comparison of codes refuses a moved code and a wrong scale (planted here, on the CPU)."""
    rng = np.random.RandomState(4)
    x = rng.randn(5, 200)
    q, s = P.encode(x)
    buf = np.zeros((5, 208), np.uint8)
    buf[:, :200] = q
    sc = np.zeros((2, 8), np.uint8)
    sc[:, :5] = s
    pair = lambda: (torch.from_numpy(buf.copy()), torch.from_numpy(sc.copy()))  # noqa: E731
    G.check_codes(pair(), x, np.zeros_like(x), 5, 200)
    for at, to in (((2, 7), buf[2, 7] ^ 1), ((0, 0), buf[0, 0] ^ 0x80), ((4, 205), 1)):
        p = pair()
        p[0][at] = int(to)
        with pytest.raises(AssertionError):
            G.check_codes(p, x, np.zeros_like(x), 5, 200)
    for d in (-1, 1):
        p = pair()
        p[1][1, 3] += d
        with pytest.raises(AssertionError):
            G.check_codes(p, x, np.zeros_like(x), 5, 200)


def test_packed_head_record(L):
    """The binding's packed opt_heads has the fields of its ctypes class, in their places."""
    values = [7, 1, 2, 3, 4, 5, 6, 0.5, 11, 12, 13, 14, 15, 16, *range(20, 44)]
    r = L.OptHeads.from_buffer_copy(L._HEADS.pack(*values))

    def flat(s):
        for name, kind in s._fields_:
            v = getattr(s, name)
            yield from flat(v) if isinstance(v, ctypes.Structure) else [v]

    assert list(flat(r)) == values
