"""GPU tests of the operators between a layer's products at the ends of their
ranges: values that are not finite, and what they may reach."""
import numpy as np
import pytest

from tests import layer_plain as G
from tests import pass_plain as P
from tests.test_gpu_layer import coded, gpu, head_data, head_out, laid  # noqa: F401 (gpu: a fixture)
from tests.test_gpu_pass import dev, host

pytestmark = pytest.mark.gpu

# dim, rot, neighbouring pairs: part of a head turned, for each way a pair is found (whole and unfilled lanes, by lanes, within a
# lane, element by element, an end inside a lane's eight), and nothing turned
PARTS = [(128, 64, False), (96, 64, False), (64, 32, True), (64, 12, True), (80, 6, True), (128, 20, False), (100, 20, False), (7, 4, False),
         (7, 4, True), (128, 0, False), (100, 0, False)]


@pytest.mark.parametrize("dim,rot,near", PARTS)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_infinity_beyond_the_rotation(dim, rot, near, dtype):
    """An infinite element or weight that does not turn reaches no other element."""
    import torch
    import optimizer_step_amd as osa
    x = head_data(dim, 4, 5, dim, dtype)
    x[0, 0, rot + 1] = np.inf                       # its neighbour does not turn either
    x[1, 4, dim - 1] = -np.inf
    w = P.rounded(0.5 + np.random.RandomState(dim).rand(dim), dtype)
    tab, pos = G.table(50, max(rot, 2)), np.array([3, 9, 20, 49])
    kw = dict(table=torch.from_numpy(tab).cuda() if rot else None, positions=torch.from_numpy(pos).cuda(), interleaved=near)
    for at in (None, rot + 1, dim - 1, 0):          # an infinite weight too
        v = w.copy()
        if at is not None:
            v[at] = np.inf
        y = head_out(4, 5, dim, dtype, "packed")
        osa.opt_head_norm(laid(x, dtype, "packed"), None, dev(v, dtype), q_out=y, **kw)
        with np.errstate(invalid="ignore"):
            want, bound = G.heads(x, v, tab, pos, 1e-6, rot, near)
        G.check_values(host(y), want, np.where(np.isfinite(want), G.stored(want, bound, dtype), 0))


@pytest.mark.parametrize("dim,rot,near", PARTS)
def test_tiny_heads_beyond_the_rotation(dim, rot, near):
    """Where r is infinite an element that does not turn is infinite, or NaN if it is zero."""
    import torch
    import optimizer_step_amd as osa
    x = np.where(np.arange(2 * 3 * dim).reshape(2, 3, dim) % 3 == 0, -1e-40, 1e-40).astype(np.float32)
    x[0, 1, dim - 1] = 0
    y = head_out(2, 3, dim, "f32", "packed")
    tab = torch.from_numpy(G.table(9, max(rot, 2))).cuda() if rot else None
    osa.opt_head_norm(laid(x, "f32", "packed"), None, table=tab, eps=0.0, interleaved=near, q_out=y)
    want = np.where(x == 0, np.nan, np.copysign(np.inf, x))[..., rot:]
    assert np.array_equal(host(y)[..., rot:], want, equal_nan=True)


@pytest.mark.parametrize("dim,rot,near", PARTS)
@pytest.mark.parametrize("dtype,from_codes", [("f32", False), ("bf16", True), ("f16", False)])
def test_infinite_gradient_beyond_the_rotation(dim, rot, near, dtype, from_codes):
    """A gradient that is not finite, of an element that does not turn, reaches its own head's dx and its own dweight alone."""
    import torch
    import optimizer_step_amd as osa
    x, dy = head_data(dim, 6, 3, dim, dtype), head_data(dim + 1, 6, 3, dim, dtype, 0.1)
    dy[0, 0, rot + 1] = np.inf
    dy[1, 2, dim - 1] = np.nan
    dy[2, 1, rot + 1] = np.inf
    x[0, 0, rot + 1] = x[2, 1, rot + 1] = 0.75      # the two infinities have one sign in dweight
    w = P.rounded(0.5 + np.random.RandomState(dim).rand(dim), "f32")
    tab, pos = G.table(50, max(rot, 2)), np.array([3, 9, 20, 49, 1, 7])
    if from_codes:
        xin, held = coded(x.reshape(-1, dim))
        x = held.reshape(x.shape)
    else:
        xin = laid(x, dtype, "packed")
    dx, dw = head_out(6, 3, dim, dtype, "packed"), torch.zeros(dim, device="cuda")
    osa.opt_head_norm_backward(laid(dy, dtype, "packed"), None, xin, None, dev(w, "f32"), interleaved=near, dq=dx, dweight_q=dw,
                               table=torch.from_numpy(tab).cuda() if rot else None, positions=torch.from_numpy(pos).cuda())
    with np.errstate(invalid="ignore"):
        (want, bound), (want_w, terms) = G.head_gradients(dy, x, w, tab, pos, 1e-6, rot, near)
    bad = np.arange(dim) == dim - 1
    assert np.isnan(want_w[bad]).all() and np.isfinite(want_w[~bad]).sum() == dim - 2 and np.isinf(want_w[rot + 1])
    G.check_values(host(dx), want, np.where(np.isfinite(want), G.stored(want, bound, dtype), 0))
    # dn and x r to 4 units, r to 1; 18 heads' terms added
    G.check_values(host(dw), want_w, np.where(np.isfinite(want_w), (5 + 18) * P.U32 * terms * 1.05, 0))


@pytest.mark.parametrize("dim,rot,near,dtype,from_codes", [(8, 0, False, "f32", False), (7, 0, False, "bf16", False), (8, 2, True, "f16", True),
                                                           (64, 64, False, "bf16", True), (128, 32, False, "bf16", False)])
def test_long_sums_of_dweight(dim, rot, near, dtype, from_codes):
    """dweight's error does not grow with the tokens: ones first, then terms of which a binary32 sum of one would take none."""
    import torch
    import optimizer_step_amd as osa
    waves, each = 4096, 256
    tokens, small = waves * each, 2.0 ** -25 if dtype != "f16" else 2.0 ** -24
    dy = torch.full((tokens, 1, dim), small, dtype=P.TYPES[dtype], device="cuda")
    dy[:waves] = 1
    x = torch.ones(tokens, 1, dim, dtype=P.TYPES[dtype], device="cuda")
    xin = x
    if from_codes:
        xin = osa.block_buffers(tokens, dim)
        osa.opt_block_cast(x.view(tokens, dim), codes=xin)
    dx = [torch.empty_like(x) for _ in range(2)]
    dw = [torch.full((dim,), -5.0, device="cuda") for _ in range(2)]
    table = osa.rotation_table(1, rot) if rot else None            # position 0: cos 1, sin 0
    osa.opt_head_norm_backward(dy, dy, xin, xin, table=table, positions=torch.zeros(tokens, dtype=torch.int32, device="cuda"), eps=0.0,
                               interleaved=near, dq=dx[0], dk=dx[1], dweight_q=dw[0], dweight_k=dw[1])
    want = waves * (1 + (each - 1) * small)                        # r = 1: every term is dy's, exactly
    for w in dw:
        # three additions in binary32 at most before a sum is widened, half a step of 1 each; the result's rounding
        assert bool(((w.double() - want).abs() <= 4 * P.U32 * want).all()), float(w[0])


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_far_gates_in_32_bits(act, monkeypatch):
    """Where sigma is below the normal numbers, x sigma still is one: 32-bit results keep their units down to the subnormals."""
    import torch
    import optimizer_step_amd as osa
    monkeypatch.setattr(G, "FLUSH", 2.0 ** -148)        # s, sigma and their products each off by half a subnormal at most
    x = np.linspace(*((-104, -60) if act == "silu" else (-10.7, -8)), 8192).astype(np.float32).reshape(16, 512)
    u, dy = (np.random.RandomState(i).uniform(0.5, 2, x.shape).astype(np.float32) for i in (1, 2))
    want, bound = G.gate(x, u, act, "f32")
    tail = (np.abs(want) > 2.0 ** -126) & (np.abs(want / u / x) < 2.0 ** -126)
    assert tail.sum() > 100                             # normal results of a sigma that is none
    y, dg, du = (torch.empty(16, 512, device="cuda") for _ in range(3))
    osa.opt_gated_act(dev(x, "f32"), dev(u, "f32"), act, y=y)
    osa.opt_gated_act_backward(dev(dy, "f32"), dev(x, "f32"), dev(u, "f32"), act, dgate=dg, dup=du)
    (wg, bg), (wu, bu), _ = G.gate_gradients(dy, x, u, act, "f32")
    for got, w, b in ((y, want, bound), (dg, wg, bg), (du, wu, bu)):
        G.check_values(host(got), w, G.stored(w, b, "f32"))
    # the tiles too
    t = osa.block_buffers(512, 16)
    osa.opt_gated_act_backward(dev(dy, "f32"), dev(x, "f32"), dev(u, "f32"), act, dgate=(a := torch.empty_like(dg)), dup=(b := torch.empty_like(du)),
                               y_codes_t=t)
    assert torch.equal(a, dg) and torch.equal(b, du)


def test_slope_beside_a_saturated_gate():
    """16-bit dgate = u s'(x) rounds as the exact value does where that is 7 to 25 units of binary32 from a tie: its
    binary32 form is off by 3 (1 + e, the reciprocal), 0.7 (the tail s (1 - sigma) p', below 0.013 and off by 50 units
    of itself), 1 (their sum) and 1 (the product with u).  1 - sigma formed by a subtraction would be off by 3 units of
    1, and the tail by 10 to 25 times as many."""
    import torch
    import optimizer_step_amd as osa
    x = np.arange(3, 4.5, 2.0 ** -8)
    u = np.arange(1, 2, 2.0 ** -10)
    x, u = (v.reshape(-1) for v in np.meshgrid(x, u))
    (want, _), _, _ = G.gate_gradients(np.ones_like(x), x, u, "gelu", "f16")
    step = 2.0 ** (np.floor(np.log2(want)) - 10)
    off = np.abs(want / step - np.floor(want / step) - 0.5) * step / want / P.U32
    near = (off > 7) & (off < 25)
    assert near.sum() > 1000
    x, u, want = (v[near][:near.sum() // 128 * 128].reshape(-1, 128) for v in (x, u, want))
    dg, tile = (torch.empty(*x.shape, dtype=torch.float16, device="cuda") for _ in range(2))
    one = torch.ones_like(dg)
    osa.opt_gated_act_backward(one, dev(x, "f16"), dev(u, "f16"), "gelu", dgate=dg)
    osa.opt_gated_act_backward(one, dev(x, "f16"), dev(u, "f16"), "gelu", dgate=tile, y_codes_t=osa.block_buffers(128, x.shape[0]))
    assert np.array_equal(host(dg), want.astype(np.float16).astype(np.float32)) and torch.equal(dg, tile)
