"""Host-side checks of the training-pass operators that need no GPU: refusals
of the C entry points (made-up addresses: every refused call ends before any
device work), workspace sizes, the record layouts, and the plain forms the GPU
tests compare with."""
import ctypes
import os

import numpy as np
import pytest
import torch

from tests import pass_plain as P

EINVAL, EUNSUP, EALIGN = -1, -2, -3


@pytest.fixture(scope="module")
def L():
    import optimizer_step_amd as osa
    if not os.path.exists(osa.LIB_PATH):
        from optimizer_step_amd import build
        build.build()
    return osa


def _codes(L, codes=1 << 20, ld=128, scales=1 << 21, lds=64):
    return L.OptCodes(codes or None, ld, scales or None, lds)


def _dropout(L, x=4096, res=None, out=8192, n=100, dtype=1, p=0.5, base=0):
    return L.lib().opt_dropout(x, res, out, n, dtype, p, 1, 2, base, None)


@pytest.mark.parametrize("kw,status", [
    (dict(p=-0.1), EINVAL), (dict(p=1.5), EINVAL), (dict(p=float("nan")), EINVAL), (dict(n=-1), EINVAL),
    (dict(n=(1 << 46) + 1), EINVAL), (dict(dtype=3), EINVAL), (dict(x=None), EINVAL), (dict(out=None), EINVAL),
    (dict(base=4), EINVAL), (dict(base=-8), EINVAL), (dict(base=1 << 60), EINVAL), (dict(x=4097), EALIGN),
    (dict(out=4098, dtype=0), EALIGN), (dict(res=4099), EALIGN),
])
def test_dropout_refusals(L, kw, status):
    assert _dropout(L, **kw) == status
    assert L.opt_last_error()


def _norm(L, q=None, **kw):
    a = dict(rows=4, cols=100, dtype=1, w_dtype=1, x=4096, ldx=100, residual=None, ldr=0, weight=1 << 16, h=None, ldh=0,
             y=1 << 17, ldy=100, eps=1e-6)
    a.update(kw)
    r = L.OptNorm(q=q or L.OptCodes(), **a)
    return L.lib().opt_rms_norm(ctypes.byref(r), None)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), EINVAL), (dict(cols=-5), EINVAL), (dict(rows=1 << 31), EINVAL), (dict(cols=32769, ldx=32769), EUNSUP),
    (dict(dtype=9), EINVAL), (dict(w_dtype=-1), EINVAL), (dict(x=None), EINVAL), (dict(weight=None), EINVAL),
    (dict(y=None), EINVAL), (dict(ldx=99), EINVAL), (dict(ldy=0), EINVAL), (dict(ldx=1 << 45), EINVAL),
    (dict(eps=-1e-6), EINVAL), (dict(eps=float("nan")), EINVAL), (dict(eps=float("inf")), EINVAL),
    (dict(x=4097), EALIGN), (dict(dtype=0, y=4098), EALIGN), (dict(w_dtype=0, weight=4098), EALIGN),
    (dict(h=1 << 17, ldh=100), EINVAL), (dict(residual=4096, ldr=3), EINVAL),
])
def test_norm_refusals(L, kw, status):
    assert _norm(L, **kw) == status
    assert L.opt_last_error()


@pytest.mark.parametrize("kw,status", [
    (dict(codes=(1 << 20) + 8), EALIGN), (dict(ld=120), EALIGN), (dict(ld=96), EINVAL), (dict(scales=0), EINVAL),
    (dict(scales=(1 << 21) + 2), EALIGN), (dict(lds=6), EALIGN), (dict(lds=0), EINVAL),
])
def test_code_buffer_refusals(L, kw, status):
    assert _norm(L, q=_codes(L, **kw)) == status
    r = L.OptCast(4, 100, 4096, 100, 1, 1, _codes(L, **kw), L.OptCodes())
    assert L.lib().opt_block_cast(ctypes.byref(r), None) == status
    for sides in ("a", "b"):
        q = {"a": _codes(L, codes=1 << 22), "b": _codes(L, codes=1 << 23)}
        q[sides] = _codes(L, **kw)
        r = L.OptProduct(4, 4, 112, q["a"], q["b"], 4096, 4, 1, 0)
        assert L.lib().opt_block_matmul(ctypes.byref(r), None) == status


def _grad(L, **kw):
    a = dict(rows=4, cols=100, dtype=1, w_dtype=1, dy=4096, lddy=100, h=8192, ldh=100, weight=1 << 16, dh=None, lddh=0,
             dx=1 << 17, lddx=100, dweight=1 << 18, accumulate=0, reserved=0, eps=1e-6, workspace=1 << 19, workspace_bytes=1 << 16)
    a.update(kw)
    return L.lib().opt_rms_norm_backward(ctypes.byref(L.OptNormGrad(**a)), None)


@pytest.mark.parametrize("kw,status", [
    (dict(dy=None), EINVAL), (dict(h=None), EINVAL), (dict(dx=None), EINVAL), (dict(weight=None), EINVAL),
    (dict(workspace=None), EINVAL), (dict(workspace_bytes=8), EINVAL), (dict(workspace=(1 << 19) + 4), EALIGN),
    (dict(accumulate=2), EINVAL), (dict(dx=8192), EINVAL), (dict(lddx=50), EINVAL), (dict(lddy=50), EINVAL),
    (dict(cols=40000), EUNSUP), (dict(rows=-4), EINVAL), (dict(dtype=5), EINVAL), (dict(eps=-1.0), EINVAL),
    (dict(dweight=(1 << 18) + 2), EALIGN), (dict(dh=4096, lddh=1), EINVAL),
])
def test_norm_backward_refusals(L, kw, status):
    assert _grad(L, **kw) == status
    assert L.opt_last_error()


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), EINVAL), (dict(cols=1 << 31), EINVAL), (dict(x=None), EINVAL), (dict(x=4097), EALIGN),
    (dict(ldx=10), EINVAL), (dict(dtype=4), EINVAL), (dict(block_rows=64), EINVAL), (dict(q=None), EINVAL),
])
def test_cast_refusals(L, kw, status):
    a = dict(rows=4, cols=100, x=4096, ldx=100, dtype=1, block_rows=1, q=_codes(L))
    a.update(kw)
    q = a.pop("q") or L.OptCodes()
    assert L.lib().opt_block_cast(ctypes.byref(L.OptCast(q=q, qt=L.OptCodes(), **a)), None) == status
    assert L.opt_last_error()


@pytest.mark.parametrize("kw,status", [
    (dict(k=100), EINVAL), (dict(k=-16), EINVAL), (dict(m=-1), EINVAL), (dict(n=1 << 31), EINVAL), (dict(c=None), EINVAL),
    (dict(c=4097), EALIGN), (dict(ldc=3), EINVAL), (dict(c_dtype=8), EINVAL), (dict(accumulate=-1), EINVAL),
    (dict(k=256), EINVAL),
])
def test_product_refusals(L, kw, status):
    a = dict(m=4, n=4, k=112, c=4096, ldc=4, c_dtype=1, accumulate=0)
    a.update(kw)
    r = L.OptProduct(a=_codes(L), b=_codes(L, codes=1 << 23), **a)
    assert L.lib().opt_block_matmul(ctypes.byref(r), None) == status
    assert L.opt_last_error()


def test_null_records(L):
    for fn in ("opt_rms_norm", "opt_rms_norm_backward", "opt_block_cast", "opt_block_matmul"):
        assert getattr(L.lib(), fn)(None, None) == EINVAL


def test_empty_calls_touch_nothing(L):
    """Calls of no elements return before any pointer is looked at."""
    assert _dropout(L, x=None, out=None, n=0) == 0
    assert _norm(L, rows=0, x=None, y=None) == 0
    assert _norm(L, cols=0, x=None, y=None) == 0
    assert _grad(L, rows=0, dweight=None, dy=None) == 0
    assert _grad(L, cols=0, dy=None) == 0
    assert L.lib().opt_block_cast(ctypes.byref(L.OptCast(0, 100, None, 0, 1, 1)), None) == 0
    assert L.lib().opt_block_matmul(ctypes.byref(L.OptProduct(m=0, n=4, k=112)), None) == 0
    assert L.lib().opt_block_matmul(ctypes.byref(L.OptProduct(m=4, n=4, k=0, c=4096, ldc=4, accumulate=1)), None) == 0


def test_workspace_sizes(L):
    assert L.opt_rms_norm_workspace(0, 100) == 0
    for rows, cols in ((1, 1), (7, 4096), (100000, 128), (5000, 32768)):
        n = L.opt_rms_norm_workspace(rows, cols)
        assert n >= 4 * cols and n % (4 * cols) == 0
    for bad in ((-1, 5), (5, -1), (5, 40000)):
        with pytest.raises(L.OptError):
            L.opt_rms_norm_workspace(*bad)


def test_host_tensors_are_refused_by_the_binding(L, monkeypatch):
    monkeypatch.setattr(L, "_device", lambda: 0)
    x, w = torch.zeros(4, 128, dtype=torch.bfloat16), torch.ones(128, dtype=torch.bfloat16)
    q = L.block_buffers(4, 128, device="cpu")
    for call in (lambda: L.opt_dropout(x, x, 0.1), lambda: L.opt_rms_norm(x, w, y=x), lambda: L.opt_block_cast(x, codes=q),
                 lambda: L.opt_rms_norm_backward(x, x, w, x), lambda: L.opt_block_matmul(q, q, torch.zeros(4, 4))):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_block_buffers(L):
    q, s = L.block_buffers(5, 130, device="cpu")
    assert q.shape == (5, 144) and s.shape == (2, 8) and not q.any() and not s.any()


# ---- the plain forms --------------------------------------------------------


def test_grid_is_e4m3():
    v = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(v, P.e4m3(np.arange(256)).astype(np.float32), equal_nan=True)
    x = np.concatenate([P.GRID, (P.GRID[1:] + P.GRID[:-1]) / 2, np.random.RandomState(1).uniform(0, 448, 5000)])
    lib = torch.from_numpy(x.astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(lib, P.nearest_code(x.astype(np.float32).astype(np.float64)))


def test_scale_rule():
    """The smallest power of two that keeps the block on the grid, at every boundary."""
    for e in range(-140, 128):
        for a in (2.0 ** e, 1.75 * 2.0 ** e, np.nextafter(1.75 * 2.0 ** e, np.inf), 1.99 * 2.0 ** e):
            b = int(P.scale_bytes(np.array([a]))[0])
            assert a <= 448 * 2.0 ** (b - 127)
            assert b == 0 or a > 448 * 2.0 ** (b - 128)


def test_norm_gradients_against_differences():
    rng = np.random.RandomState(3)
    h, w, t = rng.randn(3, 37), rng.rand(37) + 0.5, rng.randn(3, 37)
    eps, d = 1e-3, 1e-6
    dx, dw, _, _ = P.norm_gradients(t, h, w, None, eps)

    def loss(h, w):
        return float((P.norm(h, w, eps) * t).sum())

    for i, j in ((0, 0), (1, 17), (2, 36)):
        e = np.zeros_like(h)
        e[i, j] = d
        assert abs((loss(h + e, w) - loss(h - e, w)) / (2 * d) - dx[i, j]) < 1e-7
        e = np.zeros_like(w)
        e[j] = d
        assert abs((loss(h, w + e) - loss(h, w - e)) / (2 * d) - dw[j]) < 1e-7


def test_mask_share():
    bits = P.random_bits(40000, 5, 7)
    assert abs((bits < 0.3 * 65536).mean() - 0.3) < 4 * np.sqrt(0.21 / 40000)
    assert np.array_equal(P.random_bits(24, 5, 7, base=16), bits[16:40])
