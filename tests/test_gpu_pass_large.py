"""GPU tests of the training-pass operators at sizes whose tiles outnumber the
largest grid (2^20 workgroups), so that workgroups take a second tile."""
import numpy as np
import pytest

from tests import pass_plain as P
from tests.test_gpu_pass import coded, dev, host

pytestmark = pytest.mark.gpu

GRID = 1 << 20


@pytest.fixture(scope="module", autouse=True)
def gpu():
    import torch
    import optimizer_step_amd as osa
    assert torch.cuda.is_available()
    osa.lib()
    yield
    torch.cuda.empty_cache()


def test_dropout_past_the_grid():
    """Elements past 2^32, against calls on parts of them."""
    import torch
    import optimizer_step_amd as osa
    n = GRID * 4096 + 8 * 1000 + 3
    x = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    osa.opt_dropout(x, x, 0.5, seed=3, offset=4)
    for base in (0, 8 * 12345, GRID * 4096 - 4096, GRID * 4096, n - 3 - 8 * 500):
        part = x[base:base + 8192]
        want = torch.ones_like(part)
        osa.opt_dropout(want, want, 0.5, seed=3, offset=4, index_base=base)
        assert torch.equal(part, want)
    first = P.random_bits(64, 3, 4, GRID * 4096) >= 32768
    assert np.array_equal(host(x[GRID * 4096:GRID * 4096 + 64]), np.where(first, 2.0, 0.0))


def test_norm_past_the_grid():
    """More rows of a workgroup each than the grid has, against calls on some of them."""
    import torch
    import optimizer_step_amd as osa
    rows, cols = GRID + 37, 2056
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(rows, cols, generator=g, device="cuda", dtype=torch.bfloat16)
    w = dev(P.rounded(0.5 + np.random.RandomState(1).rand(cols), "f32"), "f32")
    q, y = osa.block_buffers(rows, cols), torch.empty_like(x)
    osa.opt_rms_norm(x, w, y=y, codes=q)
    for at in (0, 1000, GRID - 16, GRID + 16):
        s = slice(at, at + 16)
        y1, q1 = torch.empty_like(x[s]), osa.block_buffers(16, cols)
        osa.opt_rms_norm(x[s], w, y=y1, codes=q1)
        assert torch.equal(y[s], y1) and torch.equal(q[0][s], q1[0]) and torch.equal(q[1][:, s], q1[1])
    want = P.norm(host(x[GRID:GRID + 37]), host(w), 1e-6)
    assert np.all(np.abs(host(y[GRID:GRID + 37]) - want) <= P.norm_bound(want, "bf16"))


def test_product_past_the_grid():
    """More strips of 16 columns than the grid has, of one row."""
    import torch
    import optimizer_step_amd as osa
    n = 16 * GRID + 40
    a, av = coded(1, 1, 16, True)
    b, bv = coded(2, 4096, 16, True)
    big = osa.block_buffers(n, 16)
    at = torch.arange(n, device="cuda") % 4093
    big[0].copy_(b[0][at])
    big[1][:, :n].copy_(b[1][:, at])
    c = torch.empty(1, n, device="cuda")
    osa.opt_block_matmul(a, big, c)
    want = torch.from_numpy((av @ bv.T).astype(np.float32)).cuda()[:, at]
    assert torch.equal(c, want)
