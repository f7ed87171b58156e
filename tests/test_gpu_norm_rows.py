"""GPU tests of the RMS norm's backward pass where every workgroup takes three
rows (or groups of rows) in turn: both halves of its loop, with and without a
row read ahead, for every number of lanes a row has."""
import numpy as np
import pytest

from tests import pass_plain as P
from tests.test_gpu_pass import check_values, data, dev, empty, host, untouched

pytestmark = pytest.mark.gpu

# 16 lanes a row hold 16 rows a workgroup, 64 lanes 4, 256 and 1024 lanes one;
# 512 workgroups at most, 256 of 1024 lanes
SIZES = [(16401, 128), (16389, 500), (4103, 1000), (4103, 2048), (1100, 4099), (1100, 8192), (600, 8200), (600, 11008),
         (600, 16383), (523, 16392), (520, 32768)]


@pytest.fixture(scope="module", autouse=True)
def gpu():
    import torch
    import optimizer_step_amd as osa
    assert torch.cuda.is_available()
    osa.lib()


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("dtype,w_dtype,more", [("f32", "f32", True), ("f32", "bf16", False), ("bf16", "f32", False),
                                                ("f16", "f16", True)])
def test_three_rows_a_workgroup(rows, cols, dtype, w_dtype, more):
    import torch
    import optimizer_step_amd as osa
    groups = osa.opt_rms_norm_workspace(rows, cols) // (4 * cols)
    each = {16: 16, 64: 4}.get(16 if cols <= 512 else 64 if cols <= 2048 else 0, 1)
    assert rows > 2 * groups * each
    dy, h = data(cols, rows, cols, dtype, 0.1), data(cols + 1, rows, cols, dtype)
    dh = data(cols + 2, rows, cols, dtype, 0.1) if more else None
    w = P.rounded(0.5 + np.random.RandomState(cols).rand(cols), w_dtype)
    start = np.random.RandomState(cols).randn(cols).astype(np.float32) if more else np.zeros(cols, np.float32)
    dx, dw = empty(rows, cols, dtype, 3), torch.from_numpy(start.copy()).cuda()
    osa.opt_rms_norm_backward(dev(dy, dtype), dev(h, dtype, 2), dev(w, w_dtype), dx, dw, eps=1e-5,
                              dh=dev(dh, dtype) if more else None, accumulate=more)
    want, want_w, size, size_w = P.norm_gradients(dy, h, w, dh, 1e-5)
    # seven roundings at most touch a term before the last sum's and the store's
    check_values(host(dx), want, 9 * P.U32 * size + P.HALF[dtype] * (1 + 16 * P.U32) * np.abs(want) + 9 * P.U32 * P.HALF[dtype] * size
                 + P.TINY[dtype])
    assert untouched(dx)
    # three roundings a term, binary32 sums of at most `run` terms, binary64 after
    run = rows / groups + 8
    check_values(dw.cpu().numpy(), want_w + start, (3 + run) * P.U32 * size_w + 2 * P.U32 * np.abs(want_w + start))
