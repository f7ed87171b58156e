"""Host-side checks of the block product's choice of sum, and of the loss that
its 8-bit products are documented with."""
import ctypes

import numpy as np
import pytest

from tests import pass_plain as P
from tests.test_pass_cpu import L, EINVAL  # noqa: F401


@pytest.mark.parametrize("accumulate", [4, 5, -2, 1 << 30])
def test_unknown_flags_are_refused(L, accumulate):  # noqa: F811
    q = L.OptCodes(1 << 20, 128, 1 << 21, 64)
    r = L.OptProduct(4, 4, 112, q, q, 4096, 4, 1, accumulate)
    assert L.lib().opt_block_matmul(ctypes.byref(r), None) == EINVAL


def test_flags_of_an_empty_sum(L):  # noqa: F811
    """k = 0 with accumulate leaves c alone, whatever the choice of sum."""
    for accumulate in (1, 1 + L.CODE_PRODUCTS):
        assert L.lib().opt_block_matmul(ctypes.byref(L.OptProduct(m=4, n=4, k=0, c=4096, ldc=4, accumulate=accumulate)), None) == 0


def test_loss_of_code_products():
    """The documented loss on normal data: 1.4e-5 of a result; of one sign, the
    cut's bias stays of that order; a small product beside large ones is lost."""
    rng = np.random.RandomState(5)
    for data in (lambda r: rng.randn(r, 2048), lambda r: np.abs(rng.randn(r, 2048))):
        (qa, sa), (qb, sb) = P.encode(data(24).astype(np.float32)), P.encode(data(24).astype(np.float32))
        loss, size = P.code_products_loss(qa, sa, qb, sb, 2048)
        want = P.decode(qa, sa, 2048) @ P.decode(qb, sb, 2048).T
        print(np.linalg.norm(loss) / np.linalg.norm(want))
        assert np.linalg.norm(loss) <= 2e-5 * np.linalg.norm(want) and np.all(np.abs(loss) <= size)
    a, b = np.zeros((1, 8), np.float32), np.zeros((1, 8), np.float32)
    a[0, :3], b[0, :3] = (448, -448, 2.0 ** -6), (2.0 ** -9, 2.0 ** -9, 2.0 ** -6)
    qa, qb = (P.nearest_code(v) | np.where(np.signbit(v), 0x80, 0).astype(np.uint8) for v in (a, b))
    s = np.full((1, 1), 127, np.uint8)
    assert P.code_products_loss(qa, s, qb, s, 8)[0][0, 0] == 2.0 ** -12
