"""GPU tests of the block product's sums: results of every type are binary32
sums of exact products, however many rows a call has."""
import numpy as np
import pytest

from tests import pass_plain as P
from tests.test_gpu_pass import check_values, coded, dev, empty, host

pytestmark = pytest.mark.gpu

SIZES = [(300, 2600, 128), (300, 2600, 400), (2100, 4200, 128), (2100, 4200, 400)]    # 128 x 128 and 256 x 256 tiles


@pytest.fixture(scope="module", autouse=True)
def gpu():
    import torch
    import optimizer_step_amd as osa
    assert torch.cuda.is_available()
    osa.lib()


def code(v):
    return int(P.nearest_code(np.array([abs(v)]))[0]) | (0x80 if v < 0 else 0)


def cancelling(rows, k, values, seed):
    """A block-coded matrix whose rows start each 64 columns with `values`,
    with scales of 1 to 4: (pair on the device, its values)."""
    import torch
    import optimizer_step_amd as osa
    pair = osa.block_buffers(rows, k)
    codes = np.zeros((rows, k), np.uint8)
    for c in range(0, k - len(values) + 1, 64):
        codes[:, c:c + len(values)] = [code(v) for v in values]
    scales = np.random.RandomState(seed).randint(127, 130, ((k + 127) // 128, rows)).astype(np.uint8)
    pair[0][:, :k] = torch.from_numpy(codes).cuda()
    pair[1][:, :rows] = torch.from_numpy(scales).cuda()
    return pair, P.decode(codes, scales, k)


# Each 64 columns hold 448 * 2^-9, its negative and 2^-12, with signs and
# subnormal codes on either side: 2^-12 is all that stays.
LEFT, RIGHT = (448.0, -448.0, 2.0 ** -6, 2.0 ** -9), (2.0 ** -9, 2.0 ** -9, 2.0 ** -6, 0.0)


@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_small_products_beside_large_ones(m, n, k, dtype):
    """Every partial sum is exact in binary32 (fewer than 24 bits between
    2^-12 and the sum of magnitudes), so the result is the exact one, and a
    row's bits are those of a call with that row alone."""
    import torch
    import optimizer_step_amd as osa
    for left, right in ((LEFT, RIGHT), (RIGHT, LEFT)):
        a, av = cancelling(m, k, left, 1)
        b, bv = cancelling(n, k, right, 2)
        want = av @ bv.T
        assert want.min() > 0 and (np.abs(av) @ np.abs(bv).T).max() < 2.0 ** 11
        c = empty(m, n, dtype)
        osa.opt_block_matmul(a, b, c)
        assert np.array_equal(host(c), P.rounded(want, dtype))
        one = empty(4, n, dtype)
        osa.opt_block_matmul((a[0][8:12], a[1][:, 8:12]), b, one)
        assert torch.equal(one, c[8:12])


@pytest.mark.parametrize("m,n,k", [(257, 3001, 300), (2100, 4200, 400), (511, 1700, 1040)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_any_codes(m, n, k, dtype):
    """The bound of a binary32 sum in any order, each addition off by at most a
    step (2^-23) of the running magnitude, and the store's half step."""
    import optimizer_step_amd as osa
    a, _ = coded(m + k, m, k, False)
    b, _ = coded(n + k, n, k, False)
    a[1][:, :m].clamp_(max=124)                         # inside the range of binary16
    b[1][:, :n].clamp_(max=112)
    av, bv = (P.decode(q[0].cpu().numpy(), q[1].cpu().numpy()[:, :r], k) for q, r in ((a, m), (b, n)))
    c = empty(m, n, dtype)
    osa.opt_block_matmul(a, b, c)
    want, off = av @ bv.T, (k + 8) * 2.0 ** -23 * (np.abs(av) @ np.abs(bv).T)
    assert np.abs(want).max() < 6e4
    check_values(host(c), want, off + P.HALF[dtype] * (np.abs(want) + off) + P.TINY[dtype])


# ---- where the caller allows the 8-bit products -----------------------------


def matrix(kind, rows, k, seed):
    """Values of one kind, [rows, k]."""
    rng = np.random.RandomState(seed)
    x = rng.randn(rows, k)
    if kind == "positive":
        x = np.abs(x)
    elif kind == "loud":                                # two columns of 64 push the others toward subnormal codes
        x[:, ::64] *= 300
        x[:, 5::64] *= 300
    elif kind == "spread":                              # every magnitude of the grid
        x = np.sign(x) * 2.0 ** rng.uniform(-9, 8.8, (rows, k))
    return P.rounded(x, "f32")


def subnormal(rows, k, seed):
    """Codes below 2^-6 alone, but for one a block."""
    import torch
    import optimizer_step_amd as osa
    rng = np.random.RandomState(seed)
    pair = osa.block_buffers(rows, k)
    codes = (rng.randint(0, 8, (rows, k)) | (rng.randint(0, 2, (rows, k)) << 7)).astype(np.uint8)
    codes[:, 3::128] = code(448.0)
    pair[0][:, :k] = torch.from_numpy(codes).cuda()
    pair[1].fill_(127)
    return pair


@pytest.mark.parametrize("kind_a,kind_b", [("normal", "normal"), ("positive", "positive"), ("loud", "normal"), ("loud", "loud"),
                                           ("spread", "spread"), ("subnormal", "normal"), ("subnormal", "subnormal")])
@pytest.mark.parametrize("m,n,k", [(300, 2600, 4096), (2100, 4200, 528)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_code_products(kind_a, kind_b, m, n, k, dtype):
    """Off by no more than the products' cut (computed for every product of
    some rows and columns), the bound of a binary32 sum, and the store's half
    step."""
    import optimizer_step_amd as osa
    pairs = []
    for kind, rows, seed in ((kind_a, m, 1), (kind_b, n, 2)):
        if kind == "subnormal":
            pairs.append(subnormal(rows, k, seed))
        else:
            pairs.append(osa.block_buffers(rows, k))
            osa.opt_block_cast(dev(matrix(kind, rows, k, seed), "f32"), codes=pairs[-1])
    for q in pairs:                                     # results inside the range of binary16
        q[1].clamp_(max=122)
    c = empty(m, n, dtype)
    osa.opt_block_matmul(*pairs, c, exact=False)
    at = [np.random.RandomState(3).choice(r, 12, replace=False) for r in (m, n)]
    (qa, sa), (qb, sb) = ((q.cpu().numpy()[i], s.cpu().numpy()[:, i]) for (q, s), i in zip(pairs, at))
    av, bv = P.decode(qa, sa, k), P.decode(qb, sb, k)
    want = av @ bv.T
    assert np.abs(want).max() < 6e4
    off = P.code_products_loss(qa, sa, qb, sb, k)[1] + (k + 8) * 2.0 ** -23 * (np.abs(av) @ np.abs(bv).T)
    check_values(host(c)[np.ix_(*at)], want, off + P.HALF[dtype] * (np.abs(want) + off) + P.TINY[dtype])


def test_code_products_leave_the_other_calls_alone():
    """An fp32 result and one of few rows are the exact form's bits either way,
    added to or not; a 16-bit result of many rows is added to as well."""
    import torch
    import optimizer_step_amd as osa
    for m, n, k, dtype in ((300, 2600, 400, "f32"), (16, 2600, 400, "bf16"), (64, 500, 400, "f16")):
        a, b = coded(1, m, k, False)[0], coded(2, n, k, False)[0]
        a[1].clamp_(max=124)
        b[1].clamp_(max=112)
        c, d = torch.ones(m, n, dtype=P.TYPES[dtype], device="cuda"), torch.ones(m, n, dtype=P.TYPES[dtype], device="cuda")
        for accumulate in (False, True):
            osa.opt_block_matmul(a, b, c, accumulate=accumulate)
            osa.opt_block_matmul(a, b, d, accumulate=accumulate, exact=False)
            assert torch.equal(c, d)
    (a, av), (b, bv) = coded(1, 300, 400, True), coded(2, 2600, 400, True)
    c = torch.full((300, 2600), 3.0, dtype=torch.bfloat16, device="cuda")
    osa.opt_block_matmul(a, b, c, accumulate=True, exact=False)
    assert np.array_equal(host(c), P.rounded(av @ bv.T + 3.0, "bf16"))


@pytest.mark.parametrize("m,n,k", [(257, 3001, 304), (900, 900, 144), (2100, 4200, 400), (4352, 2304, 1152)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_code_products_whole(m, n, k, dtype):
    """Small whole values lose nothing: the exact result rounded once; NaN
    scales and codes stay in their own row and column."""
    import optimizer_step_amd as osa
    a, av = coded(m + k, m, k, True)
    b, bv = coded(n + k, n, k, True)
    a[1][1, 3] = 255
    b[0][n - 1, 7] = 0x7F
    c = empty(m, n, dtype, 5)
    osa.opt_block_matmul(a, b, c, exact=False)
    want = P.rounded(av @ bv.T, dtype)
    want[3, :] = np.nan
    want[:, n - 1] = np.nan
    assert np.array_equal(host(c), want, equal_nan=True)
