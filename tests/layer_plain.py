"""Plain forms, in binary64 on the host, of the operators between a layer's
products: the gated activation and its gradients, and the heads' norm with
rotation and its gradients, each with the bound its binary32 evaluation keeps.
numpy only; no code shared with the library."""
import numpy as np

from tests import pass_plain as P

U = P.U32
K, CUBE = 2 * np.sqrt(2 / np.pi), 0.044715


def inner(x, act):
    """p(x) and p'(x) of s(x) = x sigma(p(x))."""
    if act == "silu":
        return x, np.ones_like(x)
    return K * (x + CUBE * x ** 3), K * (1 + 3 * CUBE * x * x)


def logistic(p):
    """sigma(p) and 1 - sigma(p)."""
    e = np.exp(-np.abs(p))
    big, small = 1 / (1 + e), e / (1 + e)
    return np.where(p >= 0, big, small), np.where(p >= 0, small, big)


def loss(p, act, dtype):
    """Relative error of sigma and of 1 - sigma, as formed in binary32: exp(-|p|)
    to 4 units (the hardware's exp2 to 2, its correction or what |p| log2(e)
    rounds to), p itself to 5 units (its constants, two products, a sum), which
    exp makes absolute in |p|; 16-bit types leave the 1.3 |p| units of |p|
    log2(e) in; then the sum 1 + e, the hardware's reciprocal, a product."""
    a = np.minimum(np.abs(p), 110.0)                    # beyond it exp(-|p|) is 0 on both sides
    return U * (8 + a * ((0.0 if dtype == "f32" else 1.3) + (5.0 if act == "gelu" else 0.0)))


FLUSH = 2.0 ** -124                                     # a sigma below 2^-126 may be formed as 0


def gate(x, u, act, dtype):
    """(y, the bound of its binary32 form): s is sigma and one product, y one more."""
    x, u = x.astype(np.float64), u.astype(np.float64)
    p, _ = inner(x, act)
    sig, _ = logistic(p)
    y = x * sig * u
    return y, np.abs(y) * (loss(p, act, dtype) + 2 * U) + FLUSH * np.abs(x * u)


def gate_gradients(dy, x, u, act, dtype):
    """((dgate, bound), (dup, bound), (y, bound))."""
    dy, x, u = (v.astype(np.float64) for v in (dy, x, u))
    p, dp = inner(x, act)
    sig, rest = logistic(p)
    e = loss(p, act, dtype)
    s, tail = x * sig, x * sig * rest * dp
    # s rest p': sigma's and rest's errors, the products, p' to 4 units; sigma's own; their sum; two products.
    # 16-bit types form rest as 1 - sigma: off by what sigma is off, and a rounding below 1
    of_rest = np.abs(tail) * e if dtype == "f32" else np.abs(x * sig * dp) * (sig * e + U)
    size = np.abs(tail) * (e + 8 * U) + of_rest + sig * (e + 2 * U) + 3 * U * np.abs(sig + tail)
    dg, du = dy * u * (sig + tail), dy * s
    tiny = FLUSH * (1 + np.abs(x)) * (1 + np.abs(dp))
    return ((dg, np.abs(dy * u) * (size + tiny)), (du, np.abs(du) * (e + 2 * U) + np.abs(dy) * tiny),
            (s * u, np.abs(s * u) * (e + 2 * U) + np.abs(u) * tiny))


def stored(want, bound, dtype):
    """The bound of a value that is rounded to the type once more."""
    return bound + (np.abs(want) + bound) * P.HALF[dtype] + P.TINY[dtype]


def check_values(got, want, bound):
    got = got.astype(np.float64)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    ok = np.isfinite(want)
    assert np.array_equal(got[~ok & ~np.isnan(want)], want[~ok & ~np.isnan(want)])
    off = np.abs(got[ok] - want[ok]) - bound[ok]
    assert np.all(off <= 0), float(off.max())


def check_codes(pair, want, bound, rows, cols):
    """The pair codes values within `bound` of `want`: every scale is the
    rule's for a block maximum within the bound, every code within half a step
    of its grid, the padding zeros.  `want` is finite."""
    q, s = (t.cpu().numpy() for t in pair)
    nb = (cols + 127) // 128
    s = s[:nb, :rows]
    lo, hi = P.scale_bytes(P.block_maxima(np.maximum(np.abs(want) - bound, 0), 1).T), P.scale_bytes(P.block_maxima(np.abs(want) + bound, 1).T)
    assert np.all((lo <= s) & (s <= hi))
    X = np.repeat(2.0 ** (s.T.astype(np.float64) - 127), 128, 1)[:, :cols]
    got = P.decode(q[:rows], s, cols)
    step = X * 2.0 ** (np.maximum(np.floor(np.log2(np.maximum((np.abs(want) + bound) / X, 2.0 ** -6))), -6) - 3)
    check_values(got, want, step / 2 + bound)
    assert not q[:rows, cols:P.up(cols, 16)].any()


# ---- heads ------------------------------------------------------------------


def table(positions, rot, base=10000.0):
    """float32 [positions, rot] of cosines, then sines."""
    a = np.arange(positions, dtype=np.float64)[:, None] * base ** (-np.arange(0, rot, 2) / rot)
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


def pairs(rot, interleaved):
    i = np.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def turn(x, tab, pos, rot, interleaved, back=False):
    """(heads [tokens, heads, dim] turned by their tokens' angles, the sums of
    the products' magnitudes); NaN for a token the table does not hold."""
    y, size = x.copy(), np.abs(x)
    if rot:
        inside = (pos >= 0) & (pos < tab.shape[0])
        row = np.where(inside[:, None], tab[np.where(inside, pos, 0)].astype(np.float64), np.nan)
        c, s = row[:, None, :rot // 2], row[:, None, rot // 2:] * (-1 if back else 1)
        i, j = pairs(rot, interleaved)
        a, b = x[..., i], x[..., j]
        y[..., i], y[..., j] = a * c - b * s, b * c + a * s
        size[..., i], size[..., j] = np.abs(a * c) + np.abs(b * s), np.abs(b * c) + np.abs(a * s)
        y[~inside] = np.nan
        size[~inside] = np.nan
    return y, size


def heads(x, w, tab, pos, eps, rot, interleaved):
    """(y, the bound of its binary32 form): r rounds once, x r and (x r) w once
    each, the two products and their sum once each."""
    x, w = x.astype(np.float64), w.astype(np.float64)
    n = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w
    y, size = turn(n, tab, pos, rot, interleaved)
    return y, 5.1 * U * size


def head_gradients(dy, x, w, tab, pos, eps, rot, interleaved):
    """((dx, bound), (dw, its terms' magnitudes)).  dn errs by 2 units of the
    sum m of its products' magnitudes, g = dn w by 3; c's terms by those; k by
    r twice and its own rounding; then x k, the difference and r's product."""
    dy, x, w = (v.astype(np.float64) for v in (dy, x, w))
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    dn, m = turn(dy, tab, pos, rot, interleaved, back=True)
    g, m = dn * w, m * np.abs(w)
    k = r * r * (g * x).mean(-1, keepdims=True)
    dx = r * (g - x * k)
    size = 6 * r * m + 7 * r * np.abs(x * k) + 3 * r ** 3 * np.abs(x) * (m * np.abs(x)).mean(-1, keepdims=True)
    dw = (dn * x * r).sum((0, 1))
    with np.errstate(invalid="ignore"):
        terms = (m / np.where(w == 0, np.nan, np.abs(w)) * np.abs(x) * r).sum((0, 1))
    return (dx, 1.05 * U * size), (dw, terms)
