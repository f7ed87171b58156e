"""Plain forms, in binary64 on the host, of the training-pass operators: the
dropout mask from the oracle's generator, the norm and its gradients, the
block-coded format and the product, with the bounds their binary32 evaluation
keeps.  numpy only; no code shared with the library."""
import numpy as np
import torch

import oracle

U32 = 2.0 ** -24                                        # half a step of binary32, relative
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}   # half a step of the stored type
TINY = {"f32": 2.0 ** -149, "bf16": 2.0 ** -133, "f16": 2.0 ** -24}  # its smallest magnitude


def up(n, m):
    return (n + m - 1) // m * m


def rounded(x, dtype):
    """float32 array -> the stored type's values (nearest-even), as float32."""
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(TYPES[dtype]).float().numpy()


def random_bits(n, seed, offset, base=0):
    """16 random bits of elements base .. base + n - 1."""
    q = np.arange(base // 8, (base + n + 7) // 8, dtype=np.uint64)
    out = np.empty((q.size, 4), np.uint32)
    for i, v in enumerate(q.tolist()):
        out[i] = oracle.philox((v & 0xFFFFFFFF, (v >> 32) | 0x80000000, offset & 0xFFFFFFFF, offset >> 32),
                               (seed & 0xFFFFFFFF, seed >> 32))
    return out.view(np.uint16).reshape(-1)[base % 8:][:n]


def dropout(x, res, p, seed, offset, base=0):
    """The exact stored result in binary32 steps (every one is IEEE)."""
    t = int(np.floor(p * 65536 + 0.5))
    s = np.float32(1.0 / (1.0 - t / 65536.0)) if t < 65536 else np.float32(0)
    keep = random_bits(x.size, seed, offset, base).reshape(x.shape) >= t
    with np.errstate(invalid="ignore", over="ignore"):
        y = np.where(keep, x.astype(np.float32) * s, np.float32(0))
        return y if res is None else y + res.astype(np.float32)


# ---- block-coded matrices ---------------------------------------------------

GRID = np.array([(c & 7) * 2.0 ** -9 if c < 8 else (8 + (c & 7)) * 2.0 ** ((c >> 3) - 10) for c in range(127)])


def e4m3(codes):
    """Values of E4M3 code bytes."""
    c = np.asarray(codes, np.uint8)
    mag = np.append(GRID, np.nan)[c & 0x7F]
    return np.where(c & 0x80, -mag, mag)


def nearest_code(y):
    """E4M3 magnitude codes of |y| <= 448, nearest, ties to the even code."""
    y = np.abs(y)
    hi = np.clip(np.searchsorted(GRID, y, side="left"), 1, 126)
    lo = hi - 1
    dl, dh = y - GRID[lo], GRID[hi] - y
    return np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi).astype(np.uint8)


def scale_bytes(a):
    """Byte of the smallest 2^(byte - 127) with a <= 448 * 2^(byte - 127)."""
    a = np.asarray(a, np.float64)
    out = np.zeros(a.shape, np.int64)
    ok = np.isfinite(a) & (a > 0)
    e = np.ceil(np.log2(np.where(ok, a, 1.0) / 448.0))
    for _ in range(2):
        e = np.where(np.where(ok, a, 1.0) > 448.0 * 2.0 ** e, e + 1, e)
        e = np.where(np.where(ok, a, 1.0) <= 448.0 * 2.0 ** (e - 1), e - 1, e)
    out[ok] = np.maximum(e[ok], -127).astype(np.int64) + 127
    out[~np.isfinite(a)] = 255
    return out.astype(np.uint8)


def block_maxima(x, block_rows):
    """Largest magnitude (NaN as infinity) for each block, one row for each of x's, [rows, blocks]."""
    rows, cols = x.shape
    big = np.zeros((up(rows, block_rows), up(cols, 128)))
    big[:rows, :cols] = np.where(np.isnan(x), np.inf, np.abs(x.astype(np.float64)))
    m = big.reshape(big.shape[0] // block_rows, block_rows, -1, 128).max((1, 3))
    return np.repeat(m, block_rows, 0)[:rows]


def encode(x, block_rows=1):
    """(codes [rows, cols], scale bytes [blocks, rows]) of x, exactly."""
    b = scale_bytes(block_maxima(x, block_rows))
    each = np.repeat(b, 128, 1)[:, :x.shape[1]]
    y = np.where(each == 255, 0.0, x.astype(np.float64)) / 2.0 ** (each.astype(np.float64) - 127)
    sign = np.where((each != 255) & np.signbit(x), 0x80, 0).astype(np.uint8)
    return nearest_code(y) | sign, b.T.copy()


def decode(codes, scales, cols):
    """Values of a block-coded matrix; scales [blocks, rows]."""
    s = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127))
    return e4m3(codes[:, :cols]) * np.repeat(s.T, 128, 1)[:codes.shape[0], :cols]


# ---- the norm ---------------------------------------------------------------


def norm(h, w, eps):
    h, w = h.astype(np.float64), w.astype(np.float64)
    return h / np.sqrt((h * h).mean(1, keepdims=True) + eps) * w


def norm_bound(y, dtype):
    """r, h * r and (h * r) * w each round once to binary32, then the store: a
    half step of the type (or of its smallest magnitude)."""
    return (HALF[dtype] * (1 + 4 * U32) + 3.1 * U32) * np.abs(y) + TINY[dtype]


def norm_gradients(dy, h, w, dh, eps):
    """(dx, dw, bound terms) in binary64."""
    dy, h, w = (v.astype(np.float64) for v in (dy, h, w))
    r = 1 / np.sqrt((h * h).mean(1, keepdims=True) + eps)
    g = dy * w
    k = r * r * (g * h).mean(1, keepdims=True)
    dx = r * (g - h * k)
    if dh is not None:
        dx = dx + dh
    # dy*w, h*k, their difference, the product by r, the addition of dh, r
    # itself and k (r twice, its own rounding, and the roundings of dy*w under
    # the mean) each err by at most a half step of binary32 of a magnitude
    # that one of these terms bounds
    size = r * np.abs(g) + r * np.abs(h) * np.abs(k) + r ** 3 * np.abs(h) * np.abs(g * h).mean(1, keepdims=True)
    if dh is not None:
        size = size + np.abs(dh)
    return dx, (dy * h * r).sum(0), size, (np.abs(dy * h) * r).sum(0)


# ---- the 8-bit matrix products ----------------------------------------------


def exponents(codes):
    """Floor exponents of E4M3 codes, a subnormal code's as -6, a zero's far below."""
    c = np.asarray(codes, np.int64) & 0x7F
    return np.where(c == 0, -1000, np.maximum(c >> 3, 1) - 7)


def code_products_loss(qa, sa, qb, sb, k):
    """What opt_block_matmul may lose with OPT_CODE_PRODUCTS, for rows of codes
    qa [m, k] and qb [n, k] (k a multiple of 8) and scales [blocks, rows]: each
    product cut toward zero at 2^-13 of 2^E, E the largest sum of exponents in
    its eight columns.  (the sum of the losses, of their magnitudes)"""
    m, n = qa.shape[0], qb.shape[0]
    va, vb = e4m3(qa[:, :k]), e4m3(qb[:, :k])
    ea, eb = exponents(qa[:, :k]), exponents(qb[:, :k])
    loss, size = np.zeros((m, n)), np.zeros((m, n))
    for j in range(0, k, 8):
        e = (ea[:, None, j:j + 8] + eb[None, :, j:j + 8]).max(2, keepdims=True)
        p = va[:, None, j:j + 8] * vb[None, :, j:j + 8]
        unit = 2.0 ** np.maximum(e - 13.0, -60)
        lost = p - np.trunc(p / unit) * unit
        scale = 2.0 ** (sa[j // 128].astype(float)[:, None] + sb[j // 128].astype(float)[None, :] - 254)
        loss += lost.sum(2) * scale
        size += np.abs(lost).sum(2) * scale
    return loss, size
