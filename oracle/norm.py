"""Residual addition with RMS norm, its gradient, and counter-based dropout
(float64 oracle).

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

The pages adapt a decoder's linear layers; these are the definitions of what
stands between two of them:

* h = bf16(res + keep x s), s = binary32(1 / (1 - p)); y = h rstd g with
  rstd = 1 / sqrt(mean h^2 + eps).  h is rounded to bf16 before the norm, as it is
  what the next layer's residual stream holds.
* 8-bit y: per block a = max |y|, scale = fl32(a / 448) (0 below 2^-126), code =
  E4M3(fl32(y / scale)).
* dh = rstd (g dy - h mean(g dy h) rstd^2) + dH; dx = keep s dh; dg = sum dy h rstd.
* The words of Philox4x32-10 (Salmon, Moraes, Dror, Shaw, "Parallel random
  numbers: as easy as 1, 2, 3", 2011): element e takes word e mod 4 of the counter
  (e div 4, offset); it is kept where the word is at least rint(p 2^32).
"""

from __future__ import annotations

import numpy as np

M0, M1, W0, W1 = 0xD2511F53, 0xCD9E8D57, 0x9E3779B9, 0xBB67AE85


def philox4x32_10(counter, key):
    """One block: counter of four and key of two 32-bit words -> four words."""
    c, k = list(counter), list(key)
    for _ in range(10):
        a, b = M0 * c[0], M1 * c[2]
        c = [(b >> 32) ^ c[1] ^ k[0], b & 0xFFFFFFFF, (a >> 32) ^ c[3] ^ k[1], a & 0xFFFFFFFF]
        k = [(k[0] + W0) & 0xFFFFFFFF, (k[1] + W1) & 0xFFFFFFFF]
    return c


def words(seed: int, offset: int, first: int, n: int) -> np.ndarray:
    """The 32-bit words of elements first .. first + n - 1 (uint32)."""
    lo, sh = np.uint64(0xFFFFFFFF), np.uint64(32)
    b0, b1 = first // 4, (first + n + 3) // 4
    i = np.arange(b0, b1, dtype=np.uint64)
    c = [i & lo, i >> sh, np.full_like(i, offset & 0xFFFFFFFF), np.full_like(i, offset >> 32)]
    k0, k1 = seed & 0xFFFFFFFF, seed >> 32
    for _ in range(10):
        a, b = c[0] * np.uint64(M0), c[2] * np.uint64(M1)
        c = [(b >> sh) ^ c[1] ^ np.uint64(k0), b & lo, (a >> sh) ^ c[3] ^ np.uint64(k1), a & lo]
        k0, k1 = (k0 + W0) & 0xFFFFFFFF, (k1 + W1) & 0xFFFFFFFF
    w = np.stack(c, 1).astype(np.uint32).reshape(-1)
    return w[first - 4 * b0:first - 4 * b0 + n]


def keep_mask(p: float, seed: int, offset: int, M: int, n: int) -> np.ndarray:
    """The keep mask of an (M, n) tensor as bool."""
    t = np.uint32(np.rint(np.float64(np.float32(p)) * 4294967296.0))
    return (words(seed, offset, 0, M * n) >= t).reshape(M, n)


def keep_scale(p: float) -> float:
    return float(np.float32(1.0 / (1.0 - float(np.float32(p)))))


def round_bf16(a) -> np.ndarray:
    """Nearest bfloat16 (ties to even) of float64 values, in one rounding."""
    m, e = np.frexp(np.asarray(a, dtype=np.float64))
    return np.ldexp(np.rint(m * 256.0), e - 8)


def rmsnorm(x, res, g, eps, keep=None, p: float = 0.0):
    """(h, y, rstd) in float64."""
    h = np.asarray(x, np.float64)
    if keep is not None:
        h = h * (np.asarray(keep, np.float64) * keep_scale(p))
    if res is not None:
        h = h + np.asarray(res, np.float64)
    h = round_bf16(h)
    rstd = 1.0 / np.sqrt((h * h).mean(axis=1) + float(np.float32(eps)))
    return h, h * rstd[:, None] * np.asarray(g, np.float64), rstd


def rmsnorm_backward(dy, h, g, rstd, dH=None, keep=None, p: float = 0.0):
    """(dx, dh, dg) in float64 for the given h and rstd."""
    dy, h, g, rstd = (np.asarray(a, np.float64) for a in (dy, h, g, rstd))
    gh = dy * g
    c = (gh * h).mean(axis=1, keepdims=True) * rstd[:, None] ** 2
    dh = rstd[:, None] * (gh - h * c)
    if dH is not None:
        dh = dh + np.asarray(dH, np.float64)
    dx = dh if keep is None else dh * (np.asarray(keep, np.float64) * keep_scale(p))
    return dx, dh, (dy * h * rstd[:, None]).sum(axis=0)


def quantize_e4m3(y, block: int):
    """(code values, scales) of y by blocks of `block` columns (0: a whole row)."""
    from oracle.nf4 import e4m3_decode, e4m3_encode, fl32
    y = np.asarray(y, np.float64)
    M, n = y.shape
    b = y.reshape(M, -1, block or n)
    s = fl32(np.abs(b).max(axis=2) / 448.0).astype(np.float64)
    s = np.where(s < 2.0 ** -126, 0.0, s)
    safe = np.where(s > 0, s, 1.0)
    v = np.where(s[:, :, None] > 0, fl32(b / safe[:, :, None]).astype(np.float64), 0.0).reshape(-1)
    sign = np.where(v < 0, -1.0, 1.0)
    return (sign * e4m3_decode(e4m3_encode(np.abs(v).astype(np.float32)))).reshape(M, n), s
