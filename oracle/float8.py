"""8-bit floating point by table in float64: E4M3 and E5M2 (OCP FP8), the
block-scaled quantiser and product, and the AdamW step with 8-bit moments
(include/moelora.h states the definitions).  Test infrastructure only."""
from __future__ import annotations

from typing import Tuple

import numpy as np

BLOCK = 128
TINY = 2.0 ** -100


def _table(exp_bits: int, man_bits: int, bias: int, ieee: bool) -> np.ndarray:
    """Value of each code 0 .. 127 (sign 0); NaN / infinity as NaN."""
    out = np.full(128, np.nan)
    for c in range(128):
        e, m = c >> man_bits, c & ((1 << man_bits) - 1)
        if (ieee and e == (1 << exp_bits) - 1) or (not ieee and c == 127):
            continue
        frac = m / 2 ** man_bits
        out[c] = frac * 2.0 ** (1 - bias) if e == 0 else (1 + frac) * 2.0 ** (e - bias)
    return out


E4M3 = _table(4, 3, 7, False)
E5M2 = _table(5, 2, 15, True)
FORMATS = {"e4m3": (E4M3, 448.0, 3), "e5m2": (E5M2, 57344.0, 2)}
LOWEST = {"e4m3": -6, "e5m2": -14}  # exponent of the smallest normal value, and of all below it


def decode(codes: np.ndarray, fmt: str) -> np.ndarray:
    t = FORMATS[fmt][0]
    c = codes.astype(np.int64)
    return np.where(c >= 128, -1.0, 1.0) * t[c & 127]


def nearest(y: np.ndarray, fmt: str) -> np.ndarray:
    """Codes of the nearest values, ties to the even code; |y| within range."""
    t, top, _ = FORMATS[fmt]
    grid = t[:int(np.nanargmax(t)) + 1]
    a = np.minimum(np.abs(y), top)
    hi = np.clip(np.searchsorted(grid, a), 1, grid.size - 1)
    lo = hi - 1
    dl, dh = a - grid[lo], grid[hi] - a
    c = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    return (c + np.where(np.signbit(y), 128, 0)).astype(np.uint8)


def quantize_rows(x: np.ndarray) -> Tuple[np.ndarray, np.ndarray]:
    """(codes [rows, K], scales [rows, K/128] fp32) of float64 rows."""
    b = x.reshape(x.shape[0], -1, BLOCK)
    amax = np.abs(b).max(axis=2)
    live = amax >= TINY
    y = np.where(live[:, :, None], b * (448.0 / np.where(live, amax, 1.0))[:, :, None], 0.0)
    return nearest(y, "e4m3").reshape(x.shape), np.where(live, amax / 448.0, 0.0).astype(np.float32)


def quantize_weight(w: np.ndarray) -> Tuple[np.ndarray, np.ndarray]:
    """(codes [N, K], scales [N/128, K/128] fp32) of one expert's weight."""
    N, K = w.shape
    codes, scales = np.zeros((N, K), np.uint8), np.zeros((N // BLOCK, K // BLOCK), np.float32)
    for i in range(N // BLOCK):
        for j in range(K // BLOCK):
            at = np.s_[i * BLOCK:(i + 1) * BLOCK, j * BLOCK:(j + 1) * BLOCK]
            amax = np.abs(w[at]).max()
            if amax >= TINY:
                codes[at] = nearest(w[at] * (448.0 / amax), "e4m3")
                scales[i, j] = amax / 448.0
    return codes, scales


def product(a: np.ndarray, sa: np.ndarray, w: np.ndarray, sw: np.ndarray) -> Tuple[np.ndarray, np.ndarray]:
    """(out, tol) [rows, N] of codes a [rows, K], w [N, K]; tol: how far a sum
    on the matrix core, then in fp32, may be off before its last rounding.

    Of 8 consecutive products the core cuts what lies below 2^-13 of the
    largest exponent sum 2^(ea + ew), where 2^e <= max(|value|, 2^-6) (e4m3's
    subnormals have the exponent -6): less than 8 * 2^-13 max|a| max|w| over
    the group, with the values' maxima taken apart.  The 16 groups of a block
    are joined in 24 bits by cuts (2^-23 of the magnitudes each), the blocks
    scaled and added in fp32 (scale, product and sum: 3 half steps and one a
    block)."""
    def spread(s, x):
        return np.repeat(s.astype(np.float64), x, axis=1)
    rows, K = a.shape
    va, vw = decode(a, "e4m3"), decode(w, "e4m3")
    fa, fw = spread(sa, BLOCK), np.repeat(spread(sw, BLOCK), BLOCK, axis=0)
    x, y = va * fa, vw * fw
    ga = np.maximum(np.abs(va).reshape(rows, -1, 8).max(2), 2.0 ** -6) * fa[:, ::8]
    gw = np.maximum(np.abs(vw).reshape(len(w), -1, 8).max(2), 2.0 ** -6) * fw[:, ::8]
    mag = np.abs(x) @ np.abs(y).T
    return x @ y.T, 8 * 2.0 ** -13 * (ga @ gw.T) + (16 * 2.0 ** -23 + (3 + K / BLOCK) * 2.0 ** -24) * mag


def noise(n: int, seed: int) -> np.ndarray:
    x = (np.arange(n, dtype=np.uint64) * 0x9E3779B9 + seed) & 0xFFFFFFFF
    x = ((x ^ (x >> np.uint64(16))) * 0x6A09E667) & 0xFFFFFFFF
    x = ((x ^ (x >> np.uint64(15))) * 0xBB67AE85) & 0xFFFFFFFF
    return x ^ (x >> np.uint64(16))


def moments8(x: np.ndarray, rnd16: np.ndarray, fmt: str) -> Tuple[np.ndarray, np.ndarray]:
    """(codes [n], scales [ceil(n/128)] float64) of flat moments x: |y| moved
    up by rnd / 2^16 of the format's step there and cut to whole steps."""
    _, top, man = FORMATS[fmt]
    n = x.size
    pad = -n % BLOCK
    b = np.pad(x, (0, pad)).reshape(-1, BLOCK)
    amax = np.abs(b).max(axis=1)
    live = amax >= TINY
    y = np.where(live[:, None], b * (top / np.where(live, amax, 1.0))[:, None], 0.0).reshape(-1)[:n]
    y = np.clip(y, -top, top)
    if fmt == "e5m2":
        y = np.where(x > 0, np.maximum(y, 2.0 ** -16), 0.0)
    m, e = np.frexp(np.abs(y))  # |y| = m 2^e, m in [0.5, 1)
    last = np.ldexp(1.0, np.maximum(e - 1, LOWEST[fmt]) - man)
    cut = np.where(y == 0, 0.0, np.floor(np.abs(y) / last + rnd16 / 65536.0) * last)
    return nearest(np.copysign(cut, y), fmt), np.where(live, amax / top, 0.0)


def adamw(p, g, m, v, *, lr, beta1, beta2, eps, weight_decay, step, grad_scale=1.0):
    """New (p, m, v) in float64."""
    g = np.asarray(g, np.float64) * grad_scale
    m = beta1 * m + (1 - beta1) * g
    v = beta2 * v + (1 - beta2) * g * g
    mh, vh = m / (1 - beta1 ** step), v / (1 - beta2 ** step)
    return p - lr * weight_decay * p - lr * mh / (np.sqrt(vh) + eps), m, v
