"""Expert products on the pool's rows and their gradients in float64
(include/moelora.h states the definitions).  Test infrastructure only.

Each function also returns a bound of what sums in fp32 may be off: K terms
added one after another in any grouping, each addition off by at most a unit
of the sum's last place (2^-23), are off by at most K 2^-23 sum |terms|.
"""
from __future__ import annotations

from typing import Tuple

import numpy as np


def product(a: np.ndarray, w: np.ndarray) -> Tuple[np.ndarray, np.ndarray]:
    """a [rows, K] times w [N, K] transposed."""
    return a @ w.T, a.shape[1] * 2.0 ** -23 * (np.abs(a) @ np.abs(w).T)


def weight_grad(g: np.ndarray, a: np.ndarray) -> Tuple[np.ndarray, np.ndarray]:
    """g [rows, N] transposed times a [rows, K]; no rows: zeros."""
    return g.T @ a, max(1, a.shape[0]) * 2.0 ** -23 * (np.abs(g).T @ np.abs(a))
