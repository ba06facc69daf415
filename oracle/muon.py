"""One step of the optimiser with an orthogonalised update in float64
(include/moelora.h states the definition), rounds run on the update itself.
Test infrastructure only."""
from __future__ import annotations

from typing import Tuple

import numpy as np

QUINTIC = (3.4445, -4.7750, 2.0315)


def orthogonalise(U: np.ndarray, eps: float, rounds: int, abc=QUINTIC) -> np.ndarray:
    """U [m, n] through the rounds."""
    a, b, c = abc
    X = U / (np.sqrt((U * U).sum()) + eps)
    for _ in range(rounds):
        if X.shape[0] <= X.shape[1]:
            S = X @ X.T
            X = a * X + (b * S + c * S @ S) @ X
        else:
            S = X.T @ X
            X = a * X + X @ (b * S + c * S @ S)
    return X


def by_singular_values(U: np.ndarray, eps: float, rounds: int, abc=QUINTIC) -> np.ndarray:
    """The same from the singular value decomposition: the polynomial of each singular value."""
    a, b, c = abc
    u, s, v = np.linalg.svd(U, full_matrices=False)
    s = s / (np.sqrt((s * s).sum()) + eps)
    for _ in range(rounds):
        s = a * s + b * s ** 3 + c * s ** 5
    return (u * s) @ v


def slope(rounds: int, abc=QUINTIC) -> float:
    """The largest slope of the rounds' polynomial of a singular value in [0, 1]: how far the result moves, in the
    root of the sum of squares, for a change of the normalised update."""
    a, b, c = abc
    s, d = np.linspace(0, 1, 20001), np.ones(20001)
    for _ in range(rounds):
        d = d * (a + 3 * b * s ** 2 + 5 * c * s ** 4)
        s = a * s + b * s ** 3 + c * s ** 5
    return float(np.abs(d).max())


def step(p, grad, momentum, *, lr, mu, nesterov, weight_decay, rms, eps, grad_scale, rounds=5,
         abc=QUINTIC) -> Tuple[np.ndarray, np.ndarray, np.ndarray]:
    """One matrix: (p, momentum, orthogonalised update) after the step."""
    g = grad_scale * grad
    M = mu * momentum + g
    U = g + mu * M if nesterov else M
    X = orthogonalise(U, eps, rounds, abc)
    return p - lr * (rms * np.sqrt(max(p.shape)) * X + weight_decay * p), M, X
