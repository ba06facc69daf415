"""Top-k routing, expert loads, balance loss and their gradient in float64, one
token and one expert at a time (include/moelora.h states the definition).
Test infrastructure only."""
from __future__ import annotations

from typing import Dict, Optional, Sequence

import numpy as np


def token_active(l: np.ndarray) -> bool:
    return not (np.isnan(l).any() or (l == np.inf).any()) and bool((l > -np.inf).any())


def softmax(l: np.ndarray) -> np.ndarray:
    e = np.exp(l - l.max())
    return e / e.sum()


def forward(logits: np.ndarray, k: int, renorm: bool, roots: Optional[Sequence[int]] = None,
            valid: Optional[np.ndarray] = None) -> Dict[str, np.ndarray]:
    """logits [T, E] (any float type, used as float64)."""
    l = np.asarray(logits, dtype=np.float64)
    T, E = l.shape
    roots = [0, T] if roots is None else list(roots)
    na = len(roots) - 1
    out = {"topk_idx": np.full((T, k), -1, np.int32), "topk_w": np.zeros((T, k)), "p": np.zeros((T, E)),
           "counts": np.zeros((na, E), np.int32), "active": np.zeros(na, np.int32), "loss": np.zeros(na), "bad": 0}
    for a in range(na):
        mass = np.zeros(E)
        for t in range(roots[a], roots[a + 1]):
            if valid is not None and not valid[t]:
                continue
            if not token_active(l[t]):
                out["bad"] += int(np.isnan(l[t]).any() or (l[t] == np.inf).any())
                continue
            order = sorted((e for e in range(E) if l[t, e] > -np.inf), key=lambda e: (-l[t, e], e))[:k]
            p = softmax(l[t])
            w = p[order] / (p[order].sum() if renorm else 1.0)
            out["topk_idx"][t, :len(order)] = order
            out["topk_w"][t, :len(order)] = w
            out["p"][t] = p
            out["counts"][a, order] += 1
            out["active"][a] += 1
            mass += p
        n = max(1, int(out["active"][a]))
        out["loss"][a] = E / (k * n * n) * float(out["counts"][a] @ mass)
    return out


def backward(logits: np.ndarray, fwd: Dict[str, np.ndarray], k: int, renorm: bool, grad_w: Optional[np.ndarray],
             grad_loss: Optional[np.ndarray], roots: Optional[Sequence[int]] = None):
    """(gradient, scale): the gradient to the logits, and the sum of the
    magnitudes of the terms that make each element up."""
    T, E = np.shape(logits)
    roots = [0, T] if roots is None else list(roots)
    grad, scale = np.zeros((T, E)), np.zeros((T, E))
    for a in range(len(roots) - 1):
        n = max(1, int(fwd["active"][a]))
        u = np.zeros(E) if grad_loss is None else grad_loss[a] * E / (k * n * n) * fwd["counts"][a]
        for t in range(roots[a], roots[a + 1]):
            p = fwd["p"][t]  # zeros for an inactive token
            grad[t] = p * (u - p @ u)
            scale[t] = p * (np.abs(u) + p @ np.abs(u))
            sel = fwd["topk_idx"][t][fwd["topk_idx"][t] >= 0]
            if grad_w is None or sel.size == 0:
                continue
            g = grad_w[t, :sel.size]
            if renorm:
                w = p[sel] / p[sel].sum()
                grad[t, sel] += w * (g - w @ g)
                scale[t, sel] += w * (np.abs(g) + w @ np.abs(g))
            else:
                grad[t, sel] += p[sel] * g
                grad[t] -= p * (p[sel] @ g)
                scale[t, sel] += p[sel] * np.abs(g)
                scale[t] += p * (p[sel] @ np.abs(g))
    return grad, scale
