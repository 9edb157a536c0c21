"""The Muon step in numpy and 64 bits: momentum, Newton-Schulz iteration, weight update."""
from __future__ import annotations

import numpy as np

MUON = (3.4445, -4.7750, 2.0315)


def orthogonalize(u: np.ndarray, K: int = 5, coeffs=MUON) -> np.ndarray:
    u = np.asarray(u, np.float64)
    x = u.T if u.shape[0] > u.shape[1] else u
    x = x / (np.sqrt((x * x).sum()) + 1e-7)
    for k in range(K):
        a, b, c = coeffs[k] if hasattr(coeffs[0], "__len__") else coeffs
        g = x @ x.T
        x = a * x + (b * g + c * (g @ g)) @ x
    return x.T if u.shape[0] > u.shape[1] else x
