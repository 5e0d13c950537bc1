"""Orthogonalised updates by Newton-Schulz steps, in float64.  (Oracle: test use only.)

X <- G / (|G|_F + eps), then `steps` times X <- a X + (b A + c A A) X with A = X X^T.  Not of the S3R page, which leaves
the optimizer open.
"""
from __future__ import annotations

import numpy as np

COEFFS = (3.4445, -4.7750, 2.0315)


def newton_schulz(G, steps=5, coeffs=COEFFS, eps=1e-7, noise=0.0, seed=0):
    """The steps' result.  noise: every stored value of X, A and B = b A + c A A is off by a normal error of that size
    relative to the magnitudes that were added up for it (what a product in fewer bits does)."""
    a, b, c = (np.float64(np.float32(v)) for v in coeffs)
    r = np.random.default_rng(seed)
    G = np.asarray(G, np.float64)
    tall = G.shape[0] > G.shape[1]
    X = G.T if tall else G

    def off(v, size):
        return v + noise * r.normal(size=v.shape) * size if noise else v
    d = np.sqrt((X * X).sum()) + np.float64(np.float32(eps))
    X = X / d if d else X * 0
    X = off(X, np.abs(X))
    for _ in range(steps):
        A = X @ X.T
        A = off(A, np.abs(X) @ np.abs(X.T))
        B = b * A + c * (A @ A)
        B = off(B, np.abs(b * A) + abs(c) * (np.abs(A) @ np.abs(A)))
        X = off(a * X + B @ X, np.abs(a * X) + np.abs(B) @ np.abs(X))
    return X.T if tall else X
