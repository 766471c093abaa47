"""CPU oracle for the Newton-Schulz orthogonalisation of factors.

TEST INFRASTRUCTURE.  Only the tests may import or call this module; it
shares no code with the library.

The definition itself in float64: X = N / (|N|_F + eps), then `steps` times
X <- c0 X + (c1 G + c2 G^2) X with G = X X^T.
"""
from __future__ import annotations

import numpy as np


def newton_schulz(N, steps, coef, eps):
    X = np.asarray(N, np.float64)
    X = X / (np.sqrt(np.sum(X * X)) + eps)
    for _ in range(steps):
        G = X @ X.T
        X = coef[0] * X + (coef[1] * G + coef[2] * G @ G) @ X
    return X


def left_factor(N, steps, coef, eps):
    """Q with newton_schulz(N) = Q N / (|N|_F + eps) (all iterates are
    polynomials in the first Gram matrix)."""
    X = np.asarray(N, np.float64)
    X = X / (np.sqrt(np.sum(X * X)) + eps)
    Q = np.eye(X.shape[0])
    G = X @ X.T
    for _ in range(steps):
        P = coef[0] * np.eye(X.shape[0]) + coef[1] * G + coef[2] * G @ G
        Q, G = P @ Q, P @ G @ P
    return Q


def tolerance(N, steps, coef, eps):
    """The most an element of the result may be off when the r x r matrices
    are computed in float64 and Q, N / norm and their product in float32: Q and
    N / norm are rounded (the latter by a rounded factor), the product sums r
    terms, in any order; and a Gram matrix off by (d + r) 2^-53 moves Q by at
    most (|c1| + 2 |c2|) times that, amplified by c0^2 a step in G and c0 a
    step in Q."""
    X = np.asarray(N, np.float64)
    r, d = X.shape
    X = X / (np.sqrt(np.sum(X * X)) + eps)
    Q = np.abs(left_factor(N, steps, coef, eps))
    amp = (abs(coef[1]) + 2 * abs(coef[2])) * max(1.0, abs(coef[0])) ** (3 * (steps - 1))
    return (r + 6) * 2.0 ** -24 * (Q @ np.abs(X)) + \
        amp * (d + r) * 2.0 ** -53 * np.sqrt(np.sum(X * X, axis=0))[None, :]
