"""64-bit CPU oracles of the operators between and behind the adapter layers:
the gated feed-forward block, softmax cross entropy, gradient clipping.

TEST INFRASTRUCTURE, plain definitions in float64, sharing no code with the
HIP library.
"""
from __future__ import annotations

import math

import numpy as np

_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def _sigmoid(x):
    """1 / (1 + e^-x), and 1 minus it, without cancellation."""
    e = np.exp(-np.abs(x))
    big, small = 1 / (1 + e), e / (1 + e)
    return np.where(x >= 0, big, small), np.where(x >= 0, small, big)


def activation(name: str, x):
    """act(x), act'(x) and the argument whose exponential the activation takes."""
    if name == "silu":
        p, q = _sigmoid(x)
        return x * p, p + x * p * q, x
    if name == "gelu":
        p = 0.5 * _erfc(-x / math.sqrt(2))
        return x * p, p + x * np.exp(-x * x / 2) / math.sqrt(2 * math.pi), x * x / 2
    # (1 + tanh z) / 2 = 1 / (1 + e^-2z)
    k, c = math.sqrt(2 / math.pi), 0.044715
    z = 2 * k * (x + c * x ** 3)
    p, q = _sigmoid(z)
    return x * p, p + x * p * q * 2 * k * (1 + 3 * c * x * x), z


def gated(X, W_gate_t, W_up_t, act: str, adapters=None):
    """g, u and H.  adapters(p, X) -> the adapters' term of projection p (0
    gate, 1 up)."""
    g, u = X @ W_gate_t.T, X @ W_up_t.T
    if adapters is not None:
        g, u = g + adapters(0, X), u + adapters(1, X)
    return g, u, activation(act, g)[0] * u


def gated_grad(dH, g, u, act: str):
    """dg and du."""
    a, slope, _ = activation(act, g)
    return dH * u * slope, dH * a


def cross_entropy(X, W_t, targets, weights=None, scale: float = 1.0):
    """loss [T], dX [T][d] and softmax [T][V] (zero rows for ignored tokens)."""
    T, V = X.shape[0], W_t.shape[0]
    loss, dX, P = np.zeros(T), np.zeros_like(X), np.zeros((T, V))
    for t in range(T):
        y, w = int(targets[t]), 1.0 if weights is None else float(weights[t])
        if y >= V:
            loss[t] = np.nan
        if y < 0 or y >= V or w == 0:
            continue
        l = scale * (W_t @ X[t])
        top = l.max()
        e = np.exp(l - top)
        P[t] = e / e.sum()
        others = np.delete(np.exp(l - l[y]), y).sum() if l[y] - top > -600 else np.inf
        loss[t] = w * (math.log1p(others) if others < 1e200 else math.log(e.sum()) + top - l[y])
        c = P[t].copy()
        c[y] = -np.delete(P[t], y).sum()
        dX[t] = w * scale * (c @ W_t)
    return loss, dX, P


def clip(layers, adapters, max_rank: int, max_norm: float, together: bool):
    """layers: dicts with rank, page_start, page_ids, n_pages, A, B (float64
    pages).  Norms [M + 1], infinite where float32 has no such number, and the
    clipped pages (a new dict of A and B for each layer; other pages as they were)."""
    M = len(adapters)
    taken = []
    for l in layers:
        N = len(l["rank"])
        here = {}
        for m, a in enumerate(adapters):
            a = int(a)
            if a < 0 or a >= N or a in [int(x) for x in adapters[:m]]:
                continue
            r, s = int(l["rank"][a]), int(l["page_start"][a])
            if r < 1 or r > max_rank or int(l["page_start"][a + 1]) - s != r or s < 0 or s + r > len(l["page_ids"]):
                continue
            p = np.asarray(l["page_ids"][s:s + r])
            if (p < 0).any() or (p >= l["n_pages"]).any():
                continue
            here[m] = p
        taken.append(here)
    square = np.zeros(M)
    for l, here in zip(layers, taken):
        for m, p in here.items():
            square[m] += (l["A"][p] ** 2).sum() + (l["B"][p] ** 2).sum()
    norm = np.sqrt(np.append(square, square.sum()))
    with np.errstate(over="ignore"):
        norm[np.isinf(norm.astype(np.float32))] = np.inf
    out = []
    for l, here in zip(layers, taken):
        o = {"A": l["A"].copy(), "B": l["B"].copy()}
        for m, p in here.items():
            n = norm[M] if together else norm[m]
            c = max_norm / n if np.isfinite(n) and n > max_norm else 1.0
            for f in "AB":
                o[f][p] = l[f][p] * c
        out.append(o)
    return norm, out, taken
