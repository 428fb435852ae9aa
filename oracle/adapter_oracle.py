"""Plain CPU oracle for low-rank adapters and dropout.

TEST INFRASTRUCTURE ONLY, as :mod:`oracle.bitlinear_oracle`.  float64 products
token by token and adapter by adapter, nothing rounded; the generator in Python
integers, from the published description of Philox4x32-10.
"""
from __future__ import annotations

import numpy as np


def _of(rows, A):
    """(adapter, its tokens) of every adapter that has some."""
    rows = np.asarray(rows)
    return [(a, np.flatnonzero(rows == a)) for a in range(A) if (rows == a).any()]


def low(X, rows, down):
    """T [M, R]: X[m] down[a]^T, zeros without an adapter."""
    X, down = np.asarray(X, np.float64), np.asarray(down, np.float64)
    T = np.zeros((X.shape[0], down.shape[1]))
    for a, at in _of(rows, down.shape[0]):
        T[at] = X[at] @ down[a].T
    return T


def added(T, rows, up, scales):
    """scale[a] T[m] up[a], zeros without an adapter."""
    up = np.asarray(up, np.float64)
    Y = np.zeros((T.shape[0], up.shape[2]))
    for a, at in _of(rows, up.shape[0]):
        Y[at] = float(scales[a]) * (np.asarray(T, np.float64)[at] @ up[a])
    return Y


def grads(left, right, rows, A, scales):
    """[A, R, C]: scale[a] times the sum over a's tokens of left[m]^T right[m]."""
    left, right = np.asarray(left, np.float64), np.asarray(right, np.float64)
    G = np.zeros((A, left.shape[1], right.shape[1]))
    for a, at in _of(rows, A):
        G[a] = float(scales[a]) * (left[at].T @ right[at])
    return G


def backward(dY, X, rows, down, up, scales):
    """(dX, ddown, dup) in float64."""
    V = low(dY, rows, up)
    return (added(V, rows, down, scales), grads(V, X, rows, len(down), scales),
            grads(low(X, rows, down), dY, rows, len(down), scales))


def philox(counter: int, offset: int, seed: int):
    """The four words of Philox4x32-10."""
    w = 1 << 32
    c = [counter % w, counter // w % w, offset % w, offset // w % w]
    k = [seed % w, seed // w % w]
    for _ in range(10):
        p, q = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [q // w ^ c[1] ^ k[0], q % w, p // w ^ c[3] ^ k[1], p % w]
        k = [(k[0] + 0x9E3779B9) % w, (k[1] + 0xBB67AE85) % w]
    return c


def kept(first: int, n: int, p: float, seed: int, offset: int) -> np.ndarray:
    """Which of the values first .. first + n - 1 are kept."""
    out = np.empty(n, bool)
    block, words = -1, None
    for i in range(n):
        if (first + i) // 4 != block:
            block = (first + i) // 4
            words = philox(block, offset, seed)
        out[i] = words[(first + i) % 4] >= int(p * 2.0 ** 32 + 0.5)
    return out


def dropout(x, p, seed, offset=0, residual=None):
    """float32 results, each step rounded as the definition has it."""
    x = np.asarray(x, np.float32)
    scale = np.float32(1.0 / (1.0 - p))
    y = np.where(kept(0, x.size, p, seed, offset).reshape(x.shape), x * scale, np.float32(0))
    return y if residual is None else y + np.asarray(residual, np.float32)
