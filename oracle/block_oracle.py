"""Plain CPU oracle for the operators around BitLinear: layer norm, ReLU^2 and
8-bit saved activations, with their gradients.

TEST INFRASTRUCTURE ONLY, as :mod:`oracle.bitlinear_oracle`.  Written from the
formulas in float64 (float32 only where the saved format's definition says so);
inputs are numpy arrays, outputs float64 and not rounded.

[PMV] (the produtoramaxvision.com.br article on BitNet b1.58, its section on
trade-offs) leaves the norm outside BitLinear and names RMSNorm; [MBC] (the
shadowgraph.io page, bit_layers.py) gives ReLU^2 as the activation.  The norm
here is another one, the ordinary layer norm (mean, biased variance, bias): the
library's own choice, as the saved format is.
"""
from __future__ import annotations

import numpy as np

SAVED_GROUP = 64
SAVED_SMALLEST = 2.0 ** -100  # a group whose largest magnitude is below it is saved as zeros


def save8(X: np.ndarray):
    """(codes int8 [M, Kp], scales float32 [M, G]) of float32 X [M, K]."""
    X = np.asarray(X, np.float32)
    M, K = X.shape
    G = -(-K // SAVED_GROUP)
    codes = np.zeros((M, G * SAVED_GROUP), np.int8)
    scales = np.zeros((M, G), np.float32)
    for g in range(G):
        part = X[:, g * SAVED_GROUP:min(K, (g + 1) * SAVED_GROUP)]
        bad = ~np.isfinite(part).all(axis=1)
        amax = np.abs(np.where(bad[:, None], 0, part)).max(axis=1)
        live = amax >= SAVED_SMALLEST
        with np.errstate(divide="ignore", over="ignore"):
            s = np.where(live, np.float32(127.0) / amax, np.float32(0)).astype(np.float32)
        scales[:, g] = np.where(live, amax * np.float32(1.0 / 127.0), np.float32(0))
        scales[bad, g] = np.nan
        part = np.where(bad[:, None], 0, part)
        # a float32 product is exact in float64; rint is half to even
        codes[:, g * SAVED_GROUP:g * SAVED_GROUP + part.shape[1]] = np.rint(
            part.astype(np.float64) * s[:, None].astype(np.float64)).astype(np.int8)
    return codes, scales


def restore8(codes: np.ndarray, scales: np.ndarray, K: int) -> np.ndarray:
    """float32 [M, K]: fp32(scale * code)."""
    s = np.repeat(np.asarray(scales, np.float32), SAVED_GROUP, axis=1)[:, :K]
    return s * codes[:, :K].astype(np.float32)


def layer_norm(X, weight=None, bias=None, eps=1e-5):
    """(Y, mean, rstd) in float64."""
    X = np.asarray(X, np.float64)
    mean = X.mean(axis=1)
    d = X - mean[:, None]
    rstd = 1.0 / np.sqrt((d * d).mean(axis=1) + float(np.float32(eps)))
    Y = d * rstd[:, None]
    if weight is not None:
        Y = Y * np.asarray(weight, np.float64)
    if bias is not None:
        Y = Y + np.asarray(bias, np.float64)
    return Y, mean, rstd


def layer_norm_backward(dY, X, mean, rstd, weight=None):
    """(dX, dweight, dbias) in float64, with the given mean and rstd."""
    dY, X = np.asarray(dY, np.float64), np.asarray(X, np.float64)
    mean, rstd = np.asarray(mean, np.float64)[:, None], np.asarray(rstd, np.float64)[:, None]
    xhat = (X - mean) * rstd
    g = dY if weight is None else dY * np.asarray(weight, np.float64)
    dX = rstd * (g - g.mean(axis=1, keepdims=True) - xhat * (g * xhat).mean(axis=1, keepdims=True))
    return dX, (dY * xhat).sum(axis=0), dY.sum(axis=0)


def relu2_backward(dA, H):
    """dA * 2 max(H, 0) in float64 (a NaN in H stays one)."""
    H = np.asarray(H, np.float64)
    return np.asarray(dA, np.float64) * 2.0 * np.where(H <= 0, 0.0, H)
