"""Plain CPU oracle for the gated feed-forward block and its gradients.

TEST INFRASTRUCTURE ONLY, as :mod:`oracle.bitlinear_oracle`.  G and U are the
BitLinear outputs with their float32 roundings (dequant_f32); ReLU^2 and its
gradients are the float32 products of their definition, the SiLU form is float64
and not rounded.
"""
from __future__ import annotations

import numpy as np

from .bitlinear_oracle import absmax_quantize, dequant_f32, zero_gemm


def projections(X, q_gate, g_gate, q_up, g_up):
    """(G, U) float32 from ternary codes [F, D] and scales."""
    gA, Xq, _ = absmax_quantize(X)
    return dequant_f32(zero_gemm(Xq, q_gate), g_gate, gA), dequant_f32(zero_gemm(Xq, q_up), g_up, gA)


def sigmoid(g):
    """In float64, without overflow."""
    g = np.asarray(g, np.float64)
    with np.errstate(over="ignore"):
        return np.where(g >= 0, 1.0 / (1.0 + np.exp(-np.abs(g))), np.exp(-np.abs(g)) / (1.0 + np.exp(-np.abs(g))))


def hidden(act, G, U):
    """act(G) * U: float32 for relu2, float64 for silu."""
    G, U = np.asarray(G, np.float32), np.asarray(U, np.float32)
    if act == "relu2":
        r = np.where(G <= 0, np.float32(0), G)
        return (r * r).astype(np.float32) * U
    return G.astype(np.float64) * sigmoid(G) * U.astype(np.float64)


def hidden_backward(act, dH, G, U):
    """(dG, dU): float32 for relu2, float64 for silu."""
    dH, G, U = (np.asarray(v, np.float32) for v in (dH, G, U))
    if act == "relu2":
        r = np.where(G <= 0, np.float32(0), G)
        return dH * (U * (np.float32(2) * r)), dH * (r * r)
    d, g, u, s = dH.astype(np.float64), G.astype(np.float64), U.astype(np.float64), sigmoid(G)
    return d * u * s * (1.0 + g * (1.0 - s)), d * g * s


def input_backward(dG, dU, q_gate, g_gate, q_up, g_up):
    """dX in float64: gamma_gate (dG W_gate) + gamma_up (dU W_up)."""
    p = lambda d, q, g: (np.asarray(d, np.float64) @ np.asarray(q, np.float64)) * float(np.float32(g))  # noqa: E731
    return p(dG, q_gate, g_gate) + p(dU, q_up, g_up)
