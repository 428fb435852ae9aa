"""Pins of the oracle for the operators around BitLinear: layer norm against
torch's float64 one and central differences, the saved format against its
bounds, exact ties and a literal rendering with fractions."""
import os
import re
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import block as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("M,K", [(1, 1), (3, 7), (4, 64), (2, 129)])
def test_layer_norm_and_gradients(M, K):
    rng = np.random.default_rng(M * 1000 + K)
    X, dY = rng.standard_normal((2, M, K))
    w, b = rng.standard_normal((2, K))
    eps = 1e-3
    Y, mean, rstd = B.layer_norm(X, w, b, eps)
    tx, tw, tb = (torch.from_numpy(a).requires_grad_() for a in (X, w, b))
    ty = torch.nn.functional.layer_norm(tx, (K,), tw, tb, float(np.float32(eps)))
    ty.backward(torch.from_numpy(dY))
    assert np.allclose(Y, ty.detach().numpy(), rtol=0, atol=1e-12)
    dX, dw, db = B.layer_norm_backward(dY, X, mean, rstd, w)
    for got, ref in ((dX, tx.grad), (dw, tw.grad), (db, tb.grad)):
        assert np.allclose(got, ref.numpy(), rtol=0, atol=1e-10)
    # central differences of sum(Y dY) along a direction: an error of the order h^2
    v, h = rng.standard_normal((M, K)), 1e-5
    up, down = (B.layer_norm(X + s * h * v, w, b, eps)[0] for s in (1, -1))
    assert abs(((up - down) * dY).sum() / (2 * h) - (dX * v).sum()) < 1e-6 * (1 + np.abs(dX * v).sum())


def test_relu2_gradient_by_differences():
    rng = np.random.default_rng(3)
    H, dA = rng.standard_normal((2, 5, 33))
    h = 1e-6
    diff = (np.maximum(H + h, 0) ** 2 - np.maximum(H - h, 0) ** 2) / (2 * h) * dA
    assert np.allclose(B.relu2_backward(dA, H), diff, rtol=0, atol=1e-5)


@pytest.mark.parametrize("K", [1, 63, 64, 65, 200])
def test_saved_format(K):
    rng = np.random.default_rng(K)
    X = (rng.standard_normal((4, K)) * 10.0 ** rng.integers(-20, 20, (4, 1))).astype(np.float32)
    X[0, 0] = 0 if K > 1 else 1
    codes, scales = B.save8(X)
    G = -(-K // 64)
    assert codes.shape == (4, 64 * G) and scales.shape == (4, G)
    assert not codes[:, K:].any() and np.abs(codes.astype(int)).max() == 127
    back = B.restore8(codes, scales, K)
    step = np.repeat(scales, 64, axis=1)[:, :K].astype(np.float64)
    # the code is off by half a step at most; s and scale are rounded once each
    assert np.all(np.abs(back.astype(np.float64) - X) <= step / 2 * (1 + 2.0 ** -15))
    # the nearest integer of the exact product, literally
    for m in range(4):
        for k in range(K):
            s = np.float32(127.0) / np.abs(X[m, k // 64 * 64:k // 64 * 64 + 64]).max()
            assert codes[m, k] == round(Fraction(float(X[m, k])) * Fraction(float(s)))


def test_saved_special_groups():
    X = np.zeros((6, 64), np.float32)
    X[1, 5] = 2.0 ** -101          # below the smallest kept magnitude
    X[2, 5] = 2.0 ** -100
    X[3, 5] = np.nan
    X[4, 5] = -np.inf
    X[5, :3] = [3.4e38, -3.4e38, 1e38]
    codes, scales = B.save8(X)
    assert not codes[0].any() and scales[0, 0] == 0 and not codes[1].any() and scales[1, 0] == 0
    assert codes[2, 5] == 127 and scales[2, 0] > 0
    back = B.restore8(codes, scales, 64)
    assert np.isnan(back[3]).all() and np.isnan(back[4]).all() and np.isfinite(back[5]).all()
    # ties to even: with amax 127, s is 1 and halves fall on ties
    T = np.zeros((1, 64), np.float32)
    T[0, :6] = [127, 0.5, 1.5, 2.5, -0.5, -2.5]
    assert B.save8(T)[0][0, :6].tolist() == [127, 0, 2, 2, 0, -2]


def test_saved_bound_of_the_header():
    """|x~ - x| <= scale / 2 (1 + 2^-14), where the roundings add up: values beside the borders between large codes.
    With d0..d3 the relative errors of fp32(1/127) (2^-28), s, scale and x~ (2^-24 each) and r <= 1/2 the rounding of
    x s:  x~ - x = x ((1 + d0)(1 + d1)(1 + d2)(1 + d3) - 1) + r scale (1 + d3)  and  |x| <= 127 scale (1 + 2^-23),
    which is scale / 2 (1 + 2^-24 (1 + 254 * 3.07)) at most, below 1 + 2^-14 = 1 + 1024 * 2^-24."""
    text = " ".join(open(os.path.join(ROOT, "include", "bitlinear_block.h")).read().replace("*", " ").split())
    stated = re.search(r"\|x~ - x\| <= scale / 2 \(1 \+ 2\^-(\d+)\)", text)
    assert stated
    rng = np.random.default_rng(14)
    n = 4000
    amax = (rng.uniform(1, 2, n) * 2.0 ** rng.integers(-90, 120, n)).astype(np.float32)
    amax[0] = float.fromhex("0x1.159004p+0")
    X = np.zeros((n, 64), np.float32)
    X[:, 0] = amax
    s = (np.float32(127) / amax).astype(np.float64)
    for j, code in enumerate(range(64, 127)):
        border = ((code + 0.5) / s).astype(np.float32)
        X[:, 1 + j] = np.nextafter(border, np.float32(np.inf if j % 2 else 0))
    X[0, 1] = float.fromhex("0x1.1248c6p+0")
    back = B.restore8(*B.save8(X), 64).astype(np.float64)
    half = B.save8(X)[1].astype(np.float64) / 2
    worst = (np.abs(back - X) / half - 1).max()
    assert 2.0 ** -15 < worst <= 2.0 ** -int(stated.group(1)), worst * 2 ** 24
