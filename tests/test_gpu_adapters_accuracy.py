"""The adapters' products of two float32, one term to a sum, against float64.

A product goes through as six products of bfloat16 planes, the first one exact, the
other five added in float32, u = 2^-24 of the sum each; what is left out of it is at
most 2^-24 (1 + 2^-10), since the second plane is at most 2^-8 and the third at most
2^-17 of a value's power of two. Together below 6.1 u of the product (the partial
sums are at most 1 + 2^-7 of it). All other terms of the sums are zeros, which add
exactly, and scales are 1. The values have the planes that a truncating split would
leave largest.
"""
import numpy as np
import pytest
import torch

import bitlinear_absmean_ternarise_bit_amd as bl

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
TOL, FLOOR = 6.1 * 2.0 ** -24, 2.0 ** -132
L = 64


def values(power=0):
    """1 + 2^-7 - 2^-23 and its like: low bits set below the eighth, other high bits, signs."""
    rng = np.random.default_rng(3)
    bits = np.where(np.arange(L) % 3 == 0, 0x3F80FFFF - rng.integers(0, 64, L), 0x3F80FFFF + (rng.integers(0, 127, L) << 16))
    v = bits.astype(np.uint32).view(np.float32) * np.float32(2.0 ** power)
    return v * np.where(rng.random(L) < 0.5, -1, 1).astype(np.float32)


def circulant(v, rows, cols):
    """[i, j]: v[(i + j) % L]"""
    return v[(np.arange(rows)[:, None] + np.arange(cols)) % L]


def gpu(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(DEV)


def close(got, ref, power=0):
    err = np.abs(got.double().cpu().numpy() - ref)
    assert (err <= TOL * np.abs(ref) + (FLOOR if power < -110 else 0.0)).all(), float((err / np.maximum(np.abs(ref), 1e-300)).max() * 2.0 ** 24)


def diagonal(v):
    return np.diag(v).astype(np.float32)


# `power`: also values whose last planes are below the smallest normal number
@pytest.mark.parametrize("power", [0, 100, -60, -112])
def test_first_product(power):
    a, b = values(power), values()
    one, ids = torch.ones(1, device=DEV), torch.zeros(L, dtype=torch.int32, device=DEV)
    down = circulant(b, L, L)
    ref = a.astype(np.float64)[:, None] * down.T.astype(np.float64)  # T[m, r] = X[m, m] down[r, m]
    ads = (gpu(down[None]), torch.zeros(1, L, 8, device=DEV), one)
    for M in (L, 5 * L):  # a group of 16 tokens, and of 64
        x = gpu(np.tile(diagonal(a), (M // L, 1)))
        _, t = bl.adapters_forward(x, ads, ids.repeat(M // L), torch.zeros(M, 8, device=DEV), return_low=True)
        close(t, np.tile(ref, (M // L, 1)), power)


@pytest.mark.parametrize("R", [16, L])
@pytest.mark.parametrize("power", [0, 100, -60, -112])
def test_second_product(power, R):
    a, b = values(power)[:R], values()
    down = diagonal(a)  # T = diag(a): one times a value, the sum of its planes
    one = torch.ones(1, device=DEV)
    for M, N in ((2 * R, 100), (320, 100), (1024, 4096)):
        x = gpu(np.tile(np.eye(R), (M // R, 1)))
        ids = torch.zeros(M, dtype=torch.int32, device=DEV)
        up = circulant(b, R, N)
        ref = np.tile(a.astype(np.float64)[:, None] * up.astype(np.float64), (M // R, 1))
        ads = (gpu(down[None]), gpu(up[None]), one)
        y, t = bl.adapters_forward(x, ads, ids, torch.zeros(M, N, device=DEV), return_low=True)
        low = np.tile(down.T, (M // R, 1))
        assert (np.abs(t.cpu().numpy().astype(np.float64) - low) <= (2.0 ** -134 if power < -110 else 0.0)).all()
        close(y, ref, power)
        # beside a projection of scale 0
        packed, _ = bl.quantize_weights(torch.randn(N, R, device=DEV))
        close(bl.adapted_forward(x, packed, torch.zeros(1, device=DEV), ads, ids), ref, power)


@pytest.mark.parametrize("power", [0, 100, -60, -112])
def test_gradients(power):
    a, b = values(power), values()
    one, ids = torch.ones(1, device=DEV), torch.zeros(L, dtype=torch.int32, device=DEV)
    eye, diag, other = gpu(np.eye(L)), gpu(diagonal(a)), gpu(circulant(b, L, L))
    ref = a.astype(np.float64)[:, None] * circulant(b, L, L).astype(np.float64)
    # V = diag(a); dX = V down, ddown = V^T X
    dx, dd, _ = bl.adapters_backward(eye, other, diag, (other[None], diag[None], one), ids)
    close(dx, ref, power)
    close(dd[0], ref, power)
    # dup = T^T dY
    _, _, du = bl.adapters_backward(other, eye, diag, (other[None], diag[None], one), ids, need_dx=False)
    close(du[0], ref, power)


def test_the_largest_values_stay_finite():
    # they round to more than the largest bfloat16
    top = np.finfo(np.float32).max
    x = gpu([[top, 0], [0, -top], [3.3961777e38, 0], [0, 3.39e38]])
    w = np.array([[0.5, 0.3]], np.float32)
    ids = torch.zeros(4, dtype=torch.int32, device=DEV)
    y, t = bl.adapters_forward(x, (gpu(w[None]), torch.zeros(1, 1, 8, device=DEV), torch.ones(1, device=DEV)), ids,
                               torch.zeros(4, 8, device=DEV), return_low=True)
    close(t, x.double().cpu().numpy() @ w.T.astype(np.float64))
    wide = np.zeros((1, 16), np.float32)
    wide[0, ::2] = 0.5
    wide[0, 1::2] = 0.3
    wx = torch.zeros(4, 16, device=DEV)
    wx[:, :2] = x
    _, t = bl.adapters_forward(wx, (gpu(wide[None]), torch.zeros(1, 1, 8, device=DEV), torch.ones(1, device=DEV)), ids,
                               torch.zeros(4, 8, device=DEV), return_low=True)
    close(t, x.double().cpu().numpy() @ w.T.astype(np.float64))
    for v in (float("inf"), -float("inf"), float("nan")):
        wx[1, 1] = v
        _, t2 = bl.adapters_forward(wx, (gpu(wide[None]), torch.zeros(1, 1, 8, device=DEV), torch.ones(1, device=DEV)),
                                    ids, torch.zeros(4, 8, device=DEV), return_low=True)
        assert torch.equal(t2[[0, 2, 3]], t[[0, 2, 3]]) and not torch.isfinite(t2[1]).any()
