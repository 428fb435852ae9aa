"""The gated block's oracle against torch in float64, differences and the FFN block's oracle."""
import numpy as np
import pytest
import torch

import oracle as O
from oracle import gated as GO


def problem(M, D, F, seed):
    rng = np.random.default_rng(seed)
    X = rng.standard_normal((M, D)).astype(np.float32)
    qs = [rng.integers(-1, 2, (F, D)).astype(np.int8) for _ in range(2)]
    return X, qs, [np.float32(0.013), np.float32(0.017)]


@pytest.mark.parametrize("act", ["relu2", "silu"])
@pytest.mark.parametrize("M,D,F", [(1, 1, 1), (3, 70, 33), (5, 128, 64)])
def test_hidden_and_gradients_against_torch(act, M, D, F):
    X, (qg, qu), (gg, gu) = problem(M, D, F, M * D)
    G, U = GO.projections(X, qg, gg, qu, gu)
    gA, Xq, _ = O.absmax_quantize(X)
    # the projections are the BitLinear outputs of each matrix on its own
    assert np.array_equal(G, O.dequant_f32(O.zero_gemm_naive(Xq, qg), gg, gA))
    assert np.array_equal(U, O.dequant_f32(O.zero_gemm_naive(Xq, qu), gu, gA))
    g = torch.from_numpy(G).double().requires_grad_()
    u = torch.from_numpy(U).double().requires_grad_()
    h = (torch.relu(g) ** 2 if act == "relu2" else torch.nn.functional.silu(g)) * u
    np.testing.assert_allclose(GO.hidden(act, G, U), h.detach().numpy(), rtol=3e-7, atol=1e-30)
    dH = np.random.default_rng(9).standard_normal((M, F)).astype(np.float32)
    h.backward(torch.from_numpy(dH).double())
    dG, dU = GO.hidden_backward(act, dH, G, U)
    np.testing.assert_allclose(dG, g.grad.numpy(), rtol=3e-7, atol=1e-12)
    np.testing.assert_allclose(dU, u.grad.numpy(), rtol=3e-7, atol=1e-12)
    # the input's gradient: that of the dequantised product, codes and scales held
    x = torch.zeros((M, D), dtype=torch.float64, requires_grad=True)
    wg, wu = torch.from_numpy(qg).double() * float(gg), torch.from_numpy(qu).double() * float(gu)
    ((x @ wg.T) * torch.from_numpy(np.asarray(dG, np.float64))
     + (x @ wu.T) * torch.from_numpy(np.asarray(dU, np.float64))).sum().backward()
    np.testing.assert_allclose(GO.input_backward(dG, dU, qg, gg, qu, gu), x.grad.numpy(), rtol=1e-12, atol=1e-18)


@pytest.mark.parametrize("act", ["relu2", "silu"])
def test_gradients_against_differences(act):
    rng = np.random.default_rng(3)
    G, U = (rng.standard_normal((4, 50)).astype(np.float32) * 3 for _ in range(2))
    dH = rng.standard_normal((4, 50)).astype(np.float32)
    f = lambda g, u: (np.maximum(g, 0) ** 2 if act == "relu2" else g / (1 + np.exp(-g))) * u  # noqa: E731
    g, u, e = G.astype(np.float64), U.astype(np.float64), 1e-5
    dG, dU = GO.hidden_backward(act, dH, G, U)
    # central differences: error e^2 / 6 times a third derivative below 10, plus 2^-53 / e
    np.testing.assert_allclose(dG, dH * (f(g + e, u) - f(g - e, u)) / (2 * e), rtol=1e-6, atol=1e-8)
    np.testing.assert_allclose(dU, dH * (f(g, u + e) - f(g, u - e)) / (2 * e), rtol=1e-6, atol=1e-8)


def test_sigmoid_far_out():
    g = np.array([-1e4, -800.0, 0.0, 800.0, 1e4])
    assert GO.sigmoid(g).tolist() == [0.0, 0.0, 0.5, 1.0, 1.0] and 0 < GO.sigmoid(-700.0) < 1e-300
