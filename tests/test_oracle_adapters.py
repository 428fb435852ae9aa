"""The adapters' oracle against torch's autograd in float64 and differences, and the
generator against the published known answers."""
import numpy as np
import torch

from oracle import adapters as AO


def problem(M=9, K=13, N=11, R=3, A=4, seed=0):
    rng = np.random.default_rng(seed)
    rows = rng.integers(-1, A + 2, M)
    return (rng.standard_normal((M, K)), rows, rng.standard_normal((A, R, K)), rng.standard_normal((A, R, N)),
            rng.random(A) + 0.5, rng.standard_normal((M, N)))


def test_products_and_gradients_against_torch():
    X, rows, down, up, scales, dY = problem()
    x, dn, u = (torch.from_numpy(v).requires_grad_() for v in (X, down, up))
    out = []
    for m, a in enumerate(rows):
        out.append(scales[a] * (x[m] @ dn[a].T) @ u[a] if 0 <= a < 4 else 0 * x[m].sum() * torch.ones(11, dtype=x.dtype))
    y = torch.stack(out)
    np.testing.assert_allclose(AO.added(AO.low(X, rows, down), rows, up, scales), y.detach().numpy(), atol=1e-13)
    (y * torch.from_numpy(dY)).sum().backward()
    for got, ref in zip(AO.backward(dY, X, rows, down, up, scales), (x.grad, dn.grad, u.grad)):
        np.testing.assert_allclose(got, ref.numpy(), atol=1e-12)


def test_gradients_against_differences():
    X, rows, down, up, scales, dY = problem(seed=1)
    f = lambda X, down, up: (AO.added(AO.low(X, rows, down), rows, up, scales) * dY).sum()  # noqa: E731
    rng, e = np.random.default_rng(2), 1e-4
    for i, g in enumerate(AO.backward(dY, X, rows, down, up, scales)):
        d = rng.standard_normal(g.shape)
        hi, lo = ([v + s * e * d if j == i else v for j, v in enumerate((X, down, up))] for s in (1, -1))
        assert abs((f(*hi) - f(*lo)) / (2 * e) - (g * d).sum()) < 1e-8 * (1 + abs((g * d).sum()))


def test_philox_known_answers():
    # the known-answer vectors of the generator's authors (Random123)
    assert AO.philox(0, 0, 0) == [0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8]
    ones = (1 << 64) - 1
    assert AO.philox(ones, ones, ones) == [0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd]
    assert AO.philox(0x85a308d3243f6a88, 0x0370734413198a2e, 0x299f31d0a4093822) == [0xd16cfe09, 0x94fdcceb, 0x5001e420,
                                                                                    0x24126ea1]


def test_kept_share_and_continuity():
    k = AO.kept(0, 20000, 0.25, 5, 6)
    assert abs(k.mean() - 0.75) < 5 * np.sqrt(0.25 * 0.75 / 20000)
    assert np.array_equal(AO.kept(7, 100, 0.25, 5, 6), k[7:107])
    assert AO.kept(0, 100, 0.0, 1, 2).all() and not np.array_equal(AO.kept(0, 64, 0.5, 1, 2), AO.kept(0, 64, 0.5, 1, 3))
