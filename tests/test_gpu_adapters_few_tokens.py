"""A projection and its adapters for few tokens, at every kind of rank and type, against
the oracle: up to 16 tokens in two launches, and 17 to 255 with the second product as a
pass of its own.
"""
import numpy as np
import pytest
import torch

import bitlinear_absmean_ternarise_bit_amd as bl
from test_gpu_adapters import DEV, TYPES, Problem, np_of, on_gpu

pytestmark = pytest.mark.gpu

RANKS = [1, 5, 16, 17, 33, 64, 256]


def projection(P, K, N):
    return bl.quantize_weights(on_gpu(P.rng.standard_normal((N, K)) * 0.02))


def check_kept_apart(P, packed, gamma, y, t):
    """Infinities and NaN of one adapter's tokens, of its weights and of its scale stay with them."""
    bad = torch.from_numpy(P.rows == 1).to(DEV)
    for v in (float("nan"), float("inf"), -float("inf")):
        x = P.x.clone()
        down, up, scales = (w.clone() for w in P.ads)
        x[bad], down[1], up[1], scales[1] = v, v, v, v
        y2, t2 = bl.adapted_forward(x, packed, gamma, (down, up, scales), P.ids, return_low=True)
        assert torch.equal(y2[~bad], y[~bad]) and torch.equal(t2[~bad], t[~bad])
        assert not torch.isfinite(y2[bad]).any() and not torch.isfinite(t2[bad]).any()


@pytest.mark.parametrize("xt,wt", TYPES)
@pytest.mark.parametrize("R", RANKS)
@pytest.mark.parametrize("M,K,N", [(1, 2048, 130), (5, 100, 33), (16, 250, 1003), (16, 8, 17), (2, 4099, 70)])
def test_up_to_16_tokens(M, K, N, R, xt, wt):
    print(f"few tokens M={M} K={K} N={N} R={R} {xt} {wt}", flush=True)
    for order in ("mixed", "one"):
        P = Problem(M, K, N, R, 3, xt, wt, order)
        packed, gamma = projection(P, K, N)
        base = bl.forward(P.x, packed, gamma, K)
        y, t = bl.adapted_forward(P.x, packed, gamma, P.ads, P.ids, return_low=True)
        P.check_forward(y, t, np_of(base))
        assert torch.equal(bl.adapted_forward(P.x, packed, gamma, P.ads, P.ids), y)
        check_kept_apart(P, packed, gamma, y, t)


@pytest.mark.parametrize("xt,wt", TYPES)
@pytest.mark.parametrize("M,K,N,R", [(16, 12000, 64, 40), (11, 12000, 50, 256), (16, 16400, 33, 17), (6, 11008, 100, 1)])
def test_rows_in_pieces(M, K, N, R, xt, wt):
    P = Problem(M, K, N, R, 4, xt, wt)
    packed, gamma = projection(P, K, N)
    base = bl.forward(P.x, packed, gamma, K)
    y, t = bl.adapted_forward(P.x, packed, gamma, P.ads, P.ids, return_low=True)
    P.check_forward(y, t, np_of(base))
    check_kept_apart(P, packed, gamma, y, t)


@pytest.mark.parametrize("xt,wt", TYPES)
@pytest.mark.parametrize("M,K,N,R", [(17, 300, 70, 17), (64, 4090, 130, 33), (100, 72, 300, 64), (255, 130, 257, 40),
                                     (33, 4100, 45, 256), (255, 9, 1000, 100)])
def test_17_to_255_tokens(M, K, N, R, xt, wt):
    for order in ("mixed", "requests"):
        P = Problem(M, K, N, R, 5, xt, wt, order)
        packed, gamma = projection(P, K, N)
        base = bl.forward(P.x, packed, gamma, K)
        y, t = bl.adapted_forward(P.x, packed, gamma, P.ads, P.ids, return_low=True)
        P.check_forward(y, t, np_of(base))
        check_kept_apart(P, packed, gamma, y, t)


@pytest.mark.parametrize("M,R,wt", [(1, 33, "f32"), (16, 64, "f32"), (16, 256, "bf16")])
def test_in_a_graph(M, R, wt):
    K, N = 500, 300
    P = Problem(M, K, N, R, 4, "f32", wt)
    packed, gamma = projection(P, K, N)
    call = lambda x, ids: bl.adapted_forward(x, packed, gamma, P.ads, ids, return_low=True)  # noqa: E731
    x, ids = P.x.clone(), P.ids.clone()
    call(x, ids)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(x, ids)
    for k in range(4):
        new, nid = torch.roll(P.x, (k, 7 * k), (0, 1)), (P.ids + k) % 5  # (4: none)
        x.copy_(new)
        ids.copy_(nid)
        graph.replay()
        eager = call(new, nid)
        torch.cuda.synchronize()
        assert torch.equal(out[0], eager[0]) and torch.equal(out[1], eager[1])


def test_every_token_an_adapter_of_its_own_among_many():
    M, K, N, R, A = 16, 64, 48, 3, 65535
    g = torch.Generator(device=DEV).manual_seed(2)
    x = torch.randn(M, K, generator=g, device=DEV)
    ads = (torch.randn(A, R, K, generator=g, device=DEV), torch.randn(A, R, N, generator=g, device=DEV),
           torch.rand(A, generator=g, device=DEV) + 0.5)
    ids = torch.tensor([0, A - 1, A, -1, 40000, 1, 2, 65000, 32768, 32767, 5, 5, 6, 7, 8, 9], dtype=torch.int32, device=DEV)
    packed, gamma = bl.quantize_weights(torch.randn(N, K, generator=g, device=DEV) * 0.02)
    base = bl.forward(x, packed, gamma, K)
    y = bl.adapted_forward(x, packed, gamma, ads, ids)
    for m, a in enumerate(ids.tolist()):
        if not 0 <= a < A:
            assert torch.equal(y[m], base[m])
            continue
        T, up, s = ads[0][a].double() @ x[m].double(), ads[1][a].double(), float(ads[2][a])
        aT = ads[0][a].double().abs() @ x[m].double().abs()
        terms = base[m].double().abs() + s * (aT @ up.abs())
        # as in the oracle's check: K + R additions and 144 for parts, planes and roundings
        assert ((y[m].double() - (base[m].double() + s * (T @ up))).abs() <= terms * (K + R + 144) * 2.0 ** -24).all()
        assert np.isfinite(np_of(y[m])).all()
