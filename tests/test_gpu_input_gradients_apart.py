"""A row's input gradient depends on that row of the output's gradient alone: what other
rows hold, infinities and NaN among them, does not reach it.
"""
import numpy as np
import pytest
import torch

import bitlinear_absmean_ternarise_bit_amd as bl

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


def weights(rng, N, K):
    W = torch.from_numpy((rng.standard_normal((N, K)) * 0.02).astype(np.float32)).to(DEV)
    gamma = bl.quantize_weights(W)[1]
    return bl.pack_transposed(W, gamma)[0], gamma


# F: rows that end at a boundary of 64 columns, inside one (as they lie, and through padded copies), in parts of F
@pytest.mark.parametrize("M,K,F", [(9, 70, 64), (9, 70, 72), (9, 70, 8), (300, 130, 200), (70, 65, 4104), (40, 33, 77),
                                   (1100, 4096, 1000)])
def test_rows_do_not_reach_each_other(M, K, F):
    rng = np.random.default_rng(M + K + F)
    gate, up = weights(rng, F, K), weights(rng, F, K)
    dG, dU = (torch.from_numpy(rng.standard_normal((M, F)).astype(np.float32)).to(DEV).bfloat16() for _ in range(2))
    ref = bl.gated_input_backward(dG, dU, gate, up, K)
    one = bl.backward(dG, *gate, None, None, None, K, need_dw=False)[0]
    bad = torch.arange(M, device=DEV) % 4 == 3  # a row in front of and behind each of them is not
    bad[-1] = True
    for v in (float("nan"), float("inf"), -float("inf")):
        g, u = dG.clone(), dU.clone()
        g[bad], u[bad] = v, v
        assert torch.equal(bl.gated_input_backward(g, u, gate, up, K)[~bad], ref[~bad])
        assert torch.equal(bl.gated_input_backward(g, dU, gate, up, K)[~bad], ref[~bad])
        assert torch.equal(bl.gated_input_backward(dG, u, gate, up, K)[~bad], ref[~bad])
        assert torch.equal(bl.backward(g, *gate, None, None, None, K, need_dw=False)[0][~bad], one[~bad])
