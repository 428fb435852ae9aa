"""Adapters on the GPU where 32-bit sizes, ranks and types meet, against float64."""
import pytest
import torch

import bitlinear_absmean_ternarise_bit_amd as bl

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
U24 = 2.0 ** -24


def test_an_adapter_of_more_bytes_than_a_resource_holds():
    # 64 ranks of 2^24 float32 are 2^32 bytes, of 2^23 2^31
    M, K, R = 256, 16, 64
    for N in (1 << 24, (1 << 23) + 4):
        print(f"N={N}", flush=True)
        g = torch.Generator(device=DEV).manual_seed(7)
        x = torch.randn(M, K, generator=g, device=DEV)
        packed, gamma = bl.quantize_weights(torch.randn(N, K, generator=g, device=DEV) * 0.02)
        ads = (torch.randn(1, R, K, generator=g, device=DEV), torch.randn(1, R, N, generator=g, device=DEV),
               torch.full((1,), 0.5, device=DEV))
        ids = (torch.arange(M, device=DEV) % 3 - 1).clamp(max=0).to(torch.int32)  # every third token: none
        y, t = bl.adapted_forward(x, packed, gamma, ads, ids, return_low=True)
        base = bl.forward(x, packed, gamma, K)
        assert torch.equal(y[ids < 0], base[ids < 0])
        for n0 in list(range(0, N, 1 << 21)) + [N - 4]:
            part = slice(n0, min(n0 + (1 << 12), N))
            up = ads[1][0][:, part].double()
            ref = base[:, part].double() + 0.5 * (t.double() @ up)  # (t is 0 without an adapter)
            terms = base[:, part].double().abs() + 0.5 * (t.double().abs() @ up.abs())
            # R terms of three planes' products each, their sum with the projection
            assert ((y[:, part].double() - ref).abs() <= terms * (R + 72) * U24).all()
        del y, t, base, ads, x, packed
        torch.cuda.empty_cache()
