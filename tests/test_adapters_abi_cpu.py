"""The C ABI of the adapters and of dropout on the host: exports, sizes and every
refusal (all before any HIP call; nothing is launched), and the binding's own
refusals."""
import os
import re

import pytest
import torch

import bitlinear_absmean_ternarise_bit_amd as bl
from bitlinear_absmean_ternarise_bit_amd import abi
from bitlinear_absmean_ternarise_bit_amd.build import LIB_PATH, build_library

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
I63 = (1 << 63) - 1


def at(n):
    """The n-th of many distant fake addresses (256-byte aligned, never dereferenced)."""
    return (n + 1) << 44


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(LIB_PATH):
        build_library()
    return abi.load()


def caller(fn, names, args):
    def call(**kw):
        a = list(args)
        for k, v in kw.items():
            a[names.index(k)] = v
        return fn(*a)
    return call


def test_exports_every_declared_function(lib):
    text = open(os.path.join(ROOT, "include", "bitlinear_adapters.h")).read()
    names = set(re.findall(r"\b(bitlinear_\w+)\s*\(", re.sub(r"/\*.*?\*/", "", text, flags=re.S)))
    assert names == set(abi.ADAPTER_SIGNATURES) and len(names) == 7
    for n in names:
        assert hasattr(lib, n), n
    assert not names & (set(abi.SIGNATURES) | set(abi.BLOCK_SIGNATURES) | set(abi.GATED_SIGNATURES))


def test_sizes(lib):
    f, g, h = (lib.bitlinear_adapters_workspace_bytes, lib.bitlinear_adapted_workspace_bytes,
               lib.bitlinear_adapters_backward_workspace_bytes)
    for bad in (0, -1, (1 << 40) + 1, I63, -I63 - 1):
        for i in range(4):
            a = [40, 64, 64, 16]
            a[i] = bad
            assert f(*a) == g(*a) == 0
        for i in range(5):
            a = [40, 64, 64, 4, 16]
            a[i] = bad
            assert h(*a) == 0
    assert f(40, 64, 64, 257) == 0 and h(40, 64, 64, 65536, 4) == 0
    for M, K, N, R in ((1, 1, 1, 1), (16, 4096, 4096, 16), (2048, 4096, 11008, 64), (8192, 8192, 28672, 256)):
        assert f(M, K, N, R) % 256 == 0 and 4 * M * R <= f(M, K, N, R) <= 16 * 4 * M * (R + 15) + 6 * M * (R + 15) + 512
        assert h(M, K, N, 1, R) % 256 == 0 and h(M, K, N, 1, R) >= 8 * M * R
        assert g(M, K, N, R) == f(M, K, N, R) + lib.bitlinear_forward_workspace_bytes(M, K)


SHAPES = [dict(M=0), dict(M=-1), dict(K=0), dict(N=0), dict(A=0), dict(R=0), dict(A=-1), dict(R=257), dict(A=65536),
          dict(K=(1 << 20) + 1), dict(M=(1 << 31) + 1), dict(N=1 << 31, K=4), dict(M=1 << 30, N=1 << 12),
          dict(A=65535, R=256, N=1 << 17, K=1), dict(M=1 << 62, N=1 << 62, K=1 << 62)]


def test_forward_refusals(lib):
    names = ["X", "dt", "M", "K", "N", "rows", "A", "R", "down", "up", "wdt", "sc", "Y", "T", "ws", "wsb", "s"]
    need = lib.bitlinear_adapters_workspace_bytes(40, 100, 50, 8)
    call = caller(lib.bitlinear_adapters_forward, names,
                  [at(0), abi.BF16, 40, 100, 50, at(1), 3, 8, at(2), at(3), abi.BF16, at(4), at(5), at(6), at(7), need,
                   None])
    for nm in ("X", "rows", "down", "up", "sc", "Y"):
        assert call(**{nm: None}) == abi.ERR_NULL, nm
    for kw in SHAPES:
        assert call(**kw) == abi.ERR_SHAPE, kw
    for bad in (2, -1):
        assert call(dt=bad) == call(wdt=bad) == abi.ERR_DTYPE
    for nm, off in (("X", 1), ("rows", 2), ("down", 1), ("up", 1), ("sc", 2), ("Y", 2), ("T", 1)):
        assert call(**{nm: at(names.index(nm) + 20) + off}) == abi.ERR_ALIGN, nm
    assert call(wdt=abi.F32, down=at(2) + 2) == call(wdt=abi.F32, up=at(3) + 2) == abi.ERR_ALIGN
    assert call(ws=None) == call(wsb=need - 1) == abi.ERR_WORKSPACE
    assert call(ws=at(7) + 64) == abi.ERR_ALIGN
    assert call(Y=at(0)) == call(Y=at(0) + 7996) == call(T=at(5)) == call(Y=at(1)) == call(T=at(4) + 8) == abi.ERR_ARG
    assert call(Y=at(2) + 3 * 8 * 100 * 2 - 4) == call(Y=at(3) + 3 * 8 * 50 * 2 - 4) == call(T=at(7)) == abi.ERR_ARG


def test_adapted_refusals(lib):
    names = ["X", "dt", "M", "K", "pk", "N", "gm", "rows", "A", "R", "down", "up", "wdt", "sc", "Y", "T", "path", "ws",
             "wsb", "s"]
    need = lib.bitlinear_adapted_workspace_bytes(40, 100, 50, 8)
    call = caller(lib.bitlinear_adapted_forward, names,
                  [at(0), abi.F32, 40, 100, at(8), 50, at(9), at(1), 3, 8, at(2), at(3), abi.F32, at(4), at(5), None, 0,
                   at(7), need, None])
    for nm in ("X", "pk", "gm", "rows", "down", "up", "sc", "Y"):
        assert call(**{nm: None}) == abi.ERR_NULL, nm
    for kw in SHAPES:
        assert call(**kw) == abi.ERR_SHAPE, kw
    assert call(path=abi.PATH_DECODE) == abi.ERR_SHAPE
    assert call(path=7) == abi.ERR_ARG
    assert call(dt=2) == call(wdt=2) == abi.ERR_DTYPE
    for nm, off in (("X", 2), ("pk", 8), ("gm", 2), ("rows", 2), ("down", 2), ("up", 2), ("sc", 2), ("Y", 2), ("T", 1)):
        assert call(**{nm: at(names.index(nm) + 20) + off}) == abi.ERR_ALIGN, nm
    assert call(ws=None) == call(wsb=need - 1) == abi.ERR_WORKSPACE
    assert call(ws=at(7) + 16) == abi.ERR_ALIGN
    assert call(Y=at(8)) == call(Y=at(9)) == call(Y=at(0)) == call(T=at(5) + 4) == call(ws=at(5)) == abi.ERR_ARG


def test_backward_refusals(lib):
    names = ["dY", "ddt", "X", "xdt", "T", "M", "K", "N", "rows", "A", "R", "down", "up", "wdt", "sc", "dX", "acc", "dd",
             "du", "ws", "wsb", "s"]
    need = lib.bitlinear_adapters_backward_workspace_bytes(40, 100, 50, 3, 8)
    call = caller(lib.bitlinear_adapters_backward, names,
                  [at(0), abi.BF16, at(1), abi.F32, at(2), 40, 100, 50, at(3), 3, 8, at(4), at(5), abi.BF16, at(6), at(7),
                   1, at(8), at(9), at(10), need, None])
    for nm in ("dY", "X", "T", "rows", "down", "up", "sc"):
        assert call(**{nm: None}) == abi.ERR_NULL, nm
    assert call(dX=None, dd=None, du=None) == abi.ERR_NULL
    for kw in SHAPES:
        assert call(**kw) == abi.ERR_SHAPE, kw
    for nm in ("ddt", "xdt", "wdt"):
        assert call(**{nm: 2}) == call(**{nm: -1}) == abi.ERR_DTYPE
    for nm, off in (("dY", 1), ("X", 2), ("T", 2), ("rows", 1), ("down", 1), ("up", 1), ("sc", 2), ("dX", 2), ("dd", 2),
                    ("du", 1)):
        assert call(**{nm: at(names.index(nm) + 30) + off}) == abi.ERR_ALIGN, nm
    assert call(ws=None) == call(wsb=need - 1) == abi.ERR_WORKSPACE
    assert call(ws=at(10) + 32) == abi.ERR_ALIGN
    assert call(dX=at(0)) == call(dX=at(1)) == call(dd=at(4)) == call(du=at(2)) == call(dX=at(8)) == abi.ERR_ARG
    assert call(du=at(8) + 4 * (3 * 8 * 100 - 1)) == call(dd=at(10) + need - 4) == call(dX=at(6) + 8) == abi.ERR_ARG


def test_dropout_refusals(lib):
    names = ["X", "xdt", "res", "rdt", "n", "p", "seed", "off", "Y", "ydt", "s"]
    call = caller(lib.bitlinear_dropout, names, [at(0), abi.BF16, at(1), abi.F32, 100, 0.1, 1, 2, at(2), abi.BF16, None])
    assert call(X=None) == call(Y=None) == abi.ERR_NULL
    for n in (0, -1, 1 << 40, I63):
        assert call(n=n) == abi.ERR_SHAPE
    for nm in ("xdt", "rdt", "ydt"):
        assert call(**{nm: 2}) == call(**{nm: -1}) == abi.ERR_DTYPE
    assert call(X=at(0) + 1) == call(res=at(1) + 2) == call(Y=at(2) + 1) == abi.ERR_ALIGN
    for p in (-0.1, 1.0, 2.0, float("nan"), float("inf"), -1e-30):
        assert call(p=p) == abi.ERR_ARG
    assert call(Y=at(0) + 2) == call(Y=at(0) - 198) == abi.ERR_ARG      # shifted over X
    assert call(Y=at(1)) == call(Y=at(1) + 398) == abi.ERR_ARG           # over a residual of another type
    assert call(Y=at(0), ydt=abi.F32) == abi.ERR_ARG


def test_binding_refusals():
    x, i = torch.zeros(4, 64), torch.zeros(4, dtype=torch.int32)
    ad = (torch.zeros(1, 2, 64), torch.zeros(1, 2, 8), torch.zeros(1))
    for fn in (lambda: bl.adapters_forward(x, ad, i, x), lambda: bl.adapters_backward(x, x, x, ad, i),
               lambda: bl.adapted_forward(x, i, x, ad, i, path="x"), lambda: bl.adapted_forward(x, i, x, ad, i),
               lambda: bl.dropout(x, 0.1, 0)):
        with pytest.raises(ValueError):
            fn()
