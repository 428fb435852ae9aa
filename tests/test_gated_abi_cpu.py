"""The C ABI of the gated block on the host: exports, sizes and every refusal (all
before any HIP call; nothing is launched), and the binding's own refusals."""
import os
import re

import pytest
import torch

import bitlinear_absmean_ternarise_bit_amd as bl
from bitlinear_absmean_ternarise_bit_amd import abi
from bitlinear_absmean_ternarise_bit_amd.build import LIB_PATH, build_library

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def at(n):
    """The n-th of many distant fake addresses (256-byte aligned, never dereferenced)."""
    return (n + 1) << 40


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
    text = open(os.path.join(ROOT, "include", "bitlinear_gated.h")).read()
    names = set(re.findall(r"\b(bitlinear_\w+)\s*\(", re.sub(r"/\*.*?\*/", "", text, flags=re.S)))
    assert names == set(abi.GATED_SIGNATURES) and len(names) == 7
    for n in names:
        assert hasattr(lib, n), n
    assert not names & (set(abi.SIGNATURES) | set(abi.BLOCK_SIGNATURES))


def test_sizes(lib):
    f, g = lib.bitlinear_gated_ffn_workspace_bytes, lib.bitlinear_gated_input_backward_workspace_bytes
    for bad in (0, -1, (1 << 40) + 1, (1 << 63) - 1, -(1 << 63)):
        assert f(bad, 8, 8, 8) == f(8, bad, 8, 8) == f(8, 8, bad, 8) == f(8, 8, 8, bad) == \
            g(bad, 8, 8, 1) == g(8, bad, 8, 1) == g(8, 8, bad, 1) == g(8, 8, bad, 0) == 0
    assert f(8, 2048, 5632, 2048) == 8 * 5632 * 4 + lib.bitlinear_forward_workspace_bytes(8, 5632)
    assert f(8, 8192, 64, 8192) == 8 * 64 * 4 + lib.bitlinear_forward_workspace_bytes(8, 8192)
    assert g(3, 65, 8, 1) == 2 * 768 and g(3, 65, 8, 0) == 0
    assert g(55, 10688, 238, 0) == 34 * 55 * 238 * 4 + 240  # 34 parts; to a multiple of 256
    assert g(2048, 11008, 4096, 0) == 0 and f(1 << 40, 1 << 40, 1 << 40, 1 << 40) == 0
    # the down product in 15 parts of INT32 sums
    assert f(64, 64, 11008, 128) == 64 * 11008 * 4 + lib.bitlinear_forward_workspace_bytes(64, 11008) + 15 * 64 * 128 * 4


FORWARD = ["X", "dt", "M", "D", "F", "pg", "gg", "pu", "gu", "act", "H", "hdt", "G", "U", "sdt", "path", "ws", "wsb", "s"]


def forward(lib):
    return caller(lib.bitlinear_gated_forward, FORWARD,
                  [at(0), abi.BF16, 40, 100, 50, at(1), at(2), at(3), at(4), abi.ACT_RELU2, at(5), abi.F32, at(6), at(7),
                   abi.F32, abi.PATH_AUTO, at(8), 1 << 20, None])


QUANTIZED = ["Xq", "ga", "rs", "M", "D", "F", "pg", "gg", "pu", "gu", "act", "H", "hdt", "G", "U", "sdt", "s"]


def quantized(lib):
    return caller(lib.bitlinear_gated_forward_quantized, QUANTIZED,
                  [at(0), at(9), at(10), 40, 100, 50, at(1), at(2), at(3), at(4), abi.ACT_SILU, at(5), abi.BF16, at(6),
                   at(7), abi.BF16, None])


BAD_SHAPES = [(0, 8, 8), (8, 0, 8), (8, 8, 0), (-1, 8, 8), (8, (1 << 20) + 1, 8), ((1 << 31) + 1, 1, 1),
              (1, 1 << 16, 1 << 16), (1 << 30, 8, 1 << 12), (1 << 62, 1 << 62, 1 << 62)]


@pytest.mark.parametrize("make", [forward, quantized])
def test_forward_refusals(lib, make):
    call = make(lib)
    q = make is quantized
    names = QUANTIZED if q else FORWARD
    for nm in (["Xq", "ga", "rs"] if q else ["X"]) + ["pg", "gg", "pu", "gu", "H", "G", "U"]:
        assert call(**{nm: None}) == abi.ERR_NULL, nm
    for M, D, F in BAD_SHAPES:
        assert call(M=M, D=D, F=F) == abi.ERR_SHAPE
    for bad in (2, -1):
        assert call(hdt=bad) == call(sdt=bad) == abi.ERR_DTYPE
        assert call(act=bad) == abi.ERR_ARG
    for nm, off in (("pg", 8), ("pu", 4), ("gg", 2), ("gu", 1), ("H", 1), ("G", 1), ("U", 1)):
        assert call(**{nm: at(names.index(nm) + 20) + off}) == abi.ERR_ALIGN, nm
    first = at(0)
    assert call(H=first) == call(G=first + 16) == call(U=at(6)) == call(G=at(5) + 16) == abi.ERR_ARG
    assert call(H=at(1)) == call(H=at(4) - 4) == abi.ERR_ARG
    assert call(G=at(3) + 50 * 32 - 16) == abi.ERR_ARG                  # the packed matrix' last bytes
    if q:
        assert call(Xq=at(0) + 8) == call(ga=at(9) + 2) == call(rs=at(10) + 1) == abi.ERR_ALIGN
        assert call(H=at(9) + 4 * 40 - 4) == call(H=at(10) + 4 * 39) == call(H=at(0) + 40 * 128 - 4) == abi.ERR_ARG
        return
    assert call(dt=2) == call(dt=-1) == abi.ERR_DTYPE
    assert call(X=at(0) + 1) == call(X=at(0) + 2, dt=abi.F32) == abi.ERR_ALIGN
    assert call(path=3) == call(path=-1) == abi.ERR_ARG
    assert call(path=abi.PATH_DECODE) == abi.ERR_SHAPE                  # 40 tokens
    need = lib.bitlinear_forward_workspace_bytes(40, 100, 50, 1)
    assert call(ws=None) == call(wsb=need - 1) == abi.ERR_WORKSPACE
    assert call(ws=at(8) + 128) == abi.ERR_ALIGN
    assert call(ws=at(5) + 256, wsb=need) == call(ws=at(0) - 256, wsb=need) == abi.ERR_ARG


def test_block_refusals(lib):
    names = ["X", "dt", "M", "D", "F", "Do", "pg", "gg", "pu", "gu", "act", "pd", "gd", "Y", "hid", "path", "ws", "wsb", "s"]
    need = lib.bitlinear_gated_ffn_workspace_bytes(40, 100, 50, 30)
    call = caller(lib.bitlinear_gated_ffn_forward, names,
                  [at(0), abi.F32, 40, 100, 50, 30, at(1), at(2), at(3), at(4), 0, at(5), at(6), at(7), None, 0, at(8),
                   need, None])
    for nm in ("X", "pg", "gg", "pu", "gu", "pd", "gd", "Y"):
        assert call(**{nm: None}) == abi.ERR_NULL, nm
    for M, D, F in BAD_SHAPES:
        assert call(M=M, D=D, F=F) == abi.ERR_SHAPE
    assert call(Do=0) == call(Do=1 << 31) == abi.ERR_SHAPE
    assert call(dt=2) == abi.ERR_DTYPE
    assert call(act=2) == call(path=5) == abi.ERR_ARG
    assert call(path=abi.PATH_DECODE) == abi.ERR_SHAPE
    for nm, off in (("pg", 8), ("pu", 8), ("pd", 8), ("gg", 2), ("gu", 2), ("gd", 2), ("Y", 2), ("hid", 8), ("X", 2)):
        assert call(**{nm: at(names.index(nm) + 20) + off}) == abi.ERR_ALIGN, nm
    assert call(ws=None) == call(wsb=need - 1) == abi.ERR_WORKSPACE
    assert call(M=4, ws=None) == abi.ERR_WORKSPACE                       # the decode path keeps codes there too
    assert call(ws=at(8) + 16) == abi.ERR_ALIGN
    assert call(Y=at(0)) == call(Y=at(8)) == call(hid=at(7)) == call(hid=at(5)) == call(Y=at(6)) == abi.ERR_ARG


def test_backward_refusals(lib):
    names = ["dH", "dt", "G", "U", "gdt", "M", "F", "act", "dG", "dU", "odt", "s"]
    call = caller(lib.bitlinear_gated_backward, names,
                  [at(0), abi.F32, at(1), at(2), abi.BF16, 5, 100, 0, at(3), at(4), abi.BF16, None])
    for nm in ("dH", "G", "U", "dG", "dU"):
        assert call(**{nm: None}) == abi.ERR_NULL
        assert call(**{nm: at(names.index(nm) + 20) + 1}) == abi.ERR_ALIGN
    for M, F in ((0, 8), (8, 0), (8, (1 << 20) + 1), (1 << 20, 1 << 20), ((1 << 31) + 1, 1)):
        assert call(M=M, F=F) == abi.ERR_SHAPE
    for nm in ("dt", "gdt", "odt"):
        assert call(**{nm: 2}) == call(**{nm: -1}) == abi.ERR_DTYPE
    assert call(act=2) == abi.ERR_ARG
    assert call(dG=at(1)) == call(dU=at(0) + 1996) == call(dG=at(4) + 998) == call(dU=at(2)) == abi.ERR_ARG
    names = ["dG", "dU", "M", "F", "D", "pg", "gg", "pu", "gu", "dX", "ws", "wsb", "s"]
    need = lib.bitlinear_gated_input_backward_workspace_bytes(40, 100, 50, 1)
    call = caller(lib.bitlinear_gated_input_backward, names,
                  [at(0), at(1), 40, 100, 50, at(2), at(3), at(4), at(5), at(6), at(7), need, None])
    for nm in ("dG", "dU", "pg", "gg", "pu", "gu", "dX"):
        assert call(**{nm: None}) == abi.ERR_NULL
        assert call(**{nm: at(names.index(nm) + 20) + 1}) == abi.ERR_ALIGN
    for M, D, F in BAD_SHAPES:
        assert call(M=M, D=D, F=F) == abi.ERR_SHAPE
    assert call(M=1 << 20, F=1024) == abi.ERR_SHAPE                      # 32-bit offsets
    assert call(ws=None) == call(wsb=need - 1) == abi.ERR_WORKSPACE      # F % 8 != 0
    assert call(F=104, dU=at(1) + 8, ws=None) == abi.ERR_WORKSPACE       # rows that start off 16 bytes
    assert call(ws=at(7) + 64) == abi.ERR_ALIGN
    parts = lib.bitlinear_gated_input_backward_workspace_bytes(40, 1024, 50, 0)
    assert parts > 0 and call(F=1024, wsb=parts - 1) == call(F=1024, ws=None) == abi.ERR_WORKSPACE
    assert call(dX=at(0)) == call(dX=at(2)) == call(ws=at(6)) == call(dX=at(1) - 4) == abi.ERR_ARG


def test_binding_refusals():
    x = torch.zeros(4, 64)
    w = (torch.zeros(8, 4, dtype=torch.int32), torch.zeros(1))
    for fn in (lambda: bl.gated_forward(x, w, w), lambda: bl.gated_ffn_forward(x, w, w, w),
               lambda: bl.gated_backward(x, x, x), lambda: bl.gated_input_backward(x, x, w, w, 64),
               lambda: bl.gated_forward(x, w, w, act="gelu"), lambda: bl.gated_forward(x, w, w, path="fast"),
               lambda: bl.gated_forward((x, x, x), w, w), lambda: bl.gated_backward(x, x, x, act=None)):
        with pytest.raises(ValueError):
            fn()
