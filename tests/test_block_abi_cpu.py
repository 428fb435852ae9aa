"""The C ABI of the operators around BitLinear on the host: exports, sizes and
every refusal (all before any HIP call; nothing is launched), and the Python
binding's own refusals."""
import ctypes
import os
import re

import pytest
import torch

import bitlinear_absmean_ternarise_bit_amd as bl
from bitlinear_absmean_ternarise_bit_amd import abi
from bitlinear_absmean_ternarise_bit_amd.build import LIB_PATH, build_library

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = ctypes.c_void_p
NAN, INF = float("nan"), float("inf")


def at(n):
    """The n-th of many distant fake addresses (256-byte aligned, 4 GiB apart; never dereferenced)."""
    return (n + 1) << 32


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
    text = open(os.path.join(ROOT, "include", "bitlinear_block.h")).read()
    names = set(re.findall(r"\b(bitlinear_\w+)\s*\(", re.sub(r"/\*.*?\*/", "", text, flags=re.S)))
    assert names == set(abi.BLOCK_SIGNATURES) and len(names) == 8
    for n in names:
        assert hasattr(lib, n), n
    assert not names & set(abi.SIGNATURES)


def test_sizes(lib):
    assert [lib.bitlinear_saved_groups(k) for k in (1, 64, 65, 28672)] == [1, 1, 2, 448]
    for bad in (0, -1, -(1 << 63), (1 << 40) + 1, (1 << 63) - 1):
        assert lib.bitlinear_saved_groups(bad) == 0
        assert lib.bitlinear_layer_norm_backward_workspace_bytes(bad, 64) == 0
        assert lib.bitlinear_layer_norm_backward_workspace_bytes(64, bad) == 0
    f = lib.bitlinear_layer_norm_backward_workspace_bytes
    for M, K in ((1, 1 << 20), (40, 100), (2048, 4096), (1 << 31, 64), (100, 28672), (3, 8192)):
        assert f(M, K) % 256 == 0 and 0 < f(M, K) <= 256 * 2 * 4 * K + 256
    assert f(1, 1) == f(3, 100) == f(2, 8192) == 0  # one workgroup writes the gradients


SHAPES = [(0, 8), (8, 0), (-1, 8), (8, -1), ((1 << 31) + 1, 1), (8, (1 << 20) + 1), (1 << 20, 1 << 20),
          (1 << 62, 1 << 62), (-(1 << 63), -(1 << 63))]


def shapes_refused(call):
    for M, K in SHAPES:
        assert call(M=M, K=K) == abi.ERR_SHAPE


def test_save_and_restore_refusals(lib):
    call = caller(lib.bitlinear_save_activations, ["X", "dt", "M", "K", "codes", "scales", "s"],
                  [at(0), abi.BF16, 4, 100, at(1), at(2), None])
    for nm in ("X", "codes", "scales"):
        assert call(**{nm: None}) == abi.ERR_NULL
    shapes_refused(call)
    for dt in (2, -1, 3):
        assert call(dt=dt) == abi.ERR_DTYPE
    assert call(X=at(0) + 1) == abi.ERR_ALIGN
    assert call(X=at(0) + 2, dt=abi.F32) == abi.ERR_ALIGN
    assert call(codes=at(1) + 8) == abi.ERR_ALIGN
    assert call(scales=at(2) + 2) == abi.ERR_ALIGN
    assert call(codes=at(0)) == abi.ERR_ARG                      # over X
    assert call(codes=at(0) + 16 * 49) == abi.ERR_ARG            # over X's last bytes (800)
    assert call(scales=at(1) + 4 * 128 - 4) == abi.ERR_ARG       # over the codes' end
    call = caller(lib.bitlinear_restore_activations, ["codes", "scales", "M", "K", "X", "dt", "s"],
                  [at(1), at(2), 4, 100, at(0), abi.BF16, None])
    for nm in ("X", "codes", "scales"):
        assert call(**{nm: None}) == abi.ERR_NULL
    shapes_refused(call)
    for dt in (2, -1):
        assert call(dt=dt) == abi.ERR_DTYPE
    assert call(codes=at(1) + 4) == abi.ERR_ALIGN
    assert call(scales=at(2) + 1) == abi.ERR_ALIGN
    assert call(X=at(0) + 1) == abi.ERR_ALIGN
    assert call(X=at(1) + 4 * 128 - 2) == abi.ERR_ARG


def test_layer_norm_refusals(lib):
    names = ["X", "xs", "dt", "M", "K", "w", "b", "eps", "Y", "ydt", "mean", "rstd", "saved", "ss", "s"]
    call = caller(lib.bitlinear_layer_norm, names,
                  [at(0), None, abi.BF16, 4, 100, at(1), at(2), 1e-5, at(3), abi.F32, at(4), at(5), at(6), at(7), None])
    for nm in ("X", "Y", "mean", "rstd", "saved", "ss"):
        assert call(**{nm: None}) == abi.ERR_NULL
    shapes_refused(call)
    assert call(dt=3) == abi.ERR_DTYPE and call(ydt=2) == abi.ERR_DTYPE and call(ydt=-1) == abi.ERR_DTYPE
    assert call(dt=abi.SAVED8) == abi.ERR_NULL                    # no scales
    assert call(dt=abi.SAVED8, xs=at(8)) == abi.ERR_ARG           # saved from saved
    assert call(dt=abi.SAVED8, xs=at(8), X=at(0) + 8) == abi.ERR_ALIGN
    assert call(dt=abi.SAVED8, xs=at(8) + 2) == abi.ERR_ALIGN
    for nm, off in (("X", 1), ("w", 2), ("b", 2), ("Y", 2), ("mean", 1), ("rstd", 2), ("saved", 8), ("ss", 2)):
        assert call(**{nm: at(names.index(nm) + 20) + off}) == abi.ERR_ALIGN
    for eps in (-1e-5, NAN, INF):
        assert call(eps=eps) == abi.ERR_ARG
    for nm in ("Y", "mean", "saved", "ss"):                       # an output over an input
        for other in (at(0), at(1), at(2)):
            assert call(**{nm: other}) == abi.ERR_ARG
    assert call(rstd=at(4)) == abi.ERR_ARG and call(mean=at(3) + 1596) == abi.ERR_ARG


def test_layer_norm_backward_refusals(lib):
    names = ["dY", "ddt", "X", "xs", "dt", "mean", "rstd", "M", "K", "w", "dX", "odt", "dw", "db", "ws", "wsb", "s"]
    need = lib.bitlinear_layer_norm_backward_workspace_bytes(40, 100)
    call = caller(lib.bitlinear_layer_norm_backward, names,
                  [at(0), abi.F32, at(1), None, abi.BF16, at(2), at(3), 40, 100, at(4), at(5), abi.BF16, at(6), at(7),
                   at(8), need, None])
    for nm in ("dY", "X", "mean", "rstd"):
        assert call(**{nm: None}) == abi.ERR_NULL
    assert call(dX=None, dw=None, db=None) == abi.ERR_NULL
    assert call(dt=abi.SAVED8) == abi.ERR_NULL
    shapes_refused(call)
    assert call(ddt=2) == abi.ERR_DTYPE and call(dt=5) == abi.ERR_DTYPE and call(odt=2) == abi.ERR_DTYPE
    for nm, off in (("dY", 2), ("X", 1), ("mean", 2), ("rstd", 2), ("w", 1), ("dX", 1), ("dw", 2), ("db", 2), ("ws", 16)):
        assert call(**{nm: at(names.index(nm) + 20) + off}) == abi.ERR_ALIGN
    assert call(ws=None) == abi.ERR_WORKSPACE and call(wsb=need - 1) == abi.ERR_WORKSPACE
    assert call(ws=None, wsb=0, db=None) == abi.ERR_WORKSPACE
    # a workspace that is not needed is not looked at
    assert call(M=3, ws=None, wsb=0, dw=at(0)) == abi.ERR_ARG
    for nm in ("dX", "dw", "db", "ws"):
        for other in (at(0), at(1), at(2), at(3), at(4)):
            assert call(**{nm: other}) == abi.ERR_ARG
    assert call(db=at(6)) == abi.ERR_ARG and call(dw=at(8)) == abi.ERR_ARG


def test_relu2_refusals(lib):
    names = ["H", "hs", "dt", "M", "K", "A", "adt", "saved", "ss", "s"]
    call = caller(lib.bitlinear_relu2, names, [at(0), None, abi.F32, 4, 100, at(1), abi.BF16, at(2), at(3), None])
    for nm in ("H", "A", "saved", "ss"):
        assert call(**{nm: None}) == abi.ERR_NULL
    shapes_refused(call)
    assert call(dt=3) == abi.ERR_DTYPE and call(adt=2) == abi.ERR_DTYPE
    assert call(dt=abi.SAVED8, hs=at(5)) == abi.ERR_ARG
    assert call(H=at(0) + 2) == abi.ERR_ALIGN and call(A=at(1) + 1) == abi.ERR_ALIGN
    assert call(saved=at(2) + 4) == abi.ERR_ALIGN and call(ss=at(3) + 2) == abi.ERR_ALIGN
    assert call(A=at(0)) == abi.ERR_ARG and call(saved=at(0)) == abi.ERR_ARG and call(ss=at(1)) == abi.ERR_ARG
    names = ["dA", "ddt", "H", "hs", "dt", "M", "K", "dH", "odt", "s"]
    call = caller(lib.bitlinear_relu2_backward, names,
                  [at(0), abi.F32, at(1), at(2), abi.SAVED8, 4, 100, at(3), abi.BF16, None])
    for nm in ("dA", "H", "hs", "dH"):
        assert call(**{nm: None}) == abi.ERR_NULL
    shapes_refused(call)
    assert call(ddt=2) == abi.ERR_DTYPE and call(dt=4) == abi.ERR_DTYPE and call(odt=2) == abi.ERR_DTYPE
    assert call(dA=at(0) + 2) == abi.ERR_ALIGN and call(H=at(1) + 8) == abi.ERR_ALIGN
    assert call(hs=at(2) + 2) == abi.ERR_ALIGN and call(dH=at(3) + 1) == abi.ERR_ALIGN
    for other in (at(0), at(1), at(2)):
        assert call(dH=other) == abi.ERR_ARG


@pytest.mark.skipif(torch.cuda.is_available(), reason="needs a machine without a GPU")
def test_failed_launch_is_reported(lib):
    assert lib.bitlinear_save_activations(at(0), abi.F32, 4, 100, at(1), at(2), None) == abi.ERR_HIP


def test_binding_refuses_host_tensors_and_bad_types():
    x = torch.zeros((2, 64))
    for call in (lambda: bl.layer_norm(x), lambda: bl.relu2(x), lambda: bl.save_activations(x),
                 lambda: bl.layer_norm_backward(x, x, x[:, 0], x[:, 0]), lambda: bl.relu2_backward(x, x),
                 lambda: bl.restore_activations((x.to(torch.int8), x[:, :1].contiguous()), 64)):
        with pytest.raises(ValueError, match="GPU tensor"):
            call()
    with pytest.raises(ValueError, match="K is needed"):
        bl.layer_norm((x.to(torch.int8), x))


def test_binding_launches_on_the_tensors_device():
    """A call for another device than the current one makes it current and uses that device's stream."""
    from contextlib import contextmanager
    from types import SimpleNamespace
    B = object.__new__(bl._BlockCalls)
    now, seen = [0], []

    @contextmanager
    def on_device(index):
        before, now[0] = now[0], index
        yield
        now[0] = before

    B.on_device, B.device_now, B.stream_of = on_device, lambda: now[0], lambda index: 1000 + index

    def fn(*args):
        seen.append((now[0], args))
        return abi.OK

    B.launch(fn, SimpleNamespace(index=0), 7)
    B.launch(fn, SimpleNamespace(index=3), 8)
    assert seen == [(0, (7, 1000)), (3, (8, 1003))] and now == [0]
