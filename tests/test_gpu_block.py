"""The operators around BitLinear on the GPU against the oracle (float64).

Bit-exact: codes, scales, restored values, ReLU^2 and its backward (single
float32 operations, rounded once more for bfloat16).  Layer norm: within the
first-order bound of its float32 operations, u = 2^-24 each; a sum of K values
by at least 64 lanes makes at most K / 64 + 32 roundings on any value's way,
one of M rows at most M + 16.
"""
import ctypes

import numpy as np
import pytest
import torch

import bitlinear_absmean_ternarise_bit_amd as bl
from bitlinear_absmean_ternarise_bit_amd import abi
from bitlinear_absmean_ternarise_bit_amd.workloads import bf16_bits_to_f32, f32_to_bf16_bits, random_problem
from oracle import block as B

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
U = 2.0 ** -24


def say(*a):
    print(*a, flush=True)


def on_gpu(a, dt):
    """float32 numpy values (already of type dt) as a GPU tensor."""
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(DEV).to(DT[dt])


def values(rng, shape, dt, scale=1.0):
    x = (rng.standard_normal(shape) * scale).astype(np.float32)
    return bf16_bits_to_f32(f32_to_bf16_bits(x)) if dt == "bf16" else x


def stream_values(rng, M, K, dt):
    """A residual stream: a few channels 20 times as loud, offsets, one constant row, one zero row."""
    x = rng.standard_normal((M, K)) * np.where(rng.random(K) < 0.02, 20.0, 1.0) + rng.standard_normal(K) * 0.5
    if M > 2:
        x[M // 2] = 3.0
        x[M - 1] = 0.0
    x = x.astype(np.float32)
    return bf16_bits_to_f32(f32_to_bf16_bits(x)) if dt == "bf16" else x


def np_of(t):
    return t.float().cpu().numpy()


def same_bits(a, b):
    a, b = np.asarray(a), np.asarray(b)
    return a.shape == b.shape and np.array_equal(np.isnan(a), np.isnan(b)) and np.array_equal(
        np.where(np.isnan(a), 0, a), np.where(np.isnan(b), 0, b))


def to_type(x32, dt):
    return bf16_bits_to_f32(f32_to_bf16_bits(x32)) if dt == "bf16" else np.asarray(x32, np.float32)


def inside(got, ref, tol, what):
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} outside, first at {np.argwhere(bad)[0].tolist()}: " \
                          f"{got[bad][0]} for {ref[bad][0]}, allowed {np.broadcast_to(tol, got.shape)[bad][0]}"


def half_step(ref, dt):
    return np.abs(ref) * (2.0 ** -8 if dt == "bf16" else U)


SIZES = [(1, 1), (3, 7), (2, 64), (5, 65), (37, 300), (130, 129), (9, 1001), (4, 2048), (19, 5633), (2, 28672)]


# ---- the saved format -------------------------------------------------------

@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("M,K", SIZES)
def test_save_restore_bit_exact(M, K, dt):
    say(f"save M={M} K={K} {dt}")
    rng = np.random.default_rng(M * 31 + K)
    X = stream_values(rng, M, K, dt) * np.float32(2.0 ** int(rng.integers(-30, 30)))
    codes, scales = bl.save_activations(on_gpu(X, dt))
    rc, rs = B.save8(X)
    assert np.array_equal(codes.cpu().numpy(), rc)
    assert same_bits(scales.cpu().numpy(), rs)
    back = B.restore8(rc, rs, K)
    for out in ("f32", "bf16"):
        got = bl.restore_activations((codes, scales), K, dtype=DT[out])
        assert got.dtype == DT[out] and same_bits(np_of(got), to_type(back, out))


def test_save_special_values():
    X = np.zeros((9, 130), np.float32)
    X[1, 3] = np.nan
    X[2, 70] = np.inf
    X[3, 129] = -np.inf
    X[4, :4] = [2.0 ** -101, -2.0 ** -120, 0, 1e-45]
    X[5, :3] = [2.0 ** -100, -2.0 ** -101, 0]
    X[6, :4] = [3.4028235e38, -3.4028235e38, 1e38, 1.0]
    X[7, :7] = [127, 0.5, 1.5, 2.5, -0.5, -2.5, -126.5]   # ties
    X[8] = -0.0
    for dt in ("f32", "bf16"):
        Xd = to_type(X, dt) if dt == "f32" else np_of(on_gpu(X, "bf16").cpu())
        Xd = np.where(np.isnan(X), np.float32(np.nan), Xd).astype(np.float32)
        codes, scales = bl.save_activations(on_gpu(Xd, dt))
        rc, rs = B.save8(Xd)
        assert np.array_equal(codes.cpu().numpy(), rc) and same_bits(scales.cpu().numpy(), rs)
        back = np_of(bl.restore_activations((codes, scales), 130))
        assert np.isnan(back[1, :64]).all() and np.isfinite(back[1, 64:]).all()
        assert np.isnan(back[2, 64:128]).all() and np.isnan(back[3, 128:]).all() and np.isfinite(back[3, :128]).all()
    # a NaN or an infinity comes back out of every backward pass that reads the copy
    saved = bl.save_activations(on_gpu(X, "f32"))
    dH = np_of(bl.relu2_backward(on_gpu(np.ones_like(X), "f32"), saved))
    assert np.isnan(dH[1, :64]).all() and np.isnan(dH[2, 64:128]).all() and np.isfinite(dH[0]).all()


@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_restore_of_the_largest_values(out):
    """Groups whose scale times 128 is past the largest float32."""
    top = np.float32(3.4028235e38)
    X = np.zeros((4, 130), np.float32)
    X[0, :6] = [top, -top, top / 2, -top / 3, 1e36, -3e35]
    X[1, 64:68] = [-3.3895314e38, 1e38, 3.37e38, -3.3e38]
    X[2, 128:] = [-3.38e38, 3.38e38]
    X[3, :64] = np.float32(3.375e38)
    codes, scales = B.save8(X)
    with np.errstate(over="ignore"):
        ref = to_type(B.restore8(codes, scales, 130), out)
    saved = bl.save_activations(on_gpu(X, "f32"))
    assert np.array_equal(saved[0].cpu().numpy(), codes) and same_bits(saved[1].cpu().numpy(), scales)
    assert same_bits(np_of(bl.restore_activations(saved, 130, dtype=DT[out])), ref)


# ---- ReLU^2 -------------------------------------------------------------------

@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("M,K", SIZES)
def test_relu2_bit_exact(M, K, dt, out):
    say(f"relu2 M={M} K={K} {dt} {out}")
    rng = np.random.default_rng(M * 7 + K)
    H = values(rng, (M, K), dt)
    r = np.maximum(H, np.float32(0))
    Hd = on_gpu(H, dt)
    A, saved = bl.relu2(Hd, out_dtype=DT[out], save=True)
    assert same_bits(np_of(A), to_type(r * r, out))
    assert torch.equal(A, bl.relu2(Hd, out_dtype=DT[out]))
    rc, rs = B.save8(H)
    assert np.array_equal(saved[0].cpu().numpy(), rc) and same_bits(saved[1].cpu().numpy(), rs)
    back = B.restore8(rc, rs, K)
    rb = np.maximum(back, np.float32(0))
    assert same_bits(np_of(bl.relu2(saved, K=K, out_dtype=DT[out])), to_type(rb * rb, out))
    for ddt in ("f32", "bf16"):
        dA = values(rng, (M, K), ddt, 1e-3)
        for kept, rr in ((Hd, r), (saved, rb)):
            dH = bl.relu2_backward(on_gpu(dA, ddt), kept, out_dtype=DT[out])
            assert dH.dtype == DT[out] and same_bits(np_of(dH), to_type(dA * (np.float32(2) * rr), out))


def test_relu2_nan_stays():
    H = np.array([[np.nan, -1.0, 2.0, -np.inf, np.inf, -0.0, 0.0]], np.float32)
    A = np_of(bl.relu2(on_gpu(H, "f32")))[0]
    assert np.isnan(A[0]) and A[1:].tolist() == [0.0, 4.0, 0.0, np.inf, 0.0, 0.0]


def test_relu2_small_and_large_values():
    """Results below the normal range and above the largest value."""
    H = np.array([[1e-19, 3e-20, 1e-22, 2e19, 1.5e19, 1e-30, 4e-21, 1.7e-19, 9e-20]], np.float32)
    H = bf16_bits_to_f32(f32_to_bf16_bits(H))
    with np.errstate(over="ignore", under="ignore"):
        sq = H * H
    for dt in ("f32", "bf16"):
        for out in ("f32", "bf16"):
            with np.errstate(over="ignore"):
                ref = to_type(sq, out)
            assert same_bits(np_of(bl.relu2(on_gpu(H, dt), out_dtype=DT[out])), ref), (dt, out)


# ---- layer norm ---------------------------------------------------------------

def depth(K):
    return K / 64 + 32


def check_forward(X, w, b, eps, Y, mean, rstd, ydt):
    ry, rm, rr = B.layer_norm(X, w, b, eps)
    X = np.asarray(X, np.float64)
    K, D = X.shape[1], depth(X.shape[1])
    e = float(np.float32(eps))
    me = (D * np.abs(X).mean(axis=1) + np.abs(rm)) * U
    inside(mean, rm, me, "mean")
    d = np.abs(X - rm[:, None])
    var = (d * d).mean(axis=1)
    ve = 2 * d.mean(axis=1) * me + me * me + (D + 6) * U * var
    # ve may exceed var where a row is constant: the bound on 1 / sqrt without linearising
    lo = np.maximum(var - ve, 0) + e
    re = rr * (np.sqrt((var + e) / lo) - 1) + 4 * U * rr
    inside(rstd, rr, re, "rstd")
    aw = 1.0 if w is None else np.abs(np.asarray(w, np.float64))
    tol = aw * (d * (re + 3 * U * rr)[:, None] + (me * (rr + re))[:, None]) + 2 * U * np.abs(ry)
    inside(Y, ry, tol + half_step(np.abs(ry) + tol, ydt), "Y")


def check_backward(dY, X, mean, rstd, w, dX, dw, db, odt):
    rdx, rdw, rdb = B.layer_norm_backward(dY, X, mean, rstd, w)
    dY, X = np.asarray(dY, np.float64), np.asarray(X, np.float64)
    M, K = X.shape
    rs = np.asarray(rstd, np.float64)[:, None]
    xh = (X - np.asarray(mean, np.float64)[:, None]) * rs
    g = dY if w is None else dY * np.asarray(w, np.float64)
    D = depth(K)
    if dX is not None:
        c1, c2 = np.abs(g.mean(axis=1, keepdims=True)), np.abs((g * xh).mean(axis=1, keepdims=True))
        e1 = (D + 4) * U * np.abs(g).mean(axis=1, keepdims=True)
        e2 = (D + 8) * U * np.abs(g * xh).mean(axis=1, keepdims=True)
        axh = np.abs(xh)
        tol = np.abs(rs) * (e1 + axh * e2 + 6 * U * (np.abs(g) + axh * c2 + c1)) + 2 * U * np.abs(rdx)
        inside(dX, rdx, tol + half_step(np.abs(rdx) + tol, odt), "dX")
    for got, ref, mag, nm in ((dw, rdw, np.abs(dY * xh).sum(axis=0), "dweight"),
                              (db, rdb, np.abs(dY).sum(axis=0), "dbias")):
        if got is None:
            continue
        inside(got, ref, (M + 16) * U * mag, nm)
        # errors stay far below the worst case: a lost row would show in the median
        nz = mag > 0
        if nz.any() and M > 1:
            assert np.median(np.abs(np.asarray(got, np.float64) - ref)[nz] / mag[nz]) < 2.0 ** -20, nm


LN_SIZES = SIZES + [(1, 2048), (8, 5632), (300, 64), (1100, 520), (64, 4097), (33, 8200), (5, 16392), (3, 33000),
                    (2, 100001)]


@pytest.mark.parametrize("affine", ["both", "weight", "none"])
@pytest.mark.parametrize("dt,ydt", [("f32", "f32"), ("bf16", "bf16"), ("f32", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("M,K", LN_SIZES)
def test_layer_norm_forward(M, K, dt, ydt, affine):
    say(f"layer_norm M={M} K={K} {dt} {ydt} {affine}")
    rng = np.random.default_rng(M * 13 + K)
    X = stream_values(rng, M, K, dt)
    w = None if affine == "none" else (1 + 0.3 * rng.standard_normal(K)).astype(np.float32)
    b = (0.3 * rng.standard_normal(K)).astype(np.float32) if affine == "both" else None
    wd, bd = (None if a is None else torch.from_numpy(a).to(DEV) for a in (w, b))
    Xd = on_gpu(X, dt)
    Y, mean, rstd, saved = bl.layer_norm(Xd, wd, bd, 1e-5, out_dtype=DT[ydt], save=True)
    check_forward(X, w, b, 1e-5, np_of(Y), np_of(mean), np_of(rstd), ydt)
    rc, rsc = B.save8(X)
    assert np.array_equal(saved[0].cpu().numpy(), rc) and same_bits(saved[1].cpu().numpy(), rsc)
    assert torch.equal(bl.layer_norm(Xd, wd, bd, 1e-5, out_dtype=DT[ydt]), Y)
    Y2, m2, r2 = bl.layer_norm(Xd, wd, bd, 1e-5, out_dtype=DT[ydt], return_stats=True)
    assert torch.equal(Y2, Y) and torch.equal(m2, mean) and torch.equal(r2, rstd)
    # the norm recomputed from the copy is the norm of the restored values
    Ys, ms, rs = bl.layer_norm(saved, wd, bd, 1e-5, K=K, out_dtype=DT[ydt], return_stats=True)
    check_forward(B.restore8(rc, rsc, K), w, b, 1e-5, np_of(Ys), np_of(ms), np_of(rs), ydt)


@pytest.mark.parametrize("dt,ddt,odt", [("f32", "f32", "f32"), ("bf16", "bf16", "bf16"), ("bf16", "f32", "bf16"),
                                        ("f32", "bf16", "f32")])
@pytest.mark.parametrize("M,K", LN_SIZES)
def test_layer_norm_backward(M, K, dt, ddt, odt):
    say(f"layer_norm_backward M={M} K={K} {dt} {ddt} {odt}")
    rng = np.random.default_rng(M * 17 + K)
    X, dY = stream_values(rng, M, K, dt), values(rng, (M, K), ddt, 1e-3)
    w = (1 + 0.3 * rng.standard_normal(K)).astype(np.float32)
    wd = torch.from_numpy(w).to(DEV)
    Xd, dYd = on_gpu(X, dt), on_gpu(dY, ddt)
    _, mean, rstd, saved = bl.layer_norm(Xd, wd, None, 1e-5, save=True)
    m, r = np_of(mean), np_of(rstd)
    for kept, xk in ((Xd, X), (saved, B.restore8(saved[0].cpu().numpy(), saved[1].cpu().numpy(), K))):
        for weight, wn in ((wd, w), (None, None)):
            dX, dw, db = bl.layer_norm_backward(dYd, kept, mean, rstd, weight, out_dtype=DT[odt])
            check_backward(dY, xk, m, r, wn, np_of(dX), np_of(dw), np_of(db), odt)
        only_x = bl.layer_norm_backward(dYd, kept, mean, rstd, None, out_dtype=DT[odt], need_dw=False)
        assert torch.equal(only_x[0], dX) and only_x[1] is None and only_x[2] is None
        only_w = bl.layer_norm_backward(dYd, kept, mean, rstd, None, need_dx=False)
        assert only_w[0] is None and torch.equal(only_w[1], dw) and torch.equal(only_w[2], db)


@pytest.mark.parametrize("M,K", [(5, 7), (5, 67), (37, 1000), (9, 4096), (19, 11008), (3, 20000), (2, 33000)])
def test_layer_norm_backward_every_mix(M, K):
    """x whole in either type or saved, dY and dX in either type: twelve mixes."""
    rng = np.random.default_rng(M * 19 + K)
    w = (1 + 0.3 * rng.standard_normal(K)).astype(np.float32)
    wd = torch.from_numpy(w).to(DEV)
    for dt in ("f32", "bf16", "s8"):
        X = stream_values(rng, M, K, "f32" if dt == "s8" else dt)
        kept = on_gpu(X, "f32" if dt == "s8" else dt)
        _, mean, rstd, saved = bl.layer_norm(kept, wd, None, 1e-5, save=True)
        if dt == "s8":
            kept, X = saved, B.restore8(saved[0].cpu().numpy(), saved[1].cpu().numpy(), K)
        m, r = np_of(mean), np_of(rstd)
        for ddt in ("f32", "bf16"):
            dY = values(rng, (M, K), ddt, 1e-3)
            for odt in ("f32", "bf16"):
                say(f"layer_norm_backward M={M} K={K} {dt} {ddt} {odt}")
                dX, dw, db = bl.layer_norm_backward(on_gpu(dY, ddt), kept, mean, rstd, wd, out_dtype=DT[odt])
                assert dX.dtype == DT[odt]
                check_backward(dY, X, m, r, w, np_of(dX), np_of(dw), np_of(db), odt)


@pytest.mark.parametrize("M,K", [(4100, 264), (2500, 1024), (1500, 3000), (700, 8192)])
def test_layer_norm_many_rows(M, K):
    """More rows than the card holds at once: dweight and dbias over every one of them."""
    say(f"layer_norm rows M={M} K={K}")
    rng = np.random.default_rng(M + K)
    X, dY = stream_values(rng, M, K, "bf16"), values(rng, (M, K), "f32")
    w = (1 + 0.3 * rng.standard_normal(K)).astype(np.float32)
    wd = torch.from_numpy(w).to(DEV)
    Y, mean, rstd, saved = bl.layer_norm(on_gpu(X, "bf16"), wd, None, 1e-5, save=True)
    check_forward(X, w, None, 1e-5, np_of(Y), np_of(mean), np_of(rstd), "bf16")
    dX, dw, db = bl.layer_norm_backward(on_gpu(dY, "f32"), saved, mean, rstd, wd)
    xk = B.restore8(saved[0].cpu().numpy(), saved[1].cpu().numpy(), K)
    check_backward(dY, xk, np_of(mean), np_of(rstd), w, np_of(dX), np_of(dw), np_of(db), "f32")
    again = bl.layer_norm_backward(on_gpu(dY, "f32"), saved, mean, rstd, wd)
    assert all(torch.equal(a, b) for a, b in zip(again, (dX, dw, db)))


@pytest.mark.parametrize("xdt,ddt,odt", [("f32", "f32", "f32"), ("bf16", "bf16", "bf16"), ("s8", "f32", "bf16"),
                                         ("s8", "bf16", "f32"), ("bf16", "f32", "bf16"), ("f32", "bf16", "bf16")])
@pytest.mark.parametrize("M,K", [(256, 16392), (767, 20000), (768, 16392), (770, 28672), (1030, 16448), (900, 20004)])
def test_layer_norm_backward_many_long_rows(M, K, xdt, ddt, odt):
    say(f"layer_norm_backward long rows M={M} K={K} {xdt} {ddt} {odt}")
    g = torch.Generator(device=DEV).manual_seed(M + K)
    X = torch.randn((M, K), generator=g, device=DEV).to(DT["f32" if xdt == "s8" else xdt])
    dY = torch.randn((M, K), generator=g, device=DEV).to(DT[ddt])
    w = 1 + 0.3 * torch.randn(K, generator=g, device=DEV)
    _, mean, rstd, saved = bl.layer_norm(X, w, save=True)
    x = saved if xdt == "s8" else X
    xk = np_of(bl.restore_activations(saved, K) if xdt == "s8" else X)
    dX, dw, db = bl.layer_norm_backward(dY, x, mean, rstd, w, out_dtype=DT[odt])
    check_backward(np_of(dY), xk, np_of(mean), np_of(rstd), w.cpu().numpy(), np_of(dX), np_of(dw), np_of(db), odt)
    again = bl.layer_norm_backward(dY, x, mean, rstd, w, out_dtype=DT[odt])
    assert all(torch.equal(a, b) for a, b in zip(again, (dX, dw, db)))


def test_layer_norm_large_offset_and_eps():
    """Rows far from zero (the two-pass variance) and eps as it is given."""
    rng = np.random.default_rng(0)
    X = (rng.standard_normal((6, 777)) + np.array([0, 10, 100, 1000, -1e4, 1e-3])[:, None]).astype(np.float32)
    for eps in (0.0, 1e-12, 0.5):
        Y, mean, rstd = bl.layer_norm(on_gpu(X, "f32"), eps=eps, return_stats=True)
        check_forward(X, None, None, eps, np_of(Y), np_of(mean), np_of(rstd), "f32")


def test_layer_norm_non_finite_rows_stay_apart():
    X = np.ones((4, 300), np.float32) * np.arange(300, dtype=np.float32)
    X[1, 7], X[2, 299] = np.nan, np.inf
    Y, mean, rstd, saved = bl.layer_norm(on_gpu(X, "f32"), save=True)
    Y = np_of(Y)
    assert np.isnan(Y[1]).all() and np.isnan(Y[2]).any() and np.isfinite(Y[[0, 3]]).all()
    dX, _, _ = bl.layer_norm_backward(on_gpu(np.ones_like(X), "f32"), saved, mean, rstd)
    dX = np_of(dX)
    assert np.isnan(dX[1]).all() and np.isfinite(dX[[0, 3]]).all()


@pytest.mark.parametrize("K", [100, 104, 4100])
def test_statistics_stay_with_their_row(K):
    """Infinite statistics of the first row, with teams behind the last one: dweight has that row's
    infinities and no NaN of another team's making."""
    M = 257
    g = torch.Generator(device=DEV).manual_seed(K)
    X, dY = torch.randn((M, K), generator=g, device=DEV), torch.ones((M, K), device=DEV)
    _, mean, rstd = bl.layer_norm(X, return_stats=True)
    mean[0], rstd[0] = 100.0, float("inf")  # every difference to the mean is negative
    dX, dw, db = bl.layer_norm_backward(dY, X, mean, rstd)
    assert bool((dw == -float("inf")).all()) and bool((db == M).all()) and bool(torch.isfinite(dX[1:]).all())


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("M,K", [(3, 6), (3, 10), (3, 100), (3, 104), (3, 4100), (3, 5000), (3, 20000), (3, 20004),
                                 (3, 33000), (800, 16400), (800, 28664)])
def test_layer_norm_backward_large_constant_rows(M, K, dt):
    """mean * rstd past the largest float32, xhat = 0: dX = rstd (dY - mean of dY), here rstd dY.
    Nothing rounds: the sums over dY = +1, -1, ... are sums of small integers."""
    top, rs = 2.0 ** 118, 2.0 ** 17
    X = torch.full((M, K), top, device=DEV, dtype=DT[dt])
    dY = torch.ones((M, K), device=DEV)
    dY[:, 1::2] = -1
    mean, rstd = torch.full((M,), top, device=DEV), torch.full((M,), rs, device=DEV)
    dX, dw, db = bl.layer_norm_backward(dY, X, mean, rstd, out_dtype=torch.float32)
    assert torch.equal(dX, rs * dY) and not bool(dw.any()) and torch.equal(db, M * dY[0])


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("K", [1, 5, 64, 300, 1003, 2048, 5633, 8200, 11008, 20004, 28672, 33000])
def test_layer_norm_constant_rows(K, dt):
    """A row of one value c has mean c, x - mean = 0 and rstd = 1 / sqrt(eps), whatever K c rounds to on the
    way: Y is the bias and dweight 0, bit for bit.  rstd: the sum with eps, the root and the division round once
    each (3 u, 4 allowed)."""
    say(f"layer_norm constant rows K={K} {dt}")
    c = np.array([3.0, 8000.0, 1.1, 8000.1, -1000.3, 1e-30, -123456.7, 0.0, 2.0 ** 60], np.float32)
    X = on_gpu(np.repeat(c[:, None], K, axis=1), dt)
    g = torch.Generator(device=DEV).manual_seed(K)
    w, b = torch.randn(K, generator=g, device=DEV), torch.randn(K, generator=g, device=DEV)
    dY = torch.randn((len(c), K), generator=g, device=DEV)
    for eps in (1e-5, 1e-12):
        rs = 1 / np.sqrt(float(np.float32(eps)))
        Y, mean, rstd, saved = bl.layer_norm(X, w, b, eps, out_dtype=torch.float32, save=True)
        assert torch.equal(mean, X[:, 0].float()) and torch.equal(Y, b.expand_as(Y))
        inside(np_of(rstd), np.full(len(c), rs), 4 * U * rs, "rstd")
        assert not bool(bl.layer_norm_backward(dY, X, mean, rstd, w)[1].any())
        Ys, ms, _ = bl.layer_norm(saved, w, b, eps, K=K, return_stats=True)
        assert torch.equal(ms, bl.restore_activations(saved, K)[:, 0]) and torch.equal(Ys, b.expand_as(Ys))


@pytest.mark.parametrize("K", [300, 5633, 28672, 33000])
def test_layer_norm_rows_far_from_zero(K):
    """Rows of a large value plus 0 or a few of its float32 steps.  The stored mean is the nearest float32 but for the
    sum of the differences (K / 64 + 32 roundings of their mean size) and one rounding of its own; Y and rstd are those
    of the differences to the stored mean, each of which is exact."""
    say(f"layer_norm far rows K={K}")
    rng = np.random.default_rng(K)
    top, eps = np.array([8192.0, -1e5, 2.0 ** 20, 3.0], np.float32), 1e-12
    X = top[:, None] + np.spacing(np.abs(top))[:, None] * rng.integers(0, 5, (len(top), K)).astype(np.float32)
    Y, mean, rstd = bl.layer_norm(on_gpu(X, "f32"), None, None, eps, return_stats=True)
    X, m = X.astype(np.float64), np_of(mean).astype(np.float64)
    off = np.abs(X - X.mean(axis=1, keepdims=True)).mean(axis=1)
    # differences are at most 4 steps, to the first mean at most 4 + 2 (K / 64 + 32) / 2 of them: the sums are of
    # numbers of that size
    first = off + (depth(K) + 1) * U * np.abs(X).mean(axis=1)
    inside(m, X.mean(axis=1), depth(K) * U * first + 1.001 * U * np.abs(m), "mean")
    d = X - m[:, None]
    var = (d * d).mean(axis=1)
    wide = (d * d).mean(axis=1) + first * first  # what the sum of squares about the first mean can be
    r = 1 / np.sqrt(var + float(np.float32(eps)))
    lo = np.maximum(var - 4 * (depth(K) + 8) * U * wide, 0) + float(np.float32(eps))
    inside(np_of(rstd), r, r * (np.sqrt((var + float(np.float32(eps))) / lo) - 1) + 4 * U * r, "rstd")
    rs = np_of(rstd).astype(np.float64)[:, None]
    inside(np_of(Y), d * rs, 2 * U * np.abs(d * rs), "Y")


def test_layer_norm_gradient_by_differences():
    rng = np.random.default_rng(5)
    M, K, h = 3, 96, 2.0 ** -6
    X, dY, v = (rng.standard_normal((M, K)).astype(np.float32) for _ in range(3))
    v = np.round(v * 8) / 8  # X + h v below is what the GPU sees, rounded, and v is taken from it
    w, b = (rng.standard_normal(K).astype(np.float32) for _ in range(2))
    wd, bd = torch.from_numpy(w).to(DEV), torch.from_numpy(b).to(DEV)
    up, down = (X + h * v).astype(np.float32), (X - h * v).astype(np.float32)
    step = up.astype(np.float64) - down.astype(np.float64)
    L = [(np_of(bl.layer_norm(on_gpu(a, "f32"), wd, bd)).astype(np.float64) * dY).sum() for a in (up, down)]
    R = [(B.layer_norm(a, w, b)[0] * dY).sum() for a in (up, down)]
    _, mean, rstd = bl.layer_norm(on_gpu(X, "f32"), wd, bd, return_stats=True)
    dX, _, _ = bl.layer_norm_backward(on_gpu(dY, "f32"), on_gpu(X, "f32"), mean, rstd, wd)
    along = (np_of(dX).astype(np.float64) * step).sum()
    # every Y is within 100 u of its size (K = 96), so each sum within that of the sum of sizes
    noise = 2 * 100 * U * (np.abs(B.layer_norm(X, w, b)[0]) * np.abs(dY) + np.abs(dY)).sum()
    ref = (B.layer_norm_backward(dY, X, np_of(mean), np_of(rstd), w)[0] * step).sum()
    assert abs((L[0] - L[1]) - (R[0] - R[1])) <= noise
    assert abs((L[0] - L[1]) - along) <= 2 * noise + abs((R[0] - R[1]) - ref)
    assert abs((R[0] - R[1]) - ref) < 0.05 * abs(ref)  # the step is small enough to say something


# ---- where outputs lie -----------------------------------------------------------

def test_odd_addresses_and_guards():
    """Arrays that start on any element, with guard values on both sides of every output."""
    lib, rng = abi.load(), np.random.default_rng(2)
    stream = torch.cuda.current_stream(DEV).cuda_stream

    def guarded(n, dtype, off):
        t = torch.full((n + 64,), 77, dtype=dtype, device=DEV)
        return t, t[off:off + n]

    for M, K, off in ((5, 67, 1), (90, 1003, 3), (4, 640, 5), (2, 4096, 7), (3, 20001, 3)):
        say(f"guards M={M} K={K} off={off}")
        Kp = bl.padded_k(K)
        X = values(rng, (M, K), "bf16")
        buf, x = guarded(M * K, torch.bfloat16, off)
        x.copy_(on_gpu(X, "bf16").view(-1))
        dbuf, dy = guarded(M * K, torch.float32, off)
        dy.copy_(on_gpu(values(rng, (M, K), "f32"), "f32").view(-1))
        w = torch.rand(K + 9, device=DEV)[off:off + K]
        outs = {"Y": guarded(M * K, torch.bfloat16, off), "mean": guarded(M, torch.float32, off),
                "rstd": guarded(M, torch.float32, off), "codes": guarded(M * Kp, torch.int8, 16),
                "scales": guarded(M * Kp // 64, torch.float32, off), "dX": guarded(M * K, torch.bfloat16, off),
                "dw": guarded(K, torch.float32, off), "db": guarded(K, torch.float32, off),
                "A": guarded(M * K, torch.float32, off), "dH": guarded(M * K, torch.bfloat16, off),
                "back": guarded(M * K, torch.bfloat16, off)}
        p = {k: v[1].data_ptr() for k, v in outs.items()}
        ws_bytes = lib.bitlinear_layer_norm_backward_workspace_bytes(M, K)
        wbuf = torch.full((ws_bytes + 512,), 77, dtype=torch.uint8, device=DEV)
        wp = wbuf.data_ptr() + 256
        assert wp % 256 == 0
        assert lib.bitlinear_layer_norm(x.data_ptr(), None, 1, M, K, w.data_ptr(), None, 1e-5, p["Y"], 1, p["mean"],
                                        p["rstd"], p["codes"], p["scales"], stream) == abi.OK
        assert lib.bitlinear_layer_norm_backward(dy.data_ptr(), 0, p["codes"], p["scales"], 2, p["mean"], p["rstd"],
                                                 M, K, w.data_ptr(), p["dX"], 1, p["dw"], p["db"], wp, ws_bytes,
                                                 stream) == abi.OK
        assert lib.bitlinear_relu2(x.data_ptr(), None, 1, M, K, p["A"], 0, None, None, stream) == abi.OK
        assert lib.bitlinear_relu2_backward(dy.data_ptr(), 0, p["codes"], p["scales"], 2, M, K, p["dH"], 1,
                                            stream) == abi.OK
        assert lib.bitlinear_restore_activations(p["codes"], p["scales"], M, K, p["back"], 1, stream) == abi.OK
        torch.cuda.synchronize()
        for nm, (t, v) in outs.items():
            o = 16 if nm == "codes" else off
            assert bool((t[:o] == 77).all()) and bool((t[o + v.numel():] == 77).all()), nm
        assert bool((wbuf[:256] == 77).all()) and bool((wbuf[256 + ws_bytes:] == 77).all())
        # the same values as from aligned arrays
        Xd, wd = on_gpu(X, "bf16"), w.clone()
        Y, mean, rstd, saved = bl.layer_norm(Xd, wd, None, 1e-5, save=True)
        dX, dw, db = bl.layer_norm_backward(dy.view(M, K).clone(), saved, mean, rstd, wd, out_dtype=torch.bfloat16)
        for nm, ref in (("Y", Y), ("mean", mean), ("codes", saved[0]), ("scales", saved[1]), ("dX", dX), ("dw", dw),
                        ("db", db), ("A", bl.relu2(Xd, out_dtype=torch.float32)),
                        ("dH", bl.relu2_backward(dy.view(M, K).clone(), saved, out_dtype=torch.bfloat16)),
                        ("back", bl.restore_activations(saved, K, torch.bfloat16))):
            assert torch.equal(outs[nm][1], ref.reshape(-1)), nm


def test_offsets_past_32_bits():
    """More than 2^32 values: the last rows, which lie behind every 32-bit offset."""
    M, K = 66000, 65600
    say(f"large M={M} K={K}")
    g = torch.Generator(device=DEV).manual_seed(1)
    rows = torch.randn((40, K), generator=g, device=DEV)
    X = torch.zeros((M, K), dtype=torch.bfloat16, device=DEV)
    X[-40:] = rows.to(torch.bfloat16)
    tail = X[-40:].clone()
    Y, mean, rstd, saved = bl.layer_norm(X, save=True)
    y, m, r, s = bl.layer_norm(tail, save=True)
    assert torch.equal(Y[-40:], y) and torch.equal(mean[-40:], m) and torch.equal(rstd[-40:], r)
    assert torch.equal(saved[0][-40:], s[0]) and torch.equal(saved[1][-40:], s[1])
    assert not bool(Y[:-40].any())
    del X
    dA = Y  # zero but for the last rows
    dH = bl.relu2_backward(dA, saved)
    assert torch.equal(dH[-40:], bl.relu2_backward(dA[-40:].clone(), s)) and not bool(dH[:-40].any())
    dX, dw, db = bl.layer_norm_backward(dA, saved, mean, rstd)
    dx, _, _ = bl.layer_norm_backward(dA[-40:].clone(), s, m, r)
    assert torch.equal(dX[-40:], dx) and not bool(dX[:-40].any())
    xk = np_of(bl.restore_activations(s, K))
    check_backward(np_of(dA[-40:]), xk, np_of(m), np_of(r), None, None, np_of(dw), np_of(db), "f32")


def test_more_rows_than_one_launch_takes():
    """2^28 rows of 8 chunks are one launch of the element-wise kernels; the rows behind it are the next."""
    M = (1 << 28) + 1000
    say(f"rows M={M} K=1")
    g = torch.Generator(device=DEV).manual_seed(2)
    tail = torch.randn((2000, 1), generator=g, device=DEV).to(torch.bfloat16)
    X = torch.zeros((M, 1), dtype=torch.bfloat16, device=DEV)
    X[-2000:] = tail
    A, saved = bl.relu2(X, save=True)
    a, s = bl.relu2(tail, save=True)
    assert torch.equal(A[-2000:], a) and not bool(A[:-2000].any())
    assert torch.equal(saved[0][-2000:], s[0]) and torch.equal(saved[1][-2000:], s[1])
    assert not bool(saved[1][:-2000].any())
    back = bl.restore_activations(saved, 1, torch.bfloat16)
    assert torch.equal(back[-2000:], bl.restore_activations(s, 1, torch.bfloat16)) and not bool(back[:-2000].any())
    del A, saved, back
    # every row is one value: its norm is the bias, its mean the value, and dbias is the sum of dY
    bias = torch.full((1,), 0.5, device=DEV)
    Y, mean, rstd = bl.layer_norm(X, None, bias, return_stats=True)
    assert bool((Y == 0.5).all()) and torch.equal(mean, X.view(-1).float())
    dX, dw, db = bl.layer_norm_backward(X, X, mean, rstd)
    # dX = rstd g - rstd c1 with c1 = g: the exact product less the rounded one, at most u rstd |g|
    # (and u of that again for the second rounding), of either sign
    assert bool((dX.float().abs() <= 2 * U * rstd[0] * X.float().abs()).all()) and float(dw) == 0
    assert abs(float(db) - float(tail.double().sum())) <= 2000 * U * float(tail.double().abs().sum())


@pytest.mark.parametrize("M,K", [(3, 100), (400, 520), (90, 9000), (40, 20000), (270, 20000), (1000, 28672)])
def test_gradients_one_at_a_time(M, K):
    """dX, dweight and dbias each alone, through the C ABI, equal the call for all three."""
    lib, g = abi.load(), torch.Generator(device=DEV).manual_seed(M)
    X, dY = (torch.randn((M, K), generator=g, device=DEV) for _ in range(2))
    _, mean, rstd = bl.layer_norm(X, return_stats=True)
    ref = bl.layer_norm_backward(dY, X, mean, rstd)
    need = lib.bitlinear_layer_norm_backward_workspace_bytes(M, K)
    ws = torch.empty(max(need, 1), dtype=torch.uint8, device=DEV)
    stream = torch.cuda.current_stream(DEV).cuda_stream
    for i in range(3):
        out = torch.full_like(ref[i], float("nan"))
        p = [out.data_ptr() if i == j else None for j in range(3)]
        assert lib.bitlinear_layer_norm_backward(
            dY.data_ptr(), 0, X.data_ptr(), None, 0, mean.data_ptr(), rstd.data_ptr(), M, K, None, p[0], 0, p[1], p[2],
            ws.data_ptr() if i and need else None, need if i else 0, stream) == abi.OK
        torch.cuda.synchronize()
        assert torch.equal(out, ref[i])


# ---- streams, graphs, refusals ------------------------------------------------------

def test_other_stream():
    g = torch.Generator(device=DEV).manual_seed(4)
    X = torch.randn((500, 1200), generator=g, device=DEV)
    ref = bl.layer_norm(X, save=True)
    refb = bl.layer_norm_backward(X, ref[3], ref[1], ref[2])
    s = torch.cuda.Stream(DEV)
    s.wait_stream(torch.cuda.current_stream(DEV))
    with torch.cuda.stream(s):
        got = bl.layer_norm(X, save=True)
        gotb = bl.layer_norm_backward(X, got[3], got[1], got[2])
    s.synchronize()
    for a, b in zip((*ref[:3], *ref[3], *refb), (*got[:3], *got[3], *gotb)):
        assert torch.equal(a, b)


def test_two_streams_at_once():
    g = torch.Generator(device=DEV).manual_seed(9)
    jobs = []
    for M, K in ((3000, 1000), (700, 9000)):
        X, dY = (torch.randn((M, K), generator=g, device=DEV) for _ in range(2))
        st = bl.layer_norm(X, save=True)
        jobs.append((X, dY, st, bl.layer_norm_backward(dY, st[3], st[1], st[2]), torch.cuda.Stream(DEV)))
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(6):
        for i, (X, dY, st, ref, s) in enumerate(jobs):
            with torch.cuda.stream(s):
                y = bl.layer_norm(X, save=True)
                got[i].append((y, bl.layer_norm_backward(dY, y[3], y[1], y[2])))
    torch.cuda.synchronize()
    for i, (X, dY, st, ref, s) in enumerate(jobs):
        for y, b in got[i]:
            assert all(torch.equal(u, v) for u, v in zip((*y[:3], *y[3], *b), (*st[:3], *st[3], *ref)))


def test_graph_replays_equal_eager():
    """A captured step, replayed on new inputs, with eager calls of the same shapes in between."""
    g = torch.Generator(device=DEV).manual_seed(6)
    M, K = 900, 1500
    X, dY = (torch.randn((M, K), generator=g, device=DEV) for _ in range(2))
    w, b = (torch.randn((K,), generator=g, device=DEV) for _ in range(2))
    ws = torch.empty((abi.load().bitlinear_layer_norm_backward_workspace_bytes(M, K),), dtype=torch.uint8, device=DEV)

    def step(x, dy, workspace=None):
        y, mean, rstd, saved = bl.layer_norm(x, w, b, save=True)
        dx, dw, db = bl.layer_norm_backward(dy, saved, mean, rstd, w, workspace=workspace)
        a, hs = bl.relu2(x, save=True)
        return y, dx, dw, db, a, bl.relu2_backward(dy, hs)

    step(X, dY)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(X, dY, ws)
    other = torch.cuda.CUDAGraph()  # one more of the same calls, with a workspace of its own pool
    with torch.cuda.graph(other):
        out2 = step(X, dY)
    for seed in range(4):
        g2 = torch.Generator(device=DEV).manual_seed(100 + seed)
        X.copy_(torch.randn((M, K), generator=g2, device=DEV))
        dY.copy_(torch.randn((M, K), generator=g2, device=DEV))
        graph.replay()
        other.replay()
        torch.cuda.synchronize()
        for one, two, eager in zip(out, out2, step(X.clone(), dY.clone())):
            assert torch.equal(one, eager) and torch.equal(two, eager)
        torch.cuda.synchronize()


def test_binding_refusals():
    X = torch.zeros((4, 100), device=DEV)
    saved = bl.save_activations(X)
    bad = [
        lambda: bl.layer_norm(X.t()),
        lambda: bl.layer_norm(X.half()),
        lambda: bl.layer_norm(X[0]),
        lambda: bl.layer_norm(X[:0]),
        lambda: bl.layer_norm(X, K=99),
        lambda: bl.layer_norm(X, weight=torch.zeros(99, device=DEV)),
        lambda: bl.layer_norm(X, weight=torch.zeros(100, device=DEV, dtype=torch.bfloat16)),
        lambda: bl.layer_norm(X, bias=torch.zeros(100)),
        lambda: bl.layer_norm(X, out_dtype=torch.float16),
        lambda: bl.layer_norm(X, out=torch.empty((4, 99), device=DEV)),
        lambda: bl.layer_norm(saved, K=100, save=True),
        lambda: bl.layer_norm(saved),
        lambda: bl.layer_norm(saved, K=200),
        lambda: bl.layer_norm((saved[0], saved[1][:2]), K=100),
        lambda: bl.layer_norm_backward(X, X[:3], X[:, 0].contiguous(), X[:, 0].contiguous()),
        lambda: bl.layer_norm_backward(X, X, None, None),
        lambda: bl.layer_norm_backward(X, X, X[0], X[0]),
        lambda: bl.layer_norm_backward(X, X, X[:, 0].contiguous(), X[:, 0].contiguous(), need_dx=False, need_dw=False),
        lambda: bl.restore_activations(saved, 128, dtype=torch.int8),
        lambda: bl.restore_activations(saved, 300),
        lambda: bl.relu2(saved),
        lambda: bl.relu2(saved, K=100, save=True),
        lambda: bl.relu2_backward(X, X[:3]),
        lambda: bl.relu2_backward(X, X, out=X.bfloat16(), out_dtype=torch.float32),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            say("refusal", i)
            call()
    with pytest.raises(bl.BitLinearError):
        bl.relu2(X, out=X)
    with pytest.raises(bl.BitLinearError):
        bl.layer_norm(X, eps=-1.0)
    st = X[:, 0].contiguous()
    Z = torch.zeros((400, 100), device=DEV)
    st = Z[:, 0].contiguous()
    with pytest.raises(bl.BitLinearError):
        bl.layer_norm_backward(Z, Z.clone(), st, st.clone(), workspace=torch.empty(256, dtype=torch.uint8, device=DEV))


def test_saved_pair_refusals():
    codes, scales = saved = bl.save_activations(torch.zeros((4, 100), device=DEV))
    for pair, K in (((codes[0, 0].clone(), scales), 100), ((codes[0], scales), 100), ((codes[:0], scales[:0]), 100),
                    (saved, 0), (saved, -10), (saved, 64), ((codes.float(), scales), 100), ((codes, scales.double()), 100),
                    ((codes, scales[0]), 100), ((codes.cpu(), scales), 100), ((codes, scales.cpu()), 100),
                    ((codes,), 100), ((codes, scales, scales), 100), ((codes[:, :64], scales[:, :1]), 64)):
        for call in (bl.restore_activations, bl.relu2, lambda x, K: bl.layer_norm(x, K=K)):
            with pytest.raises(ValueError):
                call(pair, K)


# ---- together, as a block trains ------------------------------------------------------

def test_block_training_step():
    """norm -> BitLinear -> ReLU^2 -> BitLinear and back, with 8-bit copies of both activations; every
    stage against the oracle on the inputs that the GPU gave it."""
    M, D, F = 150, 320, 712
    rng = np.random.default_rng(8)
    X = stream_values(rng, M, D, "bf16")
    w, b = ((0.3 * rng.standard_normal(D) + o).astype(np.float32) for o in (1, 0))
    wd, bd = torch.from_numpy(w).to(DEV), torch.from_numpy(b).to(DEV)
    Wu = torch.from_numpy(random_problem(1, D, F, seed=1).W).to(DEV)
    Wd = torch.from_numpy(random_problem(1, F, D, seed=2).W).to(DEV)
    (pu, gu), (pd, gd) = bl.quantize_weights(Wu), bl.quantize_weights(Wd)
    (tu, mu), (td, md) = bl.pack_transposed(Wu, gu), bl.pack_transposed(Wd, gd)
    # forward
    Y, mean, rstd, sx = bl.layer_norm(on_gpu(X, "bf16"), wd, bd, save=True)
    yq = bl.quantize_activations(Y)
    H = bl.forward_quantized(*yq, pu, gu, D)
    A, sh = bl.relu2(H, save=True)
    aq = bl.quantize_activations(A)
    Z = bl.forward_quantized(*aq, pd, gd, F)
    check_forward(X, w, b, 1e-5, np_of(Y), np_of(mean), np_of(rstd), "bf16")
    h = np_of(H)
    r = np.maximum(h, np.float32(0))
    assert same_bits(np_of(A), r * r)
    # the block without saving gives the same output
    assert torch.equal(Z, bl.ffn_forward(Y, (pu, gu), (pd, gd), path="prefill"))
    # backward
    dZ = on_gpu(values(rng, (M, D), "bf16", 1e-2), "bf16")
    dA, dWd = bl.backward(dZ, td, gd, aq[0], aq[1], md, F)
    dH = bl.relu2_backward(dA, sh, out_dtype=torch.bfloat16)
    dY, dWu = bl.backward(dH, tu, gu, yq[0], yq[1], mu, D)
    dX, dw, db = bl.layer_norm_backward(dY, sx, mean, rstd, wd, out_dtype=torch.bfloat16)
    hb = B.restore8(*B.save8(h), F)
    assert same_bits(np_of(dH), to_type(np_of(dA) * (np.float32(2) * np.maximum(hb, np.float32(0))), "bf16"))
    xb = B.restore8(*B.save8(X), D)
    check_backward(np_of(dY), xb, np_of(mean), np_of(rstd), w, np_of(dX), np_of(dw), np_of(db), "bf16")
    # against the step with the activations kept whole: the copies' rounding only.  A saved value is off by
    # at most half its group's scale, amax / 254; over random values that is about amax / 440 rms.
    dHk = bl.relu2_backward(dA, H, out_dtype=torch.bfloat16)
    off = (np_of(dH) - np_of(dHk)).astype(np.float64)
    bound = np.abs(np_of(dA)) * 2 * np.repeat(np.abs(np.pad(h, ((0, 0), (0, -F % 64)))).reshape(M, -1, 64).max(2), 64,
                                             axis=1)[:, :F] / 254
    assert np.all(np.abs(off) <= bound * 1.001 + 2 * 2.0 ** -8 * np.abs(np_of(dHk)) + 2.0 ** -8 * bound)
