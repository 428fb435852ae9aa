"""Low-rank adapters and dropout on the GPU against the oracle (float64).

A product's bound: a term passes at most C + 64 float32 additions (C terms; parts
and waves add a few), its operands' planes leave out at most 2^-23 of it (three
products below 2^-24, each half of that on average and at most 2^-24.4 together
by their sizes 2^-8 2^-16), and the scale and the output round twice more: an
error of at most (C + 72) u times the sum of the terms' magnitudes, u = 2^-24.
Dropout is bit-exact.
"""
import numpy as np
import pytest
import torch

import bitlinear_absmean_ternarise_bit_amd as bl
import oracle as O
from bitlinear_absmean_ternarise_bit_amd.workloads import bf16_bits_to_f32, f32_to_bf16_bits
from oracle import adapters as AO

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
U24 = 2.0 ** -24
TYPES = [("f32", "f32"), ("f32", "bf16"), ("bf16", "f32"), ("bf16", "bf16")]


def to_type(x, dt):
    x = np.asarray(x, np.float32)
    return bf16_bits_to_f32(f32_to_bf16_bits(x)) if dt == "bf16" else x


def on_gpu(a, dt="f32"):
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(DEV).to(DT[dt])


def np_of(t):
    return t.float().cpu().numpy()


class Problem:
    def __init__(self, M, K, N, R, A, xt="bf16", wt="bf16", order="mixed", seed=0):
        rng = np.random.default_rng(seed + M + 3 * K + 5 * N + 7 * R + 11 * A)
        self.A, self.R, self.rng = A, R, rng
        self.X, self.dY = to_type(rng.standard_normal((M, K)), xt), to_type(rng.standard_normal((M, N)), xt)
        self.down = to_type(rng.standard_normal((A, R, K)) / np.sqrt(K), wt)
        self.up = to_type(rng.standard_normal((A, R, N)), wt)
        self.scales = (rng.random(A) + 0.5).astype(np.float32)
        # some tokens have no adapter: -1, A, and the ends of the range
        ids = np.concatenate([np.arange(A), [-1, A, 2 ** 31 - 1, -2 ** 31]])
        if order == "mixed":
            self.rows = rng.choice(ids, M).astype(np.int32)
        elif order == "requests":
            self.rows = np.sort(rng.choice(ids, M)).astype(np.int32)
        else:
            self.rows = np.full(M, {"one": A - 1, "none": -1}[order], np.int32)
        self.x, self.dy = on_gpu(self.X, xt), on_gpu(self.dY, xt)
        self.ads = (on_gpu(self.down, wt), on_gpu(self.up, wt), on_gpu(self.scales))
        self.ids = torch.from_numpy(self.rows).to(DEV)
        self.has = (self.rows >= 0) & (self.rows < A)

    def check_forward(self, y, t, y0):
        K, R = self.X.shape[1], self.R
        T = AO.low(self.X, self.rows, self.down)
        aT = AO.low(np.abs(self.X), self.rows, np.abs(self.down))
        assert (np.abs(np_of(t) - T) <= aT * (K + 72) * U24).all()
        ref = y0 + AO.added(T, self.rows, self.up, self.scales)
        terms = np.abs(y0) + AO.added(aT, self.rows, np.abs(self.up), self.scales)
        assert (np.abs(np_of(y) - ref) <= terms * (K + R + 144) * U24).all()
        assert np.array_equal(np_of(y)[~self.has], y0[~self.has]) and not np_of(t)[~self.has].any()

    def check_backward(self, dx, dd, du, dx0):
        (M, K), N, R = self.X.shape, self.dY.shape[1], self.R
        ref = AO.backward(self.dY, self.X, self.rows, self.down, self.up, self.scales)
        terms = AO.backward(*(np.abs(v) for v in (self.dY, self.X)), self.rows, np.abs(self.down), np.abs(self.up),
                            self.scales)
        assert (np.abs(np_of(dx) - (dx0 + ref[0])) <= (np.abs(dx0) + terms[0]) * (N + R + 144) * U24).all()
        assert (np.abs(np_of(dd) - ref[1]) <= terms[1] * (N + M + 144) * U24).all()
        assert (np.abs(np_of(du) - ref[2]) <= terms[2] * (K + M + 144) * U24).all()
        assert np.array_equal(np_of(dx)[~self.has], dx0[~self.has])
        for a in range(self.A):
            if not (self.rows == a).any():
                assert not np_of(dd)[a].any() and not np_of(du)[a].any()


CASES = [(1, 1, 1, 1, 1, "mixed"), (1, 2048, 130, 16, 4, "one"), (3, 7, 9, 3, 2, "mixed"), (16, 64, 128, 16, 20, "mixed"),
         (17, 300, 1003, 8, 3, "mixed"), (16, 1003, 520, 33, 1, "one"), (40, 33, 8, 17, 5, "requests"),
         (130, 256, 300, 64, 7, "requests"), (300, 129, 257, 5, 2, "mixed"), (600, 40, 64, 80, 3, "requests"),
         (20, 15, 17, 256, 2, "mixed"), (5, 64, 64, 16, 3, "none"), (2500, 24, 31, 16, 1, "one"), (33, 9, 2000, 1, 9, "mixed")]


@pytest.mark.parametrize("xt,wt", TYPES)
@pytest.mark.parametrize("M,K,N,R,A,order", CASES)
def test_forward_and_backward(M, K, N, R, A, order, xt, wt):
    print(f"adapters M={M} K={K} N={N} R={R} A={A} {order} {xt} {wt}", flush=True)
    P = Problem(M, K, N, R, A, xt, wt, order)
    y0 = P.rng.standard_normal((M, N)).astype(np.float32)
    y = on_gpu(y0)
    out, t = bl.adapters_forward(P.x, P.ads, P.ids, y, return_low=True)
    assert out is y
    P.check_forward(y, t, y0)
    assert torch.equal(bl.adapters_forward(P.x, P.ads, P.ids, on_gpu(y0)), y)          # without T: the same bits
    dx0 = P.rng.standard_normal((M, K)).astype(np.float32)
    dx = on_gpu(dx0)
    got, dd, du = bl.adapters_backward(P.dy, P.x, t, P.ads, P.ids, dX=dx)
    assert got is dx
    P.check_backward(dx, dd, du, dx0)
    dx, dd2, du2 = bl.adapters_backward(P.dy, P.x, t, P.ads, P.ids)                    # written, not added
    P.check_backward(dx, dd2, du2, np.zeros_like(dx0))
    none, dd3, du3 = bl.adapters_backward(P.dy, P.x, t, P.ads, P.ids, need_dx=False)
    assert none is None
    for d, u in ((dd2, du2), (dd3, du3)):
        assert torch.equal(d, dd) and torch.equal(u, du)
    only, n1, n2 = bl.adapters_backward(P.dy, P.x, None, P.ads, P.ids, need_dw=False)
    assert n1 is None and n2 is None and torch.equal(only, dx)


@pytest.mark.parametrize("xt,wt", TYPES)
def test_nothing_is_rounded_to_fewer_bits(xt, wt):
    # one value of each row: T is that value times a weight, one rounding at most
    M, K, R = 40, 96, 16
    P = Problem(M, K, 32, R, 2, xt, wt, "one")
    x = np.zeros((M, K), np.float32)
    at = P.rng.integers(0, K, M)
    x[np.arange(M), at] = 1.0
    y = torch.zeros(M, 32, device=DEV)
    _, t = bl.adapters_forward(on_gpu(x, xt), P.ads, P.ids, y, return_low=True)
    assert np.array_equal(np_of(t), P.down[1][:, at].T)                                # the weights' own bits
    x[np.arange(M), at] = P.X[np.arange(M), at]
    _, t = bl.adapters_forward(on_gpu(x, xt), P.ads, P.ids, y, return_low=True)
    ref = (P.X[np.arange(M), at].astype(np.float64)[:, None] * P.down[1][:, at].T)
    # the planes' products are added in float32: at most six roundings of what is left of the value
    assert (np.abs(np_of(t) - ref) <= np.abs(ref) * 8 * U24).all()


@pytest.mark.parametrize("M,K,N", [(1, 256, 192), (16, 300, 70), (40, 128, 300), (300, 512, 256), (1, 2050, 33),
                                   (40, 4090, 300), (150, 3001, 130), (16, 4096, 130), (11, 12000, 64), (16, 16400, 50), (16, 40, 20000), (5, 7, 40)])
def test_beside_the_projection(M, K, N):
    P = Problem(M, K, N, 16, 5, "bf16", "bf16", "requests")
    packed, gamma = bl.quantize_weights(on_gpu(P.rng.standard_normal((N, K)) * 0.02))
    for path in ["auto", "prefill"] + (["decode"] if bl.decode_fits(M, K, N) else []):
        base = bl.forward(P.x, packed, gamma, K, path=path)
        y, t = bl.adapted_forward(P.x, packed, gamma, P.ads, P.ids, path=path, return_low=True)
        two, t2 = bl.adapters_forward(P.x, P.ads, P.ids, base.clone(), return_low=True)
        assert torch.equal(t, t2)
        P.check_forward(two, t2, np_of(base))
        P.check_forward(y, t, np_of(base))
        assert torch.equal(bl.adapted_forward(P.x, packed, gamma, P.ads, P.ids, path=path), y)


@pytest.mark.parametrize("xt,wt", TYPES)
@pytest.mark.parametrize("M,K,N,R,A,order", [(129, 72, 300, 16, 3, "mixed"), (200, 2050, 8, 5, 20, "requests"),
                                             (257, 72, 300, 16, 3, "mixed"), (300, 250, 8, 5, 20, "requests"),
                                             (1500, 72, 2900, 17, 4, "requests"), (1447, 9, 2905, 64, 3, "mixed"),
                                             (2300, 130, 4500, 40, 5, "requests"), (1447, 40, 2905, 65, 3, "requests"),
                                             (2048, 40, 2048, 33, 3, "requests"), (2048, 24, 9000, 16, 3, "requests"),
                                             (2048, 24, 9000, 20, 2, "requests")])
def test_in_the_projections_epilogue(M, K, N, R, A, order, xt, wt):
    P = Problem(M, K, N, R, A, xt, wt, order)
    packed, gamma = bl.quantize_weights(on_gpu(P.rng.standard_normal((N, K)) * 0.02))
    base = bl.forward(P.x, packed, gamma, K)
    y, t = bl.adapted_forward(P.x, packed, gamma, P.ads, P.ids, return_low=True)
    P.check_forward(y, t, np_of(base))
    # a request's infinities and NaN stay with it
    bad = torch.from_numpy(P.rows == 1).to(DEV)
    for v in (float("nan"), float("inf")):
        x = P.x.clone()
        down, up, scales = (w.clone() for w in P.ads)
        x[bad], down[1], up[1], scales[1] = v, v, v, v
        y2, t2 = bl.adapted_forward(x, packed, gamma, (down, up, scales), P.ids, return_low=True)
        assert torch.equal(y2[~bad], y[~bad]) and torch.equal(t2[~bad], t[~bad]) and not torch.isfinite(y2[bad]).any()


@pytest.mark.parametrize("xt,wt", TYPES)
def test_requests_do_not_reach_each_other(xt, wt):
    M, K, N, R, A = 50, 70, 90, 12, 6
    P = Problem(M, K, N, R, A, xt, wt)
    y0 = on_gpu(P.rng.standard_normal((M, N)))
    ref, rt = bl.adapters_forward(P.x, P.ads, P.ids, y0.clone(), return_low=True)
    rdx, rdd, rdu = bl.adapters_backward(P.dy, P.x, rt, P.ads, P.ids)
    bad = torch.from_numpy(P.rows == 2).to(DEV)
    good = ~bad
    for v in (float("nan"), float("inf"), -float("inf")):
        x, dy, t = P.x.clone(), P.dy.clone(), rt.clone()
        x[bad], dy[bad], t[bad] = v, v, v
        down, up, scales = (w.clone() for w in P.ads)
        down[2], up[2], scales[2] = v, v, v
        ads = (down, up, scales)
        y, tt = bl.adapters_forward(x, ads, P.ids, y0.clone(), return_low=True)
        assert torch.equal(y[good], ref[good]) and torch.equal(tt[good], rt[good]) and not torch.isfinite(y[bad]).any()
        dx, dd, du = bl.adapters_backward(dy, x, t, ads, P.ids)
        assert torch.equal(dx[good], rdx[good]) and not torch.isfinite(dx[bad]).any()
        keep = [a for a in range(A) if a != 2]
        assert torch.equal(dd[keep], rdd[keep]) and torch.equal(du[keep], rdu[keep])
        assert not torch.isfinite(dd[2]).any() and not torch.isfinite(du[2]).any()


def test_workspace_contents_do_not_matter():
    P = Problem(300, 200, 300, 20, 4)
    need = bl.abi.load().bitlinear_adapters_backward_workspace_bytes(300, 200, 300, 4, 20)
    outs = []
    for fill in (0.0, float("nan"), float("inf")):
        ws = torch.full((need // 4,), fill, device=DEV)
        y, t = bl.adapters_forward(P.x, P.ads, P.ids, torch.zeros(300, 300, device=DEV), return_low=True, workspace=ws)
        ws.fill_(fill)
        outs.append((y, t, *bl.adapters_backward(P.dy, P.x, t, P.ads, P.ids, workspace=ws)))
    for o in outs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(o, outs[0]))


def test_outputs_stay_inside_odd_addresses():
    M, K, N, R, A = 19, 37, 45, 5, 2
    P = Problem(M, K, N, R, A)

    def odd(t):  # one element off, in a larger array
        return torch.empty(t.numel() + 1, dtype=t.dtype, device=DEV)[1:].view(t.shape).copy_(t)
    ads = tuple(odd(w) for w in P.ads)
    buf = torch.full((M * N + 65,), 7.0, device=DEV)
    y = buf[1:M * N + 1].view(M, N).zero_()
    bl.adapters_forward(odd(P.x), ads, P.ids, y)
    ref, t = bl.adapters_forward(P.x, P.ads, P.ids, torch.zeros(M, N, device=DEV), return_low=True)
    assert torch.equal(y, ref) and buf[0] == 7 and (buf[M * N + 1:] == 7).all()
    dbuf = torch.full((M * K + 65,), 7.0, device=DEV)
    dx = dbuf[1:M * K + 1].view(M, K).zero_()
    _, dd, du = bl.adapters_backward(odd(P.dy), odd(P.x), odd(t), ads, P.ids, dX=dx)
    rx, rd, ru = bl.adapters_backward(P.dy, P.x, t, P.ads, P.ids)
    assert torch.equal(dx, rx) and torch.equal(dd, rd) and torch.equal(du, ru)
    assert dbuf[0] == 7 and (dbuf[M * K + 1:] == 7).all()


def test_streams_and_graph():
    M, K, N, R, A = 48, 160, 200, 16, 4
    P = Problem(M, K, N, R, A, order="requests")
    packed, gamma = bl.quantize_weights(on_gpu(P.rng.standard_normal((N, K)) * 0.02))

    def step(x, dy, ids):
        xd = bl.dropout(x, 0.25, 77, 3)
        y, t = bl.adapters_forward(xd, P.ads, ids, bl.forward(x, packed, gamma, K), return_low=True)
        dxd, dd, du = bl.adapters_backward(dy, xd, t, P.ads, ids)
        return y, bl.dropout(dxd, 0.25, 77, 3), dd, du, bl.adapted_forward(x[:1].contiguous(), packed, gamma, P.ads, ids[:1].contiguous())

    same = lambda a, b: all(torch.equal(p, q) for p, q in zip(a, b))  # noqa: E731
    ref = step(P.x, P.dy, P.ids)
    torch.cuda.synchronize()
    got = []
    for s in (torch.cuda.Stream(), torch.cuda.Stream()):
        with torch.cuda.stream(s):
            got.append(step(P.x, P.dy, P.ids))
    torch.cuda.synchronize()
    assert same(got[0], ref) and same(got[1], ref)
    x, dy, ids = P.x.clone(), P.dy.clone(), P.ids.clone()
    step(x, dy, ids)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(x, dy, ids)
    for k in range(4):
        x.copy_(torch.roll(P.x, k, 0))
        dy.copy_(torch.roll(P.dy, -k, 0))
        ids.copy_(torch.roll(P.ids, 3 * k, 0))
        graph.replay()
        eager = step(torch.roll(P.x, k, 0), torch.roll(P.dy, -k, 0), torch.roll(P.ids, 3 * k, 0))
        torch.cuda.synchronize()
        assert same(out, eager)


@pytest.mark.parametrize("M,K,N,R", [(64, 4090, 130, 16), (300, 300, 260, 16), (40, 70, 90, 33)])
def test_projection_in_a_graph(M, K, N, R):
    # K in parts, the GEMM's epilogue, and a pass of its own
    P = Problem(M, K, N, R, 4, order="requests")
    packed, gamma = bl.quantize_weights(on_gpu(P.rng.standard_normal((N, K)) * 0.02))
    call = lambda x, ids: bl.adapted_forward(x, packed, gamma, P.ads, ids, return_low=True)  # noqa: E731
    x, ids = P.x.clone(), P.ids.clone()
    call(x, ids)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(x, ids)
    for k in range(4):
        x.copy_(torch.roll(P.x, k, 0))
        ids.copy_(torch.roll(P.ids, 3 * k, 0))
        graph.replay()
        eager = call(torch.roll(P.x, k, 0), torch.roll(P.ids, 3 * k, 0))
        torch.cuda.synchronize()
        assert torch.equal(out[0], eager[0]) and torch.equal(out[1], eager[1])


def test_more_outputs_than_32_bits():
    M, K, N, R = 70000, 8, 40000, 4  # 2.8e9 outputs
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randn(M, K, generator=g, device=DEV)
    ads = (torch.randn(2, R, K, generator=g, device=DEV), torch.randn(2, R, N, generator=g, device=DEV), torch.ones(2, device=DEV))
    ids = (torch.arange(M, device=DEV) // 100 % 3).to(torch.int32)  # 2: none
    y = torch.zeros(M, N, device=DEV)
    bl.adapters_forward(x, ads, ids, y)
    for m in (0, 101, 250, 53687, 53688, 69800, M - 1):
        a = int(ids[m])
        ref = (x[m].double() @ ads[0][a].double().T) @ ads[1][a].double() if a < 2 else torch.zeros(N, dtype=torch.float64, device=DEV)
        assert (y[m].double() - ref).abs().max() <= 1e-4 * (1 if a < 2 else 0)  # 12 terms of at most 50, 2^-24 each


def test_more_codes_than_32_bits():
    # the GEMM goes through the tokens in chunks of less than 2^31 codes
    M, K, N, R = 2100, 1 << 20, 8, 16
    g = torch.Generator(device=DEV).manual_seed(3)
    x = torch.randn(M, K, generator=g, device=DEV).bfloat16()
    packed, gamma = bl.quantize_weights(torch.randn(N, K, generator=g, device=DEV) * 0.02)
    ads = (torch.randn(2, R, K, generator=g, device=DEV), torch.randn(2, R, N, generator=g, device=DEV), torch.ones(2, device=DEV))
    ids = (torch.arange(M, device=DEV) // 300 % 3).to(torch.int32)  # 2: none
    base = bl.forward(x, packed, gamma, K)
    y, t = bl.adapted_forward(x, packed, gamma, ads, ids, return_low=True)
    two, t2 = bl.adapters_forward(x, ads, ids, base.clone(), return_low=True)
    assert torch.equal(t, t2) and torch.equal(y[ids == 2], base[ids == 2])
    up = torch.cat([ads[1], torch.zeros_like(ads[1][:1])])[ids.long()].double()
    terms = base.double().abs() + (t.double().abs()[:, :, None] * up.abs()).sum(1)
    ref = base.double() + (t.double()[:, :, None] * up).sum(1)
    for out in (y, two):  # 16 terms of three planes' products, their sum with the projection
        assert ((out.double() - ref).abs() <= terms * (R + 72) * U24).all()


@pytest.mark.parametrize("M", [5, 260])
def test_gradients_of_very_long_outputs(M):
    # more than 2^24 outputs, V's sums in several parts; positive values, so a part that is lost shows
    K, N, R = 16, (1 << 24) + 12, 2
    g = torch.Generator(device=DEV).manual_seed(M)
    pos = lambda *s: torch.rand(*s, generator=g, device=DEV) + 0.5  # noqa: E731
    dy = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
    for m in range(M):
        dy[m] = pos(N)
    x, t, ads = pos(M, K), pos(M, R), (pos(2, R, K), pos(2, R, N), pos(2))
    ids = (torch.arange(M, device=DEV) % 3).to(torch.int32)  # 2: none
    need = bl.abi.load().bitlinear_adapters_backward_workspace_bytes(M, K, N, 2, R)
    ws = torch.full((need // 4,), float("nan"), device=DEV)
    dx, dd, du = bl.adapters_backward(dy, x, t, ads, ids, workspace=ws)
    V = torch.zeros(M, R, dtype=torch.float64, device=DEV)
    for m in range(M):
        if m % 3 < 2:
            V[m] = float(ads[2][m % 3]) * (ads[1][m % 3].double() @ dy[m].double())
    # a term passes at most the 2^24 / 32 / 4 steps of a wave (M = 260 has one part), four roundings each,
    # and fewer than 400 others
    tol = (4 * 131073 + 400) * U24
    for a in range(2):
        at = torch.arange(a, M, 3, device=DEV)
        ref = V[at] @ ads[0][a].double()
        assert ((dx[at] - ref).abs() <= tol * ref).all()
        ref = V[at].T @ x[at].double()
        assert ((dd[a] - ref).abs() <= tol * ref).all()
        for n0 in range(0, N, 1 << 22):
            part = slice(n0, n0 + (1 << 22))
            ref = float(ads[2][a]) * (t[at].double().T @ dy[at][:, part].double())
            assert ((du[a][:, part] - ref).abs() <= (M + 72) * U24 * ref).all()
    assert not dx[2::3].any()


def test_refused_on_the_gpu():
    P = Problem(4, 64, 32, 2, 2)
    y = torch.zeros(4, 32, device=DEV)
    dn, up, sc = P.ads
    for call in (lambda: bl.adapters_forward(P.x, (dn, up.float(), sc), P.ids, y),
                 lambda: bl.adapters_forward(P.x, (dn, up[:1], sc), P.ids, y),
                 lambda: bl.adapters_forward(P.x, (dn, up, sc[:1]), P.ids, y),
                 lambda: bl.adapters_forward(P.x, P.ads, P.ids.long(), y),
                 lambda: bl.adapters_forward(P.x, P.ads, P.ids[:3], y),
                 lambda: bl.adapters_forward(P.x, P.ads, P.ids, y[:3]),
                 lambda: bl.adapters_forward(P.x, P.ads, P.ids, y.half()),
                 lambda: bl.adapters_forward(P.x.t(), P.ads, P.ids, y),
                 lambda: bl.adapters_forward(P.x, P.ads, P.ids.cpu(), y),
                 lambda: bl.adapters_backward(P.dy, P.x, None, P.ads, P.ids),
                 lambda: bl.adapters_backward(P.dy, P.x[:2], y, P.ads, P.ids),
                 lambda: bl.adapters_backward(P.dy, P.x, y[:, :2].contiguous(), P.ads, P.ids, need_dx=False, need_dw=False),
                 lambda: bl.dropout(P.x, 1.0, 0), lambda: bl.dropout(P.x, 0.5, -1), lambda: bl.dropout(P.x, 0.5, 1 << 64),
                 lambda: bl.dropout(P.x, 0.5, 0, residual=y), lambda: bl.dropout(P.x.half(), 0.5, 0),
                 lambda: bl.dropout(P.x, 0.5, 0, out=y)):
        with pytest.raises((ValueError, bl.BitLinearError)):
            call()


# ---- dropout ------------------------------------------------------------------

@pytest.mark.parametrize("shape", [(1,), (7,), (8,), (3, 11), (130, 129), (5, 4096)])
@pytest.mark.parametrize("xt", ["f32", "bf16"])
def test_dropout_bit_exact(shape, xt):
    rng = np.random.default_rng(shape[-1])
    x, r = (to_type(rng.standard_normal(shape), xt) for _ in range(2))
    for p, seed, offset in ((0.0, 0, 0), (0.1, 3, 5), (0.5, (1 << 64) - 1, 1 << 40), (0.999, 1 << 33, (1 << 64) - 1)):
        for out in ("f32", "bf16"):
            got = bl.dropout(on_gpu(x, xt), p, seed, offset, out_dtype=DT[out])
            assert np.array_equal(np_of(got), to_type(AO.dropout(x, p, seed, offset), out))
            for rt in ("f32", "bf16"):
                rr = to_type(r, rt)
                got = bl.dropout(on_gpu(x, xt), p, seed, offset, residual=on_gpu(rr, rt), out_dtype=DT[out])
                assert np.array_equal(np_of(got), to_type(AO.dropout(x, p, seed, offset, rr), out))


def test_dropout_in_place_and_special_values():
    x = torch.randn(33, 65, device=DEV)
    r = torch.randn(33, 65, device=DEV)
    ref = bl.dropout(x, 0.4, 9, residual=r)
    for a in (0, 1):
        y = [x.clone(), r.clone()]
        assert torch.equal(bl.dropout(y[0], 0.4, 9, residual=y[1], out=y[a]), ref) and torch.equal(y[a], ref)
    keep = torch.from_numpy(AO.kept(0, x.numel(), 0.4, 9, 0).reshape(33, 65)).to(DEV)
    for v in (float("nan"), float("inf")):
        y = bl.dropout(torch.full_like(x, v), 0.4, 9)
        assert (y[~keep] == 0).all() and not torch.isfinite(y[keep]).any()
    # the gradient: the same mask and scale
    d = bl.dropout(torch.ones_like(x), 0.4, 9)
    assert torch.equal(d != 0, keep) and torch.equal(d * x, bl.dropout(x, 0.4, 9))
    # an odd address, and values behind the end
    buf = torch.full((100,), 7.0, device=DEV)
    out = bl.dropout(buf[1:52].clone(), 0.4, 9, out=buf[1:52])
    assert torch.equal(out, bl.dropout(torch.full((51,), 7.0, device=DEV), 0.4, 9)) and (buf[52:] == 7).all() and buf[0] == 7


def test_dropout_of_more_than_32_bits():
    n = (1 << 33) + (1 << 20) + 5  # over two launches, and counters whose block number passes 2^31
    x = torch.ones(n, dtype=torch.bfloat16, device=DEV)
    y = bl.dropout(x, 0.5, 11, 12, out=x)
    for first in (0, (1 << 32) - 50, (1 << 33) - 50, n - 101):
        assert np.array_equal(np_of(y[first:first + 100]) != 0, AO.kept(first, 100, 0.5, 11, 12))
    assert abs(float(y[-(1 << 20):].float().mean()) - 1.0) < 5 * 2.0 ** -10


# ---- a fine-tuning step and a served batch, as they would be used ---------------

def test_a_gated_block_with_adapters_trains_and_serves():
    """Gated block whose down projection is frozen and adapted, dropout in front of the adapter: gradients
    against the oracle stage by stage."""
    from oracle import gated as GO
    M, D, F, R, A = 70, 128, 192, 8, 2
    rng = np.random.default_rng(4)
    P = Problem(M, F, D, R, A, "f32", "f32", "requests")
    X = to_type(rng.standard_normal((M, D)), "bf16")
    x = on_gpu(X, "bf16")
    W = [(rng.standard_normal(s) * 0.02).astype(np.float32) for s in ((F, D), (F, D), (D, F))]
    q = [O.quantize_weights(w) for w in W]
    gate, up, down = (bl.quantize_weights(on_gpu(w)) for w in W)
    # forward: hidden layer, dropped copy for the adapter, both products
    codes = bl.quantize_activations(x)
    h, g, u = bl.gated_forward(codes, gate, up, K=D, save=torch.float32)
    G, U = GO.projections(X, q[0][1], q[0][0], q[1][1], q[1][0])
    H = GO.hidden("relu2", G, U)
    assert np.array_equal(np_of(h), H)
    hd = bl.dropout(h, 0.2, 5)
    Hd = AO.dropout(H, 0.2, 5)
    assert np.array_equal(np_of(hd), Hd)
    y, t = bl.adapters_forward(hd, P.ads, P.ids, bl.forward(h, *down, F), return_low=True)
    gA, Hq, _ = O.absmax_quantize(H)
    base = O.dequant_f32(O.zero_gemm(Hq, q[2][1]), q[2][0], gA)
    P.X = Hd
    P.check_forward(y, t, base)
    # backward: through both, then through the gated product
    dY = to_type(rng.standard_normal((M, D)), "bf16")
    dy = on_gpu(dY, "bf16")
    P.dY = dY
    dhd, dd, du = bl.adapters_backward(dy, hd, t, P.ads, P.ids)
    P.check_backward(dhd, dd, du, np.zeros_like(Hd))
    downT, mask = bl.pack_transposed(on_gpu(W[2]), down[1])
    dbase = bl.backward(dy, downT, down[1], None, None, None, F, need_dw=False)[0]
    dh = bl.dropout(dhd, 0.2, 5, residual=dbase)
    keep = AO.kept(0, M * F, 0.2, 5, 0).reshape(M, F)
    assert np.array_equal(np_of(dh), np.where(keep, np_of(dhd) * np.float32(1.25), np.float32(0)) + np_of(dbase))
    dG, dU = bl.gated_backward(dh, g, u)
    rG, rU = GO.hidden_backward("relu2", np_of(dh), G, U)
    assert np.array_equal(np_of(dG), to_type(rG, "bf16")) and np.array_equal(np_of(dU), to_type(rU, "bf16"))
    # serving: one token of each request, the same adapters, beside the same projection
    last = torch.tensor([5, 30, 69], device=DEV)
    served = bl.adapted_forward(h[last].contiguous(), *down, P.ads, P.ids[last].contiguous())
    whole = bl.adapted_forward(h, *down, P.ads, P.ids)
    # the products' sums may be cut into other parts: twice the bound of one
    P.X = H
    T = AO.low(np.abs(H), P.rows, np.abs(P.down))
    tol = (np.abs(base) + AO.added(T, P.rows, np.abs(P.up), P.scales)) * 2 * (F + R + 144) * U24
    at = last.cpu().numpy()
    assert (np.abs(np_of(served) - np_of(whole)[at]) <= tol[at]).all()
