"""The gated feed-forward block on the GPU against the oracle.

Bit-exact: G, U, the ReLU^2 hidden layer, its gradients and the whole ReLU^2
block (single float32 operations on exact sums, rounded once more for bfloat16).
SiLU: within the first-order bound of its float32 operations, u = 2^-24 each.
The sigmoid is off by 8 u at most: 2 for exp2, 1 for its tail's FMA, 1 for the
sum, 2 for the reciprocal, 1 for the tail's own roundings and 1 for what the two
parts of the exponent leave out.
"""
import numpy as np
import pytest
import torch

import bitlinear_absmean_ternarise_bit_amd as bl
import oracle as O
from bitlinear_absmean_ternarise_bit_amd.workloads import bf16_bits_to_f32, f32_to_bf16_bits
from oracle import gated as GO

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
U24 = 2.0 ** -24


def to_type(x, dt):
    x = np.asarray(x, np.float32)
    return bf16_bits_to_f32(f32_to_bf16_bits(x)) if dt == "bf16" else x


def on_gpu(a, dt="f32"):
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(DEV).to(DT[dt])


def np_of(t):
    return t.float().cpu().numpy()


def same(a, b):
    return a.shape == b.shape and np.array_equal(a, b)


def step(dt):  # half a step of the output type
    return 2.0 ** -8 if dt == "bf16" else U24


class Matrix:
    """A ternary matrix: float32 weights, the oracle's codes and the GPU's packed form."""

    def __init__(self, rng, N, K, backward=False):
        self.W = (rng.standard_normal((N, K)) * 0.02).astype(np.float32)
        self.gamma, self.q, _ = O.quantize_weights(self.W)
        w = on_gpu(self.W)
        self.gpu = bl.quantize_weights(w)
        if backward:
            self.T, self.mask = bl.pack_transposed(w, self.gpu[1])


class Problem:
    def __init__(self, M, D, F, seed=0, dt="f32", backward=False):
        rng = np.random.default_rng(seed + 1000 * M + D + F)
        self.rng = rng
        self.X = to_type(rng.standard_normal((M, D)) * np.where(rng.random(D) < 0.05, 10.0, 1.0), dt)
        self.x = on_gpu(self.X, dt)
        self.gate, self.up = Matrix(rng, F, D, backward), Matrix(rng, F, D, backward)
        self.G, self.U = GO.projections(self.X, self.gate.q, self.gate.gamma, self.up.q, self.up.gamma)


def silu_close(got, G, U, dt):
    ref = GO.hidden("silu", G, U)
    # 8 u of the sigmoid, two products; far below zero the sigmoid stops at 2^-126
    tol = np.abs(ref) * (11 * U24 + step(dt)) + np.abs(G.astype(np.float64) * U) * 2.0 ** -118 + 2.0 ** -130
    assert (np.abs(got.astype(np.float64) - ref) <= tol).all()


SIZES = [(1, 1, 1), (1, 64, 16), (1, 2048, 40), (1, 2050, 33), (2, 100, 17), (3, 7, 300), (8, 1003, 70), (9, 300, 129),
         (16, 520, 48), (16, 4032, 100), (17, 64, 128), (40, 129, 65), (130, 1000, 260), (257, 192, 129), (300, 65, 1)]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("M,D,F", SIZES)
def test_hidden_layer(M, D, F, dt):
    print(f"gated M={M} D={D} F={F} {dt}", flush=True)
    P = Problem(M, D, F, dt=dt)
    gate, up = P.gate.gpu, P.up.gpu
    paths = ["auto", "prefill"] + (["decode"] if bl.decode_fits(M, D, F) else [])
    H = GO.hidden("relu2", P.G, P.U)
    codes = bl.quantize_activations(P.x)
    for path in paths:
        for out in ("f32", "bf16"):
            h, g, u = bl.gated_forward(P.x, gate, up, out_dtype=DT[out], save=DT["f32"], path=path)
            assert same(np_of(g), P.G) and same(np_of(u), P.U) and h.dtype == DT[out]
            assert same(np_of(h), to_type(H, out))
            s = bl.gated_forward(P.x, gate, up, act="silu", out_dtype=DT[out], path=path)
            silu_close(np_of(s), P.G, P.U, out)
            if path == "auto":
                h2, g2, u2 = bl.gated_forward(codes, gate, up, K=D, out_dtype=DT[out], save=DT["bf16"])
                assert torch.equal(h2, h) and same(np_of(g2), to_type(P.G, "bf16")) and same(np_of(u2), to_type(P.U, "bf16"))
                assert torch.equal(bl.gated_forward(codes, gate, up, K=D, act="silu", out_dtype=DT[out]), s)


def test_tiles_of_every_kind():
    # 256 x 128 tiles alone, with a last round of 128 x 128 ones (two launches), and 128-token tiles
    for M, D, F in ((2048, 64, 4096), (2048, 128, 5000), (1024, 192, 2900), (128, 64, 3200), (300, 64, 20000),
                    (1024, 64, 11008), (500, 64, 5632), (300, 64, 11008), (33, 64, 11008), (2300, 64, 11008)):
        print(f"tiles M={M} F={F}", flush=True)
        P = Problem(M, D, F, dt="bf16")
        h, g, u = bl.gated_forward(P.x, P.gate.gpu, P.up.gpu, save=torch.float32)
        assert same(np_of(g), P.G) and same(np_of(u), P.U) and same(np_of(h), GO.hidden("relu2", P.G, P.U))


@pytest.mark.parametrize("M,D,F,Do,dt", [(1, 64, 48, 64, "f32"), (8, 300, 129, 70, "bf16"), (16, 500, 333, 40, "f32"),
                                         (33, 257, 190, 257, "bf16"), (300, 130, 450, 64, "f32"), (4, 16200, 20, 30, "bf16"),
                                         (17, 64, 2000, 130, "f32"), (64, 100, 4095, 40, "bf16"),
                                         (200, 70, 1400, 300, "f32")])
def test_block(M, D, F, Do, dt):
    P = Problem(M, D, F, dt=dt)
    down = Matrix(P.rng, Do, F)
    H = GO.hidden("relu2", P.G, P.U)
    gA, Hq, _ = O.absmax_quantize(H)
    ref = O.dequant_f32(O.zero_gemm(Hq, down.q), down.gamma, gA)
    for path in ["auto", "prefill"] + (["decode"] if bl.decode_fits(M, D, F) and bl.decode_fits(M, F, Do) else []):
        y, h = bl.gated_ffn_forward(P.x, P.gate.gpu, P.up.gpu, down.gpu, path=path, return_hidden=True)
        assert same(np_of(h), H) and same(np_of(y), ref)
        assert torch.equal(bl.gated_ffn_forward(P.x, P.gate.gpu, P.up.gpu, down.gpu, path=path), y)
    # the SiLU block from its own hidden layer
    y, h = bl.gated_ffn_forward(P.x, P.gate.gpu, P.up.gpu, down.gpu, act="silu", return_hidden=True)
    silu_close(np_of(h), P.G, P.U, "f32")
    gA, Hq, _ = O.absmax_quantize(np_of(h))
    assert same(np_of(y), O.dequant_f32(O.zero_gemm(Hq, down.q), down.gamma, gA))


@pytest.mark.parametrize("M,F", [(1, 1), (1, 7), (3, 11), (5, 64), (130, 1003), (2, 100000)])
@pytest.mark.parametrize("kept", ["f32", "bf16"])
@pytest.mark.parametrize("act", ["relu2", "silu"])
def test_activation_backward(M, F, kept, act):
    rng = np.random.default_rng(M + F)
    G, U = (to_type(rng.standard_normal((M, F)) * 4, kept) for _ in range(2))
    if F >= 7:
        G[0, :7] = [0.0, -0.0, -300.0, 300.0, -100.0, 1e-30, -90.0]
        G = to_type(G, kept)  # the oracle sees what the GPU is given
    for dh in ("f32", "bf16"):
        dH = to_type(rng.standard_normal((M, F)), dh)
        rG, rU = GO.hidden_backward(act, dH, G, U)
        for out in ("f32", "bf16"):
            dG, dU = (np_of(t) for t in bl.gated_backward(on_gpu(dH, dh), on_gpu(G, kept), on_gpu(U, kept), act=act,
                                                          out_dtype=DT[out]))
            if act == "relu2":
                assert same(dG, to_type(rG, out)) and same(dU, to_type(rU, out))
                continue
            s, g = GO.sigmoid(G), G.astype(np.float64)
            du = np.abs(dH.astype(np.float64) * U)
            # 1 - s is off by 8 u s + u, its FMA by another u of the sum; then s and two products
            tol = du * s * (9 * np.abs(g) + 1 + 12 * np.abs(1 + g * (1 - s))) * U24 + np.abs(rG) * step(out)
            assert (np.abs(dG - rG) <= tol + du * np.abs(g) * 2.0 ** -118 + 2.0 ** -130).all()
            tol = np.abs(rU) * (11 * U24 + step(out)) + np.abs(dH * g) * 2.0 ** -118 + 2.0 ** -130
            assert (np.abs(dU - rU) <= tol).all()


def test_activation_backward_special_values():
    n, i = np.nan, np.inf
    G = np.array([[n, i, -i, 1.0, 1.0, -1.0, 0.0, 2.0]], np.float32)
    U = np.array([[1.0, 1.0, 1.0, n, i, i, 3.0, 1.0]], np.float32)
    dH = np.array([[1.0, 1.0, 1.0, 1.0, 1.0, 1.0, i, n]], np.float32)
    dG, dU = (np_of(t) for t in bl.gated_backward(on_gpu(dH), on_gpu(G), on_gpu(U), out_dtype=torch.float32))
    with np.errstate(invalid="ignore"):
        rG, rU = GO.hidden_backward("relu2", dH, G, U)
    assert np.array_equal(dG, rG, equal_nan=True) and np.array_equal(dU, rU, equal_nan=True)
    sG, sU = (np_of(t) for t in bl.gated_backward(on_gpu(dH), on_gpu(G), on_gpu(U), act="silu", out_dtype=torch.float32))
    # g s = -inf 0 at minus infinity
    assert np.isnan(sG[0, [0, 3, 7]]).all() and np.isnan(sU[0, [0, 2, 7]]).all() and sU[0, 1] == i


@pytest.mark.parametrize("M,D,F", [(1, 1, 1), (3, 70, 33), (40, 200, 136), (257, 129, 200), (300, 300, 1000), (64, 4100, 64), (5, 30, 2000),
                                   (70, 65, 4099)])
def test_products_backward(M, D, F):
    print(f"products M={M} D={D} F={F}", flush=True)
    P = Problem(M, D, F, dt="bf16", backward=True)
    codes = bl.quantize_activations(P.x)
    h, g, u = bl.gated_forward(codes, P.gate.gpu, P.up.gpu, K=D, save=torch.bfloat16)
    dH = on_gpu(P.rng.standard_normal((M, F)))
    dG, dU = bl.gated_backward(dH, g, u)
    rG, rU = GO.hidden_backward("relu2", np_of(dH), np_of(g), np_of(u))
    assert same(np_of(dG), to_type(rG, "bf16")) and same(np_of(dU), to_type(rU, "bf16"))
    gateT, upT = (P.gate.T, P.gate.gpu[1]), (P.up.T, P.up.gpu[1])
    dX = np_of(bl.gated_input_backward(dG, dU, gateT, upT, D))
    a, b = np_of(dG), np_of(dU)
    ref = GO.input_backward(a, b, P.gate.q, P.gate.gamma, P.up.q, P.up.gamma)
    terms = GO.input_backward(np.abs(a), np.abs(b), np.abs(P.gate.q), P.gate.gamma, np.abs(P.up.q), P.up.gamma)
    assert (np.abs(dX - ref) <= terms * (F + 8) * U24).all()
    # odd addresses take padded copies: the same bits
    odd = [torch.empty(M * F + 1, dtype=torch.bfloat16, device=DEV)[1:].view(M, F).copy_(t) for t in (dG, dU)]
    assert same(np_of(bl.gated_input_backward(*odd, gateT, upT, D)), dX)
    # the weights' gradients come from the backward that is there
    for d, m in ((dG, P.gate), (dU, P.up)):
        dW = np_of(bl.backward(d, m.T, m.gpu[1], codes[0], codes[1], m.mask, D, need_dx=False)[1])
        gA, Xq, _ = O.absmax_quantize(P.X)
        r = O.ste_backward(np_of(d), m.q, m.gamma, Xq, gA, m.W)["dW"]
        bound = np.abs(np_of(d)).astype(np.float64).T @ np.abs(O.dequant_activations_bf16(Xq, gA)).astype(np.float64)
        assert (np.abs(dW - r) <= bound * (M + 8) * U24 + np.abs(r) * U24).all()


def test_input_gradient_of_a_zero_matrix():
    # gamma 0: the other product alone
    P = Problem(20, 64, 72, dt="bf16", backward=True)
    dG, dU = (torch.randn(20, 72, device=DEV).to(torch.bfloat16) for _ in range(2))
    zero = torch.zeros(1, device=DEV)
    for first, second, q, gamma, d in (((P.gate.T, zero), (P.up.T, P.up.gpu[1]), P.up.q, P.up.gamma, dU),
                                       ((P.gate.T, P.gate.gpu[1]), (P.up.T, zero), P.gate.q, P.gate.gamma, dG)):
        dX = np_of(bl.gated_input_backward(dG, dU, first, second, 64))
        only = np_of(bl.backward(d, (second if first[1] is zero else first)[0], torch.tensor([gamma], device=DEV), None,
                                 None, None, 64, need_dw=False)[0])
        assert same(dX, only)


def test_outputs_stay_inside():
    # rows and values behind the outputs keep their contents
    M, D, F = 19, 100, 77
    P = Problem(M, D, F, dt="bf16")
    for m in (1, 5, 19):
        buf = torch.full((m * F + 64,), 7.0, device=DEV)
        h = bl.gated_forward(P.x[:m].contiguous(), P.gate.gpu, P.up.gpu, out=buf[:m * F].view(m, F))
        assert same(np_of(h), GO.hidden("relu2", P.G[:m], P.U[:m])) and (buf[m * F:] == 7).all()
        d = torch.full((m * F + 64,), 7.0, device=DEV)
        big = torch.empty(m * F + 1, device=DEV)[1:].view(m, F).copy_(h)   # inputs at an odd address
        dG, dU = bl.gated_backward(big, h, h, out_dtype=torch.float32)
        r = GO.hidden_backward("relu2", np_of(h), np_of(h), np_of(h))
        assert same(np_of(dG), r[0]) and same(np_of(dU), r[1]) and (d == 7).all()


def test_streams_and_graph():
    M, D, F = 40, 256, 192
    P = Problem(M, D, F, dt="bf16", backward=True)
    ref_h, ref_g, ref_u = bl.gated_forward(P.x, P.gate.gpu, P.up.gpu, save=torch.bfloat16)
    one = P.x[:1].contiguous()
    ref_1 = bl.gated_forward(one, P.gate.gpu, P.up.gpu)
    gateT, upT = (P.gate.T, P.gate.gpu[1]), (P.up.T, P.up.gpu[1])
    ref_dx = bl.gated_input_backward(*bl.gated_backward(ref_h, ref_g, ref_u), gateT, upT, D)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in streams:
        with torch.cuda.stream(s):
            h, g, u = bl.gated_forward(P.x, P.gate.gpu, P.up.gpu, save=torch.bfloat16)
            got.append((h, bl.gated_input_backward(*bl.gated_backward(h, g, u), gateT, upT, D),
                        bl.gated_forward(one, P.gate.gpu, P.up.gpu)))
    torch.cuda.synchronize()
    for h, dx, h1 in got:
        assert torch.equal(h, ref_h) and torch.equal(dx, ref_dx) and torch.equal(h1, ref_1)
    x, x1 = P.x.clone(), one.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h, g, u = bl.gated_forward(x, P.gate.gpu, P.up.gpu, save=torch.bfloat16)
        dx = bl.gated_input_backward(*bl.gated_backward(h, g, u), gateT, upT, D)
        h1 = bl.gated_forward(x1, P.gate.gpu, P.up.gpu)
    for k in range(4):
        new = torch.roll(P.x, k, 0)
        x.copy_(new)
        x1.copy_(new[:1])
        graph.replay()
        eager, eg, eu = bl.gated_forward(new, P.gate.gpu, P.up.gpu, save=torch.bfloat16)
        edx = bl.gated_input_backward(*bl.gated_backward(eager, eg, eu), gateT, upT, D)
        torch.cuda.synchronize()
        assert torch.equal(h, eager) and torch.equal(dx, edx)
        assert torch.equal(h1, bl.gated_forward(new[:1].contiguous(), P.gate.gpu, P.up.gpu))


def test_parts_in_a_graph():
    # the down product in parts of K, the input's gradient in parts of F
    M, D, F = 40, 100, 4095
    P = Problem(M, D, F, dt="bf16", backward=True)
    down = Matrix(P.rng, 60, F).gpu
    gateT, upT = (P.gate.T, P.gate.gpu[1]), (P.up.T, P.up.gpu[1])
    dG, dU = (torch.randn(M, F, device=DEV).to(torch.bfloat16) for _ in range(2))
    call = lambda x, a, b: (bl.gated_ffn_forward(x, P.gate.gpu, P.up.gpu, down),  # noqa: E731
                            bl.gated_input_backward(a, b, gateT, upT, D))
    x, a, b = P.x.clone(), dG.clone(), dU.clone()
    call(x, a, b)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(x, a, b)
    for k in range(4):
        for to, src in ((x, P.x), (a, dG), (b, dU)):
            to.copy_(torch.roll(src, k, 0))
        graph.replay()
        eager = call(*(torch.roll(t, k, 0) for t in (P.x, dG, dU)))
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, eager))


@pytest.mark.parametrize("K", [1, 7, 8, 9, 63, 2041, 2049, 8191, 8193, 28671, 28673])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_codes_of_rows_of_any_length(K, dt):
    M = 6
    X = to_type(np.random.default_rng(K).standard_normal((M, K)) * 3, dt)
    X[2] = 0.0
    buf = torch.empty(M * K + 1, dtype=DT[dt], device=DEV)
    for x in (on_gpu(X, dt), buf[1:].view(M, K).copy_(on_gpu(X, dt))):  # and rows one value off
        Xq, ga, rs = bl.quantize_activations(x)
        gA, q, r = O.absmax_quantize(X)
        assert np.array_equal(Xq.cpu().numpy()[:, :K], q) and not Xq[:, K:].any()
        assert same(np_of(ga), gA) and np.array_equal(rs.cpu().numpy(), r)


def test_codes_of_more_rows_than_a_launch_has_groups():
    M, K = 1 << 24, 2049  # 69 GB, in rows that are not aligned
    if torch.cuda.mem_get_info()[0] < 140 << 30:
        pytest.skip("needs 140 GB of GPU memory")
    x = torch.zeros(M, K, dtype=torch.bfloat16, device=DEV)
    at = [0, 1, (1 << 23) + 3, M - 1]
    X = to_type(np.random.default_rng(5).standard_normal((len(at), K)), "bf16")
    for i, m in enumerate(at):
        x[m] = on_gpu(X[i], "bf16")
    Xq, ga, rs = bl.quantize_activations(x)
    del x
    gA, q, r = O.absmax_quantize(X)
    assert np.array_equal(Xq[at].cpu().numpy()[:, :K], q) and same(np_of(ga[at]), gA)
    assert np.array_equal(rs[at].cpu().numpy(), r) and int(ga.count_nonzero()) == len(at)
    del Xq
    torch.cuda.empty_cache()


def test_refused_on_the_gpu():
    P = Problem(4, 64, 32)
    w = P.gate.gpu
    other = Matrix(P.rng, 31, 64).gpu
    for call in (lambda: bl.gated_forward(P.x, w, other), lambda: bl.gated_forward(P.x[:, :60].contiguous()[:, :3].contiguous(), (w[0][:, :0], w[1]), w),
                 lambda: bl.gated_forward(P.x.half(), w, w), lambda: bl.gated_forward(P.x.t(), w, w),
                 lambda: bl.gated_forward(P.x, (w[0], w[1].cpu()), w), lambda: bl.gated_forward(P.x, w, w, out=P.x),
                 lambda: bl.gated_forward(P.x, w, w, K=65), lambda: bl.gated_forward(P.x, w, w, save=torch.float16),
                 lambda: bl.gated_backward(P.x, P.x, P.x.bfloat16()), lambda: bl.gated_backward(P.x, P.x[:2], P.x),
                 lambda: bl.gated_input_backward(P.x, P.x, w, w, 64),
                 lambda: bl.gated_forward((P.x, P.x, P.x), w, w, K=64)):
        with pytest.raises((ValueError, bl.BitLinearError)):
            call()
    with pytest.raises(bl.BitLinearError):
        bl.gated_forward(torch.zeros(40, 64, device=DEV), w, w, path="decode")
