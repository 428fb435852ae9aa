"""Gated feed-forward blocks, low-rank adapters and dropout, as they are measured.

All three stand beside the framework's ternary products: a gated block is the
FFN block with a second up projection, adapters are what a shared ternary
projection is fine-tuned and served with, and dropout stands in front of them
in training.  Shapes are those of the framework's workloads (d_model 2048 ->
FFN 5632, 4096 -> 11008, 8192 -> 28672) and odd ones of the same range.

Formulas (m: token, k: column of D, f: column of F, q: ternary codes in
{-1, 0, 1} with one float32 scale gamma a matrix, all steps in float32 as
written, fp32 where a rounding is part of the definition):

  codes   ga[m] = max_k |x|     s = fp32(127 / fp32(ga + 1e-5))
          xq = clip(rint(fp32(x s)), -128, 127)
  product P(x, q, gamma)[m, n] = (sum_k xq q[n, k]) fp32(fp32(gamma ga) / 127)
  gated   g = P(x, q_gate)      u = P(x, q_up)      h = act(g) u
          act: relu2, fp32(r r) with r = max(g, 0), or silu, g / (1 + exp(-g))
  block   y = P(h, q_down)
  grads   relu2: dg = bf16(fp32(dh fp32(u fp32(2 r))))   du = bf16(fp32(dh fp32(r r)))
          silu:  dg = bf16(dh u s (1 + g (1 - s)))       du = bf16(dh g s)     s = 1 / (1 + exp(-g))
          (from g and u as they were kept)
          dx = gamma_gate (dg q_gate) + gamma_up (du q_up)
          dW = (dg^T a) where |W| <= fp32(gamma + 1e-5), else 0    a = bf16(fp32(fp32(ga / 127) xq))
  adapted y[m] = P(x, q)[m] + scale[a] (x[m] down[a]^T) up[a]       a = rows[m]; none where a < 0
          t[m] = x[m] down[a]^T (zeros without an adapter)
          v[m] = scale[a] dy[m] up[a]^T       dx[m] += v[m] down[a]
          ddown[a] = sum_{rows = a} v^T x     dup[a] = scale[a] sum_{rows = a} t^T dy
  dropout y[i] = x[i] fp32(1 / (1 - p)) where w[i] >= round(p 2^32), else 0; plus the residual.
          w[i]: word i % 4 of Philox4x32-10 (Salmon et al. 2011) at counter
          (i / 4, offset), each 64 bits with the low word first, and key seed.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "bf16": 2}
EPS = 1e-5


def listed():
    return [
        # one token through a gated hidden layer, d_model 2048: latency, 5.8 MB of weights
        {"name": "gated 1x2048x5632 bf16", "op": "gated", "act": "relu2", "M": 1, "D": 2048, "F": 5632, "x": "bf16",
         "y": "f32"},
        # a decode batch through the whole block
        {"name": "gated block 8x2048x5632 bf16", "op": "block", "act": "relu2", "M": 8, "D": 2048, "F": 5632,
         "x": "bf16"},
        # prefill, 7B-like model, the SiLU form
        {"name": "gated 2048x4096x11008 silu", "op": "gated", "act": "silu", "M": 2048, "D": 4096, "F": 11008,
         "x": "bf16", "y": "bf16"},
        # prefill, 70B-like widths: the largest product
        {"name": "gated 8192x8192x28672 bf16", "op": "gated", "act": "relu2", "M": 8192, "D": 8192, "F": 28672,
         "x": "bf16", "y": "bf16"},
        # a ragged batch through the block of an odd-width model, float32
        {"name": "gated block 777x1003x2701 f32", "op": "block", "act": "relu2", "M": 777, "D": 1003, "F": 2701,
         "x": "f32"},
        # a training step of the gated hidden layer, 7B-like: forward, dX and both weights' gradients
        {"name": "gated step 2048x4096x11008", "op": "gated_step", "act": "relu2", "M": 2048, "D": 4096, "F": 11008,
         "x": "bf16", "y": "f32", "kept": "bf16", "products": True},
        # one token of one request with its adapter
        {"name": "adapted 1x2048x2048 r16", "op": "adapted", "M": 1, "K": 2048, "N": 2048, "R": 16, "A": 4,
         "requests": 1, "x": "bf16", "w": "bf16"},
        # a decode batch of sixteen requests with sixteen adapters
        {"name": "adapted 16x4096x4096 r16", "op": "adapted", "M": 16, "K": 4096, "N": 4096, "R": 16, "A": 16,
         "requests": 16, "x": "bf16", "w": "bf16"},
        # prefill of seven requests of ragged lengths, 7B-like up projection
        {"name": "adapted 2048x4096x11008 r16", "op": "adapted", "M": 2048, "K": 4096, "N": 11008, "R": 16, "A": 8,
         "requests": 7, "x": "bf16", "w": "bf16"},
        # a fine-tuning step of one adapter, float32 master weights, dropout in front of it, the projection frozen
        {"name": "adapter step 2048x4096x4096 r64", "op": "adapter_step", "M": 2048, "K": 4096, "N": 4096, "R": 64,
         "A": 1, "requests": 1, "x": "bf16", "w": "f32", "p": 0.1},
        # dropout of a branch added to the residual stream, 7B-like
        {"name": "dropout 2048x4096 residual", "op": "dropout", "M": 2048, "K": 4096, "x": "bf16", "y": "bf16",
         "residual": True, "p": 0.1},
        # the same without the residual, 70B-like width, float32 in
        {"name": "dropout 8192x8192 f32 to bf16", "op": "dropout", "M": 8192, "K": 8192, "x": "f32", "y": "bf16",
         "residual": False, "p": 0.25},
    ]


def draw(rng):
    def size(lo, hi, half=64):
        v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
        # half of the widths as models choose them, half as they fall
        return max(lo, v // half * half) if rng.random() < 0.5 else v

    t = lambda: rng.choice(["f32", "bf16"])  # noqa: E731
    op = rng.choice(["gated", "block", "gated_step", "adapted", "adapted", "adapter_step", "dropout"])
    M = size(1, 8192, 1)
    if op == "dropout":
        return {"op": op, "M": M, "K": size(1, 8192), "x": t(), "y": t(), "residual": rng.random() < 0.5,
                "p": rng.choice([0.0, 0.05, 0.1, 0.5, 0.9])}
    if op in ("gated", "block", "gated_step"):
        D, F = size(64, 8192), size(64, 11008)
        M = max(1, min(M, (1 << 36) // (D * F)))
        case = {"op": op, "act": "relu2", "M": M, "D": D, "F": F, "x": t()}
        if op != "block":
            case.update(act=rng.choice(["relu2", "silu"]), y=t())
        if op == "gated_step":
            # the products' gradients follow dg and du rounded to bfloat16, which the SiLU's
            # exponential does not pin: they are taken with relu2
            case.update(kept=t(), products=case["act"] == "relu2")
        return case
    K, N, R = size(64, 8192), size(64, 11008), rng.choice([4, 8, 16, 16, 32, 64, rng.randint(1, 64)])
    M = max(1, min(M, (1 << 36) // (K * N)))
    requests = max(1, min(M, int(round(math.exp(rng.uniform(0, math.log(16)))))))
    case = {"op": op, "M": M, "K": K, "N": N, "R": R, "A": rng.randint(1, 16), "requests": requests, "x": t(),
            "w": t()}
    if op == "adapter_step":
        case.update(p=rng.choice([0.0, 0.1]))
    return case


# ---- inputs ------------------------------------------------------------------

def padded(K):
    return (K + 63) // 64 * 64


def pack(q):
    """int8 codes in {-1, 0, 1} [N, K] in the 2-bit format: int32 [N, padded / 16]."""
    N, K = q.shape
    Kp = padded(K)
    c = torch.ones((N, Kp), dtype=torch.uint8, device=q.device)
    c[:, :K] = (q + 1).to(torch.uint8)
    c = c.view(N, Kp // 16, 4, 4)  # word, field i, byte b
    b = c[:, :, 0] | (c[:, :, 1] << 2) | (c[:, :, 2] << 4) | (c[:, :, 3] << 6)
    units = b.reshape(N, Kp // 64, 16)  # 16 bytes of 64 codes
    U, whole, last = Kp // 64, N // 16 * 16, Kp // 64 % 4
    parts = []

    def block(rows):  # [blocks, R, U, 16] -> blocks in chunks of four units, a chunk's rows one after another
        nb, R = rows.shape[:2]
        full = rows[:, :, :U - last].reshape(nb, R, (U - last) // 4, 64).transpose(1, 2).reshape(nb, -1)
        rest = rows[:, :, U - last:].reshape(nb, -1)
        return torch.cat([full, rest], dim=1).reshape(-1)

    if whole:
        parts.append(block(units[:whole].view(-1, 16, U, 16)))
    if N > whole:
        parts.append(block(units[whole:].unsqueeze(0)))
    return torch.cat(parts).view(torch.int32).view(N, Kp // 16)


def pack_bits(mask):
    """Truth values [N, K] as int32 [N, ceil(K / 32)], bit k % 32 of word k / 32."""
    N, K = mask.shape
    W = (K + 31) // 32
    m = torch.zeros((N, W * 32), dtype=torch.bool, device=mask.device)
    m[:, :K] = mask
    weight = 2 ** torch.arange(8, device=mask.device)
    return (m.view(N, W * 4, 8) * weight).sum(dim=2).to(torch.uint8).view(torch.int32)


def ternary(g, N, K, backward=False):
    """A ternary matrix as a program keeps it: codes, scale and packed form; for training also the
    packed transpose and the range mask."""
    dev = g.device
    w = 0.02 * torch.randn((N, K), generator=g, device=dev)
    gamma = w.abs().mean().view(1)
    d = gamma + EPS
    q = (torch.sign(w) * (w.abs() > 0.5 * d)).to(torch.int8)
    out = {"q": q, "gamma": gamma, "packed": pack(q)}
    if backward:
        out["inside"] = w.abs() <= d
        out["packedT"], out["mask"] = pack(q.T.contiguous()), pack_bits(out["inside"])
    return out


def stream(g, M, K):
    """A residual stream: a few loud channels, each channel with an offset of its own."""
    loud = torch.rand((K,), generator=g, device=g.device) < 0.01
    x = torch.randn((M, K), generator=g, device=g.device) * torch.where(loud, 10.0, 1.0)
    return x + 0.25 * torch.randn((K,), generator=g, device=g.device)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed))
    c, op, M = dict(case), case["op"], case["M"]
    s = {"case": c}
    if op == "dropout":
        s["x"] = stream(g, M, c["K"]).to(DTYPES[c["x"]])
        s["residual"] = stream(g, M, c["K"]).to(DTYPES[c["x"]]) if c["residual"] else None
        s["seed"], s["offset"] = 1234567890123 + int(seed), 7 * int(seed)
        return s
    if op in ("gated", "block", "gated_step"):
        D, F = c["D"], c["F"]
        s["x"] = stream(g, M, D).to(DTYPES[c["x"]])
        train = op == "gated_step" and c["products"]
        s["gate"], s["up"] = ternary(g, F, D, train), ternary(g, F, D, train)
        if op == "block":
            s["down"] = ternary(g, D, F)
        if op == "gated_step":
            s["dh"] = 1e-3 * torch.randn((M, F), generator=g, device=dev)  # as the down projection's backward writes it
        return s
    K, N, R, A = c["K"], c["N"], c["R"], c["A"]
    s["x"] = stream(g, M, K).to(DTYPES[c["x"]])
    s["base"] = ternary(g, N, K, op == "adapter_step")
    s["down"] = (torch.randn((A, R, K), generator=g, device=dev) / math.sqrt(K)).to(DTYPES[c["w"]])
    s["up"] = (0.5 * torch.randn((A, R, N), generator=g, device=dev) / math.sqrt(R)).to(DTYPES[c["w"]])
    s["scales"] = 0.5 + torch.rand((A,), generator=g, device=dev)
    # requests one after another, their lengths ragged, each with one adapter; every eighth has none
    cuts = torch.sort(torch.rand((c["requests"] - 1,), generator=g, device=dev)).values
    request = torch.searchsorted(cuts, (torch.arange(M, device=dev) + 0.5) / M)
    if M == c["requests"]:
        request = torch.arange(M, device=dev)
    ids = torch.randperm(max(A, c["requests"]), generator=g, device=dev) % A
    ids = ids[:c["requests"]].to(torch.int32)
    if c["requests"] > 1:
        ids[7::8] = -1
    s["rows"] = ids[request].contiguous()
    if op == "adapter_step":
        s["dy"] = (1e-3 * torch.randn((M, N), generator=g, device=dev)).to(torch.bfloat16)
        s["seed"] = 987654321 + int(seed)
    return s


def run(state):
    return run_own(state) if own else run_plain(state)


# ---- the framework's calls ----------------------------------------------------

def run_own(s):
    import bitlinear_absmean_ternarise_bit_amd as bl
    c, op, x = s["case"], s["case"]["op"], s["x"]
    if op == "dropout":
        return bl.dropout(x, c["p"], s["seed"], s["offset"], residual=s["residual"], out_dtype=DTYPES[c["y"]])
    if op in ("gated", "block", "gated_step"):
        gate, up = (s["gate"]["packed"], s["gate"]["gamma"]), (s["up"]["packed"], s["up"]["gamma"])
        if op == "gated":
            return bl.gated_forward(x, gate, up, act=c["act"], out_dtype=DTYPES[c["y"]])
        if op == "block":
            down = (s["down"]["packed"], s["down"]["gamma"])
            y, h = bl.gated_ffn_forward(x, gate, up, down, act=c["act"], return_hidden=True)
            return {"y": y, "h": h}
        codes = bl.quantize_activations(x)
        h, g, u = bl.gated_forward(codes, gate, up, K=c["D"], act=c["act"], out_dtype=DTYPES[c["y"]],
                                   save=DTYPES[c["kept"]])
        dg, du = bl.gated_backward(s["dh"], g, u, act=c["act"])
        if not c["products"]:
            return {"h": h, "dg": dg, "du": du}
        dx = bl.gated_input_backward(dg, du, (s["gate"]["packedT"], gate[1]), (s["up"]["packedT"], up[1]), c["D"])
        dwg, dwu = (bl.backward(d, w["packedT"], w["gamma"], codes[0], codes[1], w["mask"], c["D"], need_dx=False)[1]
                    for d, w in ((dg, s["gate"]), (du, s["up"])))
        return {"h": h, "dg": dg, "du": du, "dx": dx, "dwg": dwg, "dwu": dwu}
    base, adapters = s["base"], (s["down"], s["up"], s["scales"])
    if op == "adapted":
        return bl.adapted_forward(x, base["packed"], base["gamma"], adapters, s["rows"])
    if c["p"] == 0.0:
        y, t = bl.adapted_forward(x, base["packed"], base["gamma"], adapters, s["rows"], return_low=True)
        dx = bl.backward(s["dy"], base["packedT"], base["gamma"], None, None, None, c["K"], need_dw=False)[0]
        dx, ddown, dup = bl.adapters_backward(s["dy"], x, t, adapters, s["rows"], dX=dx)
        return {"y": y, "t": t, "dx": dx, "ddown": ddown, "dup": dup}
    xd = bl.dropout(x, c["p"], s["seed"])
    y = bl.forward(x, base["packed"], base["gamma"], c["K"])
    y, t = bl.adapters_forward(xd, adapters, s["rows"], y, return_low=True)
    dxd, ddown, dup = bl.adapters_backward(s["dy"], xd, t, adapters, s["rows"])
    dx = bl.backward(s["dy"], base["packedT"], base["gamma"], None, None, None, c["K"], need_dw=False)[0]
    dx = bl.dropout(dxd, c["p"], s["seed"], residual=dx, out=dxd)
    return {"y": y, "t": t, "dx": dx, "ddown": ddown, "dup": dup}


# ---- the plain forms ------------------------------------------------------------

def over(a, b):
    """a / b, one rounded division (by a number torch would multiply with its reciprocal)."""
    a = a if torch.is_tensor(a) else torch.full_like(b, a)
    return a / (b if torch.is_tensor(b) else torch.full_like(a, b))


def plain_codes(x):
    ga = x.abs().amax(dim=1, keepdim=True)
    s = over(127.0, ga + EPS)
    return torch.clamp(torch.round(x * s), -128.0, 127.0), ga


def plain_product(codes, w):
    xq, ga = codes
    return (xq @ w["q"].float().T) * over(w["gamma"] * ga, 127.0)  # sums of whole numbers below 2^24: exact


def plain_words(n, seed, offset, dev):
    """The n random words (as int64) of dropout's mask."""
    low = 0xffffffff
    i = torch.arange((n + 3) // 4, device=dev)
    c = [i & low, i >> 32, torch.full_like(i, offset & low), torch.full_like(i, offset >> 32 & low)]
    k0, k1 = seed & low, seed >> 32 & low

    def times(a, b):  # high and low words of a b
        return ((a >> 16) * b + ((a & 0xffff) * b >> 16)) >> 16, a * b & low

    for _ in range(10):
        h0, l0 = times(0xD2511F53, c[0])
        h1, l1 = times(0xCD9E8D57, c[2])
        c = [h1 ^ c[1] ^ k0, l1, h0 ^ c[3] ^ k1, l0]
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    return torch.stack(c, dim=1).view(-1)[:n]


def plain_dropout(x, p, seed, offset=0):
    keep = plain_words(x.numel(), seed, offset, x.device).view(x.shape) >= int(p * 2.0 ** 32 + 0.5)
    return torch.where(keep, x * (1.0 / (1.0 - p)), torch.zeros_like(x))


def plain_gated_grads(act, dh, g, u):
    if act == "relu2":
        r = torch.where(g > 0, g, torch.zeros_like(g))
        return dh * (u * (2.0 * r)), dh * (r * r)
    s = 1.0 / (1.0 + torch.exp(-g))
    return dh * u * (s * (1.0 + g * (1.0 - s))), dh * (g * s)


def run_plain(s):
    c, op = s["case"], s["case"]["op"]
    x = s["x"].float()
    if op == "dropout":
        y = plain_dropout(x, c["p"], s["seed"], s["offset"])
        return (y if s["residual"] is None else y + s["residual"].float()).to(DTYPES[c["y"]])
    if op in ("gated", "block", "gated_step"):
        codes = plain_codes(x)
        g, u = plain_product(codes, s["gate"]), plain_product(codes, s["up"])
        if c["act"] == "relu2":
            r = torch.where(g > 0, g, torch.zeros_like(g))
            h = r * r * u
        else:
            h = g / (1.0 + torch.exp(-g)) * u
        if op == "gated":
            return h.to(DTYPES[c["y"]])
        if op == "block":
            return {"y": plain_product(plain_codes(h), s["down"]), "h": h}
        g, u = g.to(DTYPES[c["kept"]]).float(), u.to(DTYPES[c["kept"]]).float()
        dg, du = (d.to(torch.bfloat16) for d in plain_gated_grads(c["act"], s["dh"], g, u))
        out = {"h": h.to(DTYPES[c["y"]]), "dg": dg, "du": du}
        if c["products"]:
            a = (over(codes[1], 127.0) * codes[0]).to(torch.bfloat16).float()
            out["dx"] = s["gate"]["gamma"] * (dg.float() @ s["gate"]["q"].float()) \
                + s["up"]["gamma"] * (du.float() @ s["up"]["q"].float())
            out["dwg"] = (dg.float().T @ a) * s["gate"]["inside"]
            out["dwu"] = (du.float().T @ a) * s["up"]["inside"]
        return out
    # every adapter for every token, and of those the token's own
    A, R = c["A"], c["R"]
    down, up = s["down"].float().view(A * R, -1), s["up"].float().view(A * R, -1)
    mine = (s["rows"].view(-1, 1) == torch.arange(A, device=x.device)).float()
    mine, scaled = mine.repeat_interleave(R, dim=1), (mine * s["scales"]).repeat_interleave(R, dim=1)
    y = plain_product(plain_codes(x), s["base"])
    drop = op == "adapter_step" and c["p"] > 0.0
    xd = plain_dropout(x, c["p"], s["seed"]).to(s["x"].dtype).float() if drop else x
    low = xd @ down.T
    y = y + (low * scaled) @ up
    if op == "adapted":
        return y
    dy = s["dy"].float()
    v = (dy @ up.T) * scaled
    dxd = v @ down
    if drop:
        dxd = plain_dropout(dxd, c["p"], s["seed"])
    return {"y": y, "t": (low * mine).view(-1, A, R).sum(dim=1),
            "dx": s["base"]["gamma"] * (dy @ s["base"]["q"].float()) + dxd,
            "ddown": (v.T @ xd).view(A, R, -1), "dup": ((low * scaled).T @ dy).view(A, R, -1)}


def work(case):
    """Each input read and each output written once.  A training step's backward comes after the
    rest of the network's passes, so what it needs of the forward is written and read again."""
    c, op, M = case, case["op"], case["M"]
    if op == "dropout":
        n = M * c["K"]
        return {"bytes": n * (BYTES[c["x"]] * (2 if c["residual"] else 1) + BYTES[c["y"]]), "flops": 2 * n}
    if op in ("gated", "block", "gated_step"):
        D, F = c["D"], c["F"]
        b, f = M * D * BYTES[c["x"]] + 2 * F * padded(D) / 4, 4.0 * M * D * F
        if op == "block":
            return {"bytes": b + D * padded(F) / 4 + 4.0 * M * (F + D), "flops": f + 2.0 * M * D * F}
        b += M * F * BYTES[c["y"]]
        if op == "gated_step":
            # g and u out and back, dh in, dg and du out
            b += M * F * (4 * BYTES[c["kept"]] + 4 + 4)
            f += 10 * M * F
            if c["products"]:
                # dg and du back, codes out and back, the weights again, dx, both dW with their masks
                b += M * F * 4 + 2 * M * padded(D) + 2 * D * padded(F) / 4 + 4.0 * M * D + 2 * F * D * (4 + 1 / 8)
                f += 8.0 * M * D * F
        return {"bytes": b, "flops": f}
    K, N, R = c["K"], c["N"], c["R"]
    used = min(c["A"], c["requests"])
    w = used * R * (K + N) * BYTES[c["w"]]
    b = M * K * BYTES[c["x"]] + N * padded(K) / 4 + w + 4.0 * M * N + 4 * M
    f = 2.0 * M * K * N + 2.0 * M * R * (K + N)
    if op == "adapter_step":
        # x (its dropped form follows from it) and t again, dy, both weights again, dx and the gradients
        b += M * K * BYTES[c["x"]] + 8.0 * M * R + 2 * M * N + K * padded(N) / 4 + w + 4.0 * M * K \
            + c["A"] * R * (K + N) * 4
        f += 2.0 * M * K * N + 4.0 * M * R * (K + N)
    return {"bytes": b, "flops": f}


# ---- 64 bits ----------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    c, op, M = case, case["op"], case["M"]
    f32 = lambda v: v.to(torch.float32).double()  # noqa: E731  a rounding that the definition has
    x = s["x"].double()

    def codes_of(v):  # v: float32 numbers
        top = v.abs().max(dim=1).values[:, None]
        per = f32(127.0 / f32(top + float(torch.tensor(EPS, dtype=torch.float32))))
        return f32(v * per).round().clamp(-128, 127), top

    def product(cd, w, rounded=False):
        gamma = w["gamma"].double()
        acc = torch.mm(cd[0], w["q"].t().double())
        return f32(acc * f32(f32(gamma * cd[1]) / 127.0)) if rounded else acc.mul_(gamma * cd[1] / 127.0)

    def kept_words(shape, sd, offset):
        n, low = shape[0] * shape[1], (1 << 32) - 1
        at = torch.arange((n + 3) // 4, device=x.device)
        w0, w1, w2, w3 = at % (1 << 32), at // (1 << 32), at * 0 + offset % (1 << 32), at * 0 + offset // (1 << 32)
        key = [sd % (1 << 32), sd // (1 << 32)]
        for r in range(10):
            ka, kb = (key[0] + r * 0x9E3779B9) & low, (key[1] + r * 0xBB67AE85) & low
            # products in two halves of the second factor
            p0, p1 = 0xD2511F53 * (w0 & 0xffff), 0xD2511F53 * (w0 >> 16)
            r0, r1 = 0xCD9E8D57 * (w2 & 0xffff), 0xCD9E8D57 * (w2 >> 16)
            m0, n0 = p1 + (p0 >> 16), r1 + (r0 >> 16)
            w0, w1, w2, w3 = (n0 >> 16) ^ w1 ^ ka, (n0 << 16 | r0 & 0xffff) & low, \
                (m0 >> 16) ^ w3 ^ kb, (m0 << 16 | p0 & 0xffff) & low
        return torch.stack([w0, w1, w2, w3], dim=-1).flatten()[:n].reshape(shape)

    def dropped(v, p, sd, offset=0):
        by = float(torch.tensor(1.0 / (1.0 - p), dtype=torch.float32))
        return (v * by).masked_fill(kept_words(v.shape, sd, offset) < int(p * (1 << 32) + 0.5), 0.0)

    if op == "dropout":
        y = dropped(x, c["p"], s["seed"], s["offset"])
        return y if s["residual"] is None else y + s["residual"].double()
    if op in ("gated", "block", "gated_step"):
        cd = codes_of(x)
        del x
        if op == "gated":
            g = product(cd, s["gate"])
            g = g.clamp_(min=0).square_() if c["act"] == "relu2" else g.mul_(torch.sigmoid(g))
            return g.mul_(product(cd, s["up"]))
        g, u = product(cd, s["gate"], True), product(cd, s["up"], True)
        if op == "block":
            h = f32(f32(g.clamp(min=0).square()) * u)
            return {"y": product(codes_of(h), s["down"]), "h": h}
        h = (g.clamp(min=0).square() if c["act"] == "relu2" else g * torch.sigmoid(g)) * u
        g, u = (v.to(DTYPES[c["kept"]]).double() for v in (g, u))
        dh = s["dh"].double()
        if c["act"] == "silu":
            sg = torch.sigmoid(g)
            return {"h": h, "dg": dh * u * sg * (1.0 + g * (1.0 - sg)), "du": dh * g * sg}
        r = g.clamp(min=0)
        dg = f32(dh * f32(u * (2.0 * r))).to(torch.bfloat16).double()
        du = f32(dh * f32(r.square())).to(torch.bfloat16).double()
        out = {"h": h, "dg": dg, "du": du}
        if c["products"]:
            a = f32(f32(cd[1] / 127.0) * cd[0]).to(torch.bfloat16).double()
            dx = torch.mm(dg, s["gate"]["q"].double()) * s["gate"]["gamma"].double()
            out["dx"] = dx.add_(torch.mm(du, s["up"]["q"].double()) * s["up"]["gamma"].double())
            out["dwg"] = torch.mm(dg.t(), a).masked_fill_(~s["gate"]["inside"], 0.0)
            out["dwu"] = torch.mm(du.t(), a).masked_fill_(~s["up"]["inside"], 0.0)
        return out
    y = product(codes_of(x), s["base"])
    step = op == "adapter_step"
    xd = dropped(x, c["p"], s["seed"]).to(s["x"].dtype).double() if step and c["p"] > 0.0 else x
    if step:
        dy = s["dy"].double()
        low, dxd = torch.zeros((M, c["R"]), dtype=torch.float64, device=x.device), torch.zeros_like(x)
        ddown, dup = torch.zeros_like(s["down"], dtype=torch.float64), torch.zeros_like(s["up"], dtype=torch.float64)
    for a in range(c["A"]):
        at = (s["rows"] == a).nonzero().view(-1)
        if at.numel() == 0:
            continue
        dn, upw, sc = s["down"][a].double(), s["up"][a].double(), float(s["scales"][a])
        lo = torch.mm(xd[at], dn.t())
        y[at] += sc * torch.mm(lo, upw)
        if step:
            low[at] = lo
            v = sc * torch.mm(dy[at], upw.t())
            dxd[at] = torch.mm(v, dn)
            ddown[a], dup[a] = torch.mm(v.t(), xd[at]), sc * torch.mm(lo.t(), dy[at])
    if not step:
        return y
    if c["p"] > 0.0:
        dxd = dropped(dxd, c["p"], s["seed"])
    dx = torch.mm(dy, s["base"]["q"].double()) * s["base"]["gamma"].double() + dxd
    return {"y": y, "t": low, "dx": dx, "ddown": ddown, "dup": dup}
