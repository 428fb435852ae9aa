"""The operators around BitLinear in a BitNet block, as they are measured.

A pre-norm BitNet block runs  LayerNorm -> BitLinear (up) -> ReLU^2 ->
(sub-LayerNorm ->) BitLinear (down).  The cases here are what lies between the
ternary products: layer norm's forward, a training step's forward and backward
of layer norm and of ReLU^2 with the activation kept in 8 bits between the two,
and the 8-bit save and restore on their own.  Shapes are those of the
framework's workloads (d_model 2048 -> FFN 5632, 4096 -> 11008, 8192 -> 28672)
and odd ones of the same range.

Formulas (m: token row, k: column, K columns):

  mean = sum_k x / K     var = sum_k (x - mean)^2 / K    rstd = 1 / sqrt(var + eps)
  y    = (x - mean) rstd w + b
  dx   = rstd (g - sum_k g / K - xhat sum_k (g xhat) / K)    xhat = (x - mean) rstd, g = dy w
  dw   = sum_m dy xhat     db = sum_m dy
  a    = max(h, 0)^2       dh = da 2 max(h, 0)

8-bit saved activations: groups of 64 consecutive columns of a row (the last
one may be shorter), amax the largest magnitude in the group, all in float32:
  scale = fp32(amax fp32(1 / 127))    s = fp32(127 / amax)
  code  = the integer nearest x s (the exact product, ties to even)
  x~    = fp32(scale code)
"""
import math

import torch

own = False

EPS = 1e-5
GROUP = 64
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "bf16": 2}


def listed():
    return [
        # one token's norm in front of the d_model-2048 projection: latency alone
        {"name": "norm 1x2048 bf16", "op": "norm", "M": 1, "K": 2048, "x": "bf16", "y": "bf16"},
        # sub-norm of a decode batch's FFN hidden layer, which the framework forms in float32
        {"name": "norm 8x5632 f32", "op": "norm", "M": 8, "K": 5632, "x": "f32", "y": "f32"},
        # prefill, 7B-like model
        {"name": "norm 2048x4096 bf16", "op": "norm", "M": 2048, "K": 4096, "x": "bf16", "y": "bf16"},
        # a ragged batch of an odd-width model, float32 in, bfloat16 out
        {"name": "norm 777x1003 f32 to bf16", "op": "norm", "M": 777, "K": 1003, "x": "f32", "y": "bf16"},
        # training, 7B-like: 8-bit saved input, dY as the BitLinear backward writes it (float32)
        {"name": "norm step saved 2048x4096", "op": "norm_step", "M": 2048, "K": 4096, "x": "bf16", "y": "bf16",
         "dy": "f32", "dx": "bf16", "saved": True},
        # training, 70B-like width
        {"name": "norm step saved 8192x8192", "op": "norm_step", "M": 8192, "K": 8192, "x": "bf16", "y": "bf16",
         "dy": "f32", "dx": "bf16", "saved": True},
        # training, the sub-norm over a 7B-like FFN hidden layer, its input kept whole
        {"name": "norm step kept 2048x11008 f32", "op": "norm_step", "M": 2048, "K": 11008, "x": "f32", "y": "f32",
         "dy": "f32", "dx": "f32", "saved": False},
        # training on a short ragged batch, odd width
        {"name": "norm step saved 333x1001", "op": "norm_step", "M": 333, "K": 1001, "x": "f32", "y": "bf16",
         "dy": "bf16", "dx": "f32", "saved": True},
        # a residual stream put by and taken back, 7B-like
        {"name": "save restore 2048x4096 bf16", "op": "save", "M": 2048, "K": 4096, "x": "bf16"},
        # an odd-width float32 hidden layer
        {"name": "save restore 1999x5633 f32", "op": "save", "M": 1999, "K": 5633, "x": "f32"},
        # ReLU^2 of a training step, 7B-like FFN; dH in bfloat16 is what the BitLinear backward takes
        {"name": "relu2 step saved 2048x11008", "op": "relu2_step", "M": 2048, "K": 11008, "x": "f32", "y": "f32",
         "dy": "f32", "dx": "bf16", "saved": True},
        # the same, 70B-like FFN: the largest array
        {"name": "relu2 step saved 8192x28672", "op": "relu2_step", "M": 8192, "K": 28672, "x": "f32", "y": "f32",
         "dy": "f32", "dx": "bf16", "saved": True},
    ]


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_step", "norm_step", "save", "relu2_step"])
    K = int(round(math.exp(rng.uniform(math.log(64), math.log(28672)))))
    if rng.random() < 0.5:
        K = max(64, K // 64 * 64)  # half of the widths as models choose them, half as they fall
    M = int(round(math.exp(rng.uniform(0.0, math.log(8192)))))
    M = max(1, min(M, 8192 * 8192 // K))
    t = lambda: rng.choice(["f32", "bf16"])  # noqa: E731
    case = {"op": op, "M": M, "K": K, "x": t()}
    if op != "save":
        case["y"] = t()
    if op.endswith("step"):
        case.update(dy=t(), dx=t(), saved=rng.random() < 0.6)
    return case


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed))
    M, K = case["M"], case["K"]
    x = torch.randn((M, K), generator=g, device=dev)
    if case["op"] != "relu2_step":
        # a residual stream: some channels 20 times the others, each with an offset of its own
        loud = torch.rand((K,), generator=g, device=dev) < 0.01
        x = x * torch.where(loud, 20.0, 1.0) + 0.25 * torch.randn((K,), generator=g, device=dev)
    s = {"case": dict(case), "x": x.to(DTYPES[case["x"]])}
    if case["op"].startswith("norm"):
        s["w"] = 1.0 + 0.1 * torch.randn((K,), generator=g, device=dev)
        s["b"] = 0.1 * torch.randn((K,), generator=g, device=dev)
    if case["op"].endswith("step"):
        s["dy"] = (1e-3 * torch.randn((M, K), generator=g, device=dev)).to(DTYPES[case["dy"]])
    return s


def run(state):
    return run_own(state) if own else run_plain(state)


def run_own(s):
    import bitlinear_absmean_ternarise_bit_amd as bl
    c, x = s["case"], s["x"]
    if c["op"] == "norm":
        return bl.layer_norm(x, s["w"], s["b"], EPS, out_dtype=DTYPES[c["y"]])
    if c["op"] == "norm_step":
        if c["saved"]:
            y, mean, rstd, kept = bl.layer_norm(x, s["w"], s["b"], EPS, out_dtype=DTYPES[c["y"]], save=True)
        else:
            y, mean, rstd = bl.layer_norm(x, s["w"], s["b"], EPS, out_dtype=DTYPES[c["y"]], return_stats=True)
            kept = x
        dx, dw, db = bl.layer_norm_backward(s["dy"], kept, mean, rstd, s["w"], out_dtype=DTYPES[c["dx"]])
        return {"y": y, "mean": mean, "rstd": rstd, "dx": dx, "dw": dw, "db": db}
    if c["op"] == "save":
        return bl.restore_activations(bl.save_activations(x), c["K"], dtype=DTYPES[c["x"]])
    if c["saved"]:
        a, kept = bl.relu2(x, out_dtype=DTYPES[c["y"]], save=True)
    else:
        a, kept = bl.relu2(x, out_dtype=DTYPES[c["y"]]), x
    return {"a": a, "dh": bl.relu2_backward(s["dy"], kept, out_dtype=DTYPES[c["dx"]])}


def plain_saved(x):
    """x~: what the 8-bit codes and scales of x (float32) stand for."""
    M, K = x.shape
    pad = -K % GROUP
    if pad:
        x = torch.cat([x, x.new_zeros((M, pad))], dim=1)
    v = x.view(M, -1, GROUP)
    amax = v.abs().amax(dim=2, keepdim=True)
    s = torch.where(amax > 0, torch.full_like(amax, 127.0) / amax, torch.zeros_like(amax))  # one rounded division
    codes = torch.round(v.double() * s.double()).to(torch.int8)  # 64 bits: products next to a half
    return (codes.float() * (amax * (1.0 / 127.0))).view(M, -1)[:, :K]


def run_plain(s):
    c = s["case"]
    x = s["x"].float()
    if c["op"] == "save":
        return plain_saved(x).to(DTYPES[c["x"]])
    if c["op"] == "relu2_step":
        r = torch.where(x > 0, x, torch.zeros_like(x))
        a = (r * r).to(DTYPES[c["y"]])
        kept = plain_saved(x) if c["saved"] else x
        dh = s["dy"].float() * (2.0 * torch.where(kept > 0, kept, torch.zeros_like(kept)))
        return {"a": a, "dh": dh.to(DTYPES[c["dx"]])}
    K = c["K"]
    mean = x.sum(dim=1, keepdim=True) / K
    d = x - mean
    rstd = 1.0 / torch.sqrt((d * d).sum(dim=1, keepdim=True) / K + EPS)
    y = (d * rstd * s["w"] + s["b"]).to(DTYPES[c["y"]])
    if c["op"] == "norm":
        return y
    xhat = ((plain_saved(x) if c["saved"] else x) - mean) * rstd
    dy = s["dy"].float()
    g = dy * s["w"]
    dx = rstd * (g - g.sum(dim=1, keepdim=True) / K - xhat * ((g * xhat).sum(dim=1, keepdim=True) / K))
    return {"y": y, "mean": mean.view(-1), "rstd": rstd.view(-1), "dx": dx.to(DTYPES[c["dx"]]),
            "dw": (dy * xhat).sum(dim=0), "db": dy.sum(dim=0)}


def work(case):
    """Each input read and each output written once.  A step's backward comes
    after the rest of the network's passes, so what it needs of x is written
    and read as 8-bit codes with a float32 scale for each 64, or read again."""
    M, K, op = case["M"], case["K"], case["op"]
    n = M * K
    kept = 1.0 + 4.0 / GROUP  # bytes of a saved value
    b = n * BYTES[case["x"]]
    if op == "save":
        return {"bytes": b * 2 + 2 * kept * n, "flops": 6 * n}
    b += n * BYTES[case["y"]]
    if op == "norm":
        return {"bytes": b + 8 * K, "flops": 8 * n}
    b += n * (BYTES[case["dy"]] + BYTES[case["dx"]])
    b += n * (2 * kept if case["saved"] else BYTES[case["x"]])
    if op == "relu2_step":
        return {"bytes": b, "flops": 5 * n}
    # weight and bias forward, weight backward, their gradients; mean and rstd out and back
    return {"bytes": b + 20 * K + 16 * M, "flops": 22 * n}


def exact(case, seed):
    s = prepare(case, seed)
    M, K, op = case["M"], case["K"], case["op"]
    x64 = s["x"].to(torch.float64)

    def through_8_bits():
        out = torch.empty_like(x64)
        inv127 = float(torch.tensor(1.0 / 127.0, dtype=torch.float32))
        whole = K // GROUP * GROUP
        for lo, hi, width in ((0, whole, GROUP), (whole, K, K - whole)):
            if lo == hi:
                continue
            part = x64[:, lo:hi].reshape(M, (hi - lo) // width, width)
            top = part.abs().max(dim=2).values.unsqueeze(2)
            # scale and s are float32 numbers by definition
            s32 = torch.where(top > 0, torch.full_like(top, 127.0).div(top).to(torch.float32).double(), 0.0)
            scale = (top * inv127).to(torch.float32).double()
            out[:, lo:hi] = ((part * s32).round() * scale).reshape(M, hi - lo)
        return out

    if op == "save":
        return through_8_bits()
    if op == "relu2_step":
        h = through_8_bits() if case["saved"] else x64
        return {"a": x64.clamp(min=0.0).square(), "dh": s["dy"].double().mul_(2.0).mul_(h.clamp_(min=0.0))}
    mean = x64.mean(dim=1)
    rstd = (x64.var(dim=1, unbiased=False) + EPS).rsqrt()
    w = s["w"].double()
    y = torch.addcmul(s["b"].double(), (x64 - mean[:, None]) * rstd[:, None], w)
    if op == "norm":
        return y
    xhat = ((through_8_bits() if case["saved"] else x64) - mean[:, None]) * rstd[:, None]
    dy = s["dy"].double()
    dw, db = (dy * xhat).sum(dim=0), dy.sum(dim=0)
    g = dy.mul_(w)
    c1, c2 = g.mean(dim=1), (g * xhat).mean(dim=1)
    dx = (g - c1[:, None] - xhat * c2[:, None]) * rstd[:, None]
    return {"y": y, "mean": mean, "rstd": rstd, "dx": dx, "dw": dw, "db": db}
