"""BitNet b1.58 BitLinear forward on MI355X (gfx950).

A thin torch-facing binding over the C ABI in ``include/bitlinear.h``,
``bitlinear_block.h``, ``bitlinear_gated.h`` and ``bitlinear_adapters.h``: these functions
only check and marshal arguments (device pointers, sizes, the current HIP stream); every step of the computation runs in the HIP kernels of
``libbitlinear.so``.  There is no CPU fallback: without the built library or a
GPU the calls raise.

    packed, gamma = quantize_weights(W)           # W: float32 [N, K] on the GPU
    Y = forward(X, packed, gamma, K)              # X: float32/bfloat16 [M, K] -> float32 [M, N]
"""
from __future__ import annotations

from . import abi
from .abi import BitLinearError

__all__ = [
    "BitLinearError",
    "padded_k",
    "packed_words",
    "quantize_weights",
    "quantize_activations",
    "forward",
    "forward_batched",
    "forward_quantized",
    "forward_noalloc",
    "max_decode_m",
    "decode_fits",
    "ffn_forward",
    "pack_transposed",
    "backward",
    "r3_padded_k",
    "r3_row_bytes",
    "r3_decode_fits",
    "quantize_weights_r3",
    "forward_r3",
    "save_activations",
    "restore_activations",
    "layer_norm",
    "layer_norm_backward",
    "relu2",
    "relu2_backward",
    "gated_forward",
    "gated_ffn_forward",
    "gated_backward",
    "gated_input_backward",
    "adapters_forward",
    "adapted_forward",
    "adapters_backward",
    "dropout",
]


def _torch():
    import torch
    return torch


def _stream(t):
    torch = _torch()
    return ctypes_void(torch.cuda.current_stream(t.device).cuda_stream)


def ctypes_void(v):
    import ctypes
    return ctypes.c_void_p(v)


def _ptr(t):
    import ctypes
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _require_cuda(t, name):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def padded_k(K: int) -> int:
    return int(abi.load().bitlinear_padded_k(K))


def packed_words(K: int) -> int:
    """uint32 words per packed row."""
    return padded_k(K) // 16


def max_decode_m() -> int:
    return int(abi.load().bitlinear_max_decode_m())


def decode_fits(M: int, K: int, N: int) -> bool:
    """Whether the decode kernel takes an M x K activation against N weight rows."""
    lib = abi.load()
    return (M <= lib.bitlinear_max_decode_m()
            and M * (padded_k(K) + 16) <= lib.bitlinear_max_decode_codes()
            and M * N < (1 << 29))


def _x_dtype(X):
    torch = _torch()
    if X.dtype == torch.float32:
        return abi.F32
    if X.dtype == torch.bfloat16:
        return abi.BF16
    raise ValueError("X must be float32 or bfloat16")


def quantize_weights(W, out_packed=None, out_gamma=None, workspace=None):
    """AbsMean ternarisation + 2-bit packing of a float32 [N, K] GPU tensor.

    Returns (packed int32 [N, padded_k(K) // 16] holding uint32 words, gamma float32 [1]);
    ``out_packed`` / ``out_gamma`` / ``workspace`` may be given to avoid allocations.
    """
    torch = _torch()
    _require_cuda(W, "W")
    if W.dtype != torch.float32 or W.dim() != 2:
        raise ValueError("W must be a float32 [N, K] tensor")
    lib = abi.load()
    N, K = W.shape
    packed = out_packed if out_packed is not None else torch.empty(
        (N, packed_words(K)), dtype=torch.int32, device=W.device)
    gamma = out_gamma if out_gamma is not None else torch.empty((1,), dtype=torch.float32,
                                                                device=W.device)
    if packed.shape != (N, packed_words(K)) or packed.element_size() != 4 or gamma.numel() < 1:
        raise ValueError("output buffers have the wrong shape")
    _require_cuda(packed, "out_packed")
    if workspace is not None:
        _require_cuda(workspace, "workspace")
        ws = workspace
        ws_bytes = workspace.numel() * workspace.element_size()
    else:
        ws_bytes = lib.bitlinear_quantize_workspace_bytes()
        ws = torch.empty((ws_bytes,), dtype=torch.uint8, device=W.device)
    abi.check("bitlinear_quantize_weights",
              lib.bitlinear_quantize_weights(_ptr(W), N, K, _ptr(packed), _ptr(gamma), _ptr(ws),
                                             ws_bytes, _stream(W)))
    return packed, gamma


def quantize_activations(X):
    """Per-token AbsMax INT8 codes: (Xq int8 [M, padded_k(K)], gamma_a float32 [M], rowsum int32 [M])."""
    torch = _torch()
    _require_cuda(X, "X")
    if X.dim() != 2:
        raise ValueError("X must be [M, K]")
    lib = abi.load()
    M, K = X.shape
    Xq = torch.empty((M, padded_k(K)), dtype=torch.int8, device=X.device)
    ga = torch.empty((M,), dtype=torch.float32, device=X.device)
    rs = torch.empty((M,), dtype=torch.int32, device=X.device)
    abi.check("bitlinear_quantize_activations",
              lib.bitlinear_quantize_activations(_ptr(X), _x_dtype(X), M, K, _ptr(Xq), _ptr(ga),
                                                 _ptr(rs), _stream(X)))
    return Xq, ga, rs


_PATHS = {"auto": abi.PATH_AUTO, "decode": abi.PATH_DECODE, "prefill": abi.PATH_PREFILL}


def forward(X, packed, gamma, K: int | None = None, path: str = "auto", return_acc: bool = False,
            out=None, workspace=None):
    """Y = dequant(A_q x W_q^T) for X [M, K] (float32 or bfloat16) -> float32 [M, N].

    ``path`` forces the decode or prefill kernels; ``return_acc`` also returns
    the exact INT32 accumulator [M, N].
    """
    torch = _torch()
    _require_cuda(X, "X")
    _require_cuda(packed, "packed")
    _require_cuda(gamma, "gamma")
    if X.dim() != 2 or packed.dim() != 2:
        raise ValueError("X must be [M, K] and packed [N, words]")
    M, Kx = X.shape
    K = Kx if K is None else K
    if K != Kx:
        raise ValueError("K does not match X")
    N = packed.shape[0]
    if packed.shape[1] != packed_words(K) or packed.element_size() != 4:
        raise ValueError("packed does not hold padded_k(K) // 16 32-bit words per row")
    lib = abi.load()
    Y = out if out is not None else torch.empty((M, N), dtype=torch.float32, device=X.device)
    acc = torch.empty((M, N), dtype=torch.int32, device=X.device) if return_acc else None
    ws_bytes = 0
    ws = workspace
    if ws is None and not (path == "decode" or (path == "auto" and decode_fits(M, K, N))):
        ws_bytes = lib.bitlinear_forward_workspace_bytes(M, K)
        ws = torch.empty((ws_bytes,), dtype=torch.uint8, device=X.device)
    elif ws is not None:
        ws_bytes = ws.numel() * ws.element_size()
    abi.check("bitlinear_forward_ex",
              lib.bitlinear_forward_ex(_ptr(X), _x_dtype(X), M, K, _ptr(packed), N, _ptr(gamma),
                                       _ptr(Y), _ptr(acc), _PATHS[path], _ptr(ws), ws_bytes,
                                       _stream(X)))
    return (Y, acc) if return_acc else Y


def forward_noalloc(X, packed, gamma, K: int | None = None, out=None):
    """bitlinear_forward_noalloc: the same forward with the library's own
    per-GPU scratch array as the prefill workspace (the C call allocates
    nothing; pass ``out`` to allocate nothing here either).  Calls that overlap
    on one GPU share that array and must be serialised."""
    torch = _torch()
    _require_cuda(X, "X")
    _require_cuda(packed, "packed")
    _require_cuda(gamma, "gamma")
    if X.dim() != 2 or packed.dim() != 2:
        raise ValueError("X must be [M, K] and packed [N, words]")
    M, Kx = X.shape
    K = Kx if K is None else K
    if K != Kx:
        raise ValueError("K does not match X")
    N = packed.shape[0]
    if packed.shape[1] != packed_words(K) or packed.element_size() != 4:
        raise ValueError("packed does not hold padded_k(K) // 16 32-bit words per row")
    Y = out if out is not None else torch.empty((M, N), dtype=torch.float32, device=X.device)
    if Y.shape != (M, N) or Y.dtype != torch.float32:
        raise ValueError("out must be float32 [M, N]")
    _require_cuda(Y, "out")
    lib = abi.load()
    abi.check("bitlinear_forward_noalloc",
              lib.bitlinear_forward_noalloc(_ptr(X), _x_dtype(X), M, K, _ptr(packed), N, _ptr(gamma),
                                            _ptr(Y), _stream(X)))
    return Y


def forward_quantized(Xq, gamma_a, rowsum, packed, gamma, K: int, return_acc: bool = False, out=None):
    """Contraction + rescale from activation codes (as quantize_activations returns them)."""
    torch = _torch()
    for t, nm in ((Xq, "Xq"), (gamma_a, "gamma_a"), (rowsum, "rowsum"), (packed, "packed"),
                  (gamma, "gamma")):
        _require_cuda(t, nm)
    M = Xq.shape[0]
    if Xq.dtype != torch.int8 or Xq.shape[1] != padded_k(K):
        raise ValueError("Xq must be int8 [M, padded_k(K)]")
    N = packed.shape[0]
    if packed.shape[1] != packed_words(K):
        raise ValueError("packed does not hold padded_k(K) // 16 words per row")
    lib = abi.load()
    Y = out if out is not None else torch.empty((M, N), dtype=torch.float32, device=Xq.device)
    acc = torch.empty((M, N), dtype=torch.int32, device=Xq.device) if return_acc else None
    abi.check("bitlinear_forward_quantized",
              lib.bitlinear_forward_quantized(_ptr(Xq), _ptr(gamma_a), _ptr(rowsum), M, K,
                                              _ptr(packed), N, _ptr(gamma), _ptr(Y), _ptr(acc),
                                              _stream(Xq)))
    return (Y, acc) if return_acc else Y


def forward_batched(X, packed, gamma, K: int | None = None, out=None):
    """L decode forwards in one launch: X [L, M, K], packed [L, N, words], gamma [L] -> Y [L, M, N]."""
    torch = _torch()
    for t, nm in ((X, "X"), (packed, "packed"), (gamma, "gamma")):
        _require_cuda(t, nm)
    if X.dim() != 3 or packed.dim() != 3:
        raise ValueError("X must be [L, M, K] and packed [L, N, words]")
    L, M, Kx = X.shape
    K = Kx if K is None else K
    if K != Kx or packed.shape[0] != L or gamma.numel() != L:
        raise ValueError("inconsistent batched shapes")
    N = packed.shape[1]
    if packed.shape[2] != packed_words(K):
        raise ValueError("packed does not hold padded_k(K) // 16 words per row")
    lib = abi.load()
    Y = out if out is not None else torch.empty((L, M, N), dtype=torch.float32, device=X.device)
    abi.check("bitlinear_forward_batched",
              lib.bitlinear_forward_batched(L, _ptr(X), _x_dtype(X), M, K, _ptr(packed), N,
                                            _ptr(gamma), _ptr(Y), _stream(X)))
    return Y


# ---- radix-3 weights (five per byte) --------------------------------------

def r3_padded_k(K: int) -> int:
    return int(abi.load().bitlinear_r3_padded_k(K))


def r3_row_bytes(K: int) -> int:
    """Bytes per radix-3 packed row."""
    return r3_padded_k(K) // 5


def r3_decode_fits(M: int, K: int, N: int) -> bool:
    lib = abi.load()
    return (M <= lib.bitlinear_max_decode_m()
            and M * (r3_padded_k(K) + 16) <= lib.bitlinear_max_decode_codes()
            and M * N < (1 << 29))


def quantize_weights_r3(W, out_packed=None, out_gamma=None, workspace=None):
    """AbsMean ternarisation of a float32 [N, K] GPU tensor, packed five weights per byte.

    Returns (packed uint8 [N, r3_row_bytes(K)], gamma float32 [1]); gamma and the
    ternary codes are bit-identical to :func:`quantize_weights`.
    """
    torch = _torch()
    _require_cuda(W, "W")
    if W.dtype != torch.float32 or W.dim() != 2:
        raise ValueError("W must be a float32 [N, K] tensor")
    lib = abi.load()
    N, K = W.shape
    packed = out_packed if out_packed is not None else torch.empty(
        (N, r3_row_bytes(K)), dtype=torch.uint8, device=W.device)
    gamma = out_gamma if out_gamma is not None else torch.empty((1,), dtype=torch.float32,
                                                                device=W.device)
    if packed.shape != (N, r3_row_bytes(K)) or packed.element_size() != 1 or gamma.numel() < 1:
        raise ValueError("output buffers have the wrong shape")
    _require_cuda(packed, "out_packed")
    if workspace is not None:
        _require_cuda(workspace, "workspace")
        ws = workspace
        ws_bytes = workspace.numel() * workspace.element_size()
    else:
        ws_bytes = lib.bitlinear_quantize_workspace_bytes()
        ws = torch.empty((ws_bytes,), dtype=torch.uint8, device=W.device)
    abi.check("bitlinear_quantize_weights_r3",
              lib.bitlinear_quantize_weights_r3(_ptr(W), N, K, _ptr(packed), _ptr(gamma), _ptr(ws),
                                                ws_bytes, _stream(W)))
    return packed, gamma


def forward_r3(X, packed, gamma, K: int | None = None, return_acc: bool = False, out=None):
    """Decode forward over radix-3 weights.

    X [M, K] with packed [N, r3_row_bytes(K)] and gamma [1], or X [L, M, K] with
    packed [L, N, r3_row_bytes(K)] and gamma [L] (L layers in one launch).
    Returns Y float32 [M, N] / [L, M, N] (and the INT32 accumulators if asked).
    """
    torch = _torch()
    for t, nm in ((X, "X"), (packed, "packed"), (gamma, "gamma")):
        _require_cuda(t, nm)
    batched = X.dim() == 3
    if batched:
        if packed.dim() != 3:
            raise ValueError("X [L, M, K] needs packed [L, N, bytes]")
        L, M, Kx = X.shape
        N = packed.shape[1]
        if packed.shape[0] != L or gamma.numel() != L:
            raise ValueError("inconsistent batched shapes")
    else:
        if X.dim() != 2 or packed.dim() != 2:
            raise ValueError("X must be [M, K] and packed [N, bytes]")
        L = 1
        M, Kx = X.shape
        N = packed.shape[0]
    K = Kx if K is None else K
    if K != Kx:
        raise ValueError("K does not match X")
    if packed.shape[-1] != r3_row_bytes(K) or packed.element_size() != 1:
        raise ValueError("packed does not hold r3_row_bytes(K) bytes per row")
    lib = abi.load()
    shape = (L, M, N) if batched else (M, N)
    Y = out if out is not None else torch.empty(shape, dtype=torch.float32, device=X.device)
    acc = torch.empty(shape, dtype=torch.int32, device=X.device) if return_acc else None
    abi.check("bitlinear_forward_r3",
              lib.bitlinear_forward_r3(L, _ptr(X), _x_dtype(X), M, K, _ptr(packed), N, _ptr(gamma),
                                       _ptr(Y), _ptr(acc), _stream(X)))
    return (Y, acc) if return_acc else Y


# ---- LUT contraction (comparison variant) ----------------------------------

def lut_workspace_bytes(L: int, M: int, K: int) -> int:
    return int(abi.load().bitlinear_lut_workspace_bytes(L, M, K))


def forward_lut(X, packed, gamma, K: int | None = None, return_acc: bool = False, out=None, workspace=None):
    """Decode forward through 81-entry LUTs over 2-bit weights (a comparison to ``forward``).

    X [M, K] with packed [N, words] and gamma [1], or X [L, M, K] with
    packed [L, N, words] and gamma [L].  Returns Y float32 [M, N] / [L, M, N]
    (and the INT32 accumulators if asked).
    """
    torch = _torch()
    for t, nm in ((X, "X"), (packed, "packed"), (gamma, "gamma")):
        _require_cuda(t, nm)
    batched = X.dim() == 3
    if batched:
        if packed.dim() != 3:
            raise ValueError("X [L, M, K] needs packed [L, N, words]")
        L, M, Kx = X.shape
        N = packed.shape[1]
        if packed.shape[0] != L or gamma.numel() != L:
            raise ValueError("inconsistent batched shapes")
    else:
        if X.dim() != 2 or packed.dim() != 2:
            raise ValueError("X must be [M, K] and packed [N, words]")
        L = 1
        M, Kx = X.shape
        N = packed.shape[0]
    K = Kx if K is None else K
    if K != Kx:
        raise ValueError("K does not match X")
    if packed.shape[-1] != packed_words(K):
        raise ValueError("packed does not hold padded_k(K) // 16 words per row")
    lib = abi.load()
    ws_bytes = int(lib.bitlinear_lut_workspace_bytes(L, M, K))
    if workspace is None:
        workspace = torch.empty((max(ws_bytes, 1),), dtype=torch.uint8, device=X.device)
    shape = (L, M, N) if batched else (M, N)
    Y = out if out is not None else torch.empty(shape, dtype=torch.float32, device=X.device)
    acc = torch.empty(shape, dtype=torch.int32, device=X.device) if return_acc else None
    abi.check("bitlinear_forward_lut",
              lib.bitlinear_forward_lut(L, _ptr(X), _x_dtype(X), M, K, _ptr(packed), N, _ptr(gamma),
                                        _ptr(Y), _ptr(acc), _ptr(workspace),
                                        workspace.numel() * workspace.element_size(), _stream(X)))
    return (Y, acc) if return_acc else Y


# ---- the BitNet FFN block --------------------------------------------------

def ffn_forward(X, up, down, path: str = "auto", return_hidden: bool = False, out=None, workspace=None):
    """Y = BitLinear_down(ReLU^2(BitLinear_up(X))).

    ``up`` = (packed [F, words(D)], gamma [1]) and ``down`` = (packed [D_out, words(F)],
    gamma [1]) as :func:`quantize_weights` returns them, with X [M, D]; or X
    [L, M, D] with packed [L, ...] and gamma [L] for L layers.  Returns Y float32
    [(L,) M, D_out] (and the hidden ReLU^2 activations [(L,) M, F] if asked).
    """
    torch = _torch()
    (pu, gu), (pd, gd) = up, down
    for t, nm in ((X, "X"), (pu, "packed_up"), (gu, "gamma_up"), (pd, "packed_down"), (gd, "gamma_down")):
        _require_cuda(t, nm)
    batched = X.dim() == 3
    if batched:
        L, M, D = X.shape
        F, Do = pu.shape[1], pd.shape[1]
        if pu.dim() != 3 or pd.dim() != 3 or pu.shape[0] != L or pd.shape[0] != L or gu.numel() != L \
                or gd.numel() != L:
            raise ValueError("inconsistent batched shapes")
    else:
        L = 1
        M, D = X.shape
        F, Do = pu.shape[0], pd.shape[0]
    if pu.shape[-1] != packed_words(D) or pd.shape[-1] != packed_words(F):
        raise ValueError("packed weights do not match D and F")
    lib = abi.load()
    shape = (L, M, Do) if batched else (M, Do)
    Y = out if out is not None else torch.empty(shape, dtype=torch.float32, device=X.device)
    hid = torch.empty((L, M, F) if batched else (M, F), dtype=torch.float32, device=X.device) \
        if return_hidden else None
    if workspace is None:
        ws_bytes = lib.bitlinear_ffn_workspace_bytes(L, M, D, F)
        workspace = torch.empty((ws_bytes,), dtype=torch.uint8, device=X.device)
    ws_bytes = workspace.numel() * workspace.element_size()
    abi.check("bitlinear_ffn_forward",
              lib.bitlinear_ffn_forward(L, _ptr(X), _x_dtype(X), M, D, F, Do, _ptr(pu), _ptr(gu), _ptr(pd),
                                        _ptr(gd), _ptr(Y), _ptr(hid), _PATHS[path], _ptr(workspace), ws_bytes,
                                        _stream(X)))
    return (Y, hid) if return_hidden else Y


# ---- backward with the straight-through estimator ---------------------------

def pack_transposed(W, gamma, out=None, mask_out=None):
    """What the backward needs from W (once per weight update): the codes of
    W^T ([K, padded_k(N) // 16] words, for dX) and the range mask (int32
    [N, ceil(K / 32)] bit words, for dW); gamma from quantize_weights(W)."""
    torch = _torch()
    _require_cuda(W, "W")
    _require_cuda(gamma, "gamma")
    N, K = W.shape
    lib = abi.load()
    packedT = out if out is not None else torch.empty((K, packed_words(N)), dtype=torch.int32, device=W.device)
    mask = mask_out if mask_out is not None else torch.empty((N, (K + 31) // 32), dtype=torch.int32,
                                                             device=W.device)
    abi.check("bitlinear_pack_transposed",
              lib.bitlinear_pack_transposed(_ptr(W), N, K, _ptr(gamma), _ptr(packedT), _ptr(mask), _stream(W)))
    return packedT, mask


def backward(dY, packedT, gamma, Xq, gamma_a, mask, K: int, need_dx: bool = True, need_dw: bool = True,
             workspace=None):
    """STE gradients (dX [M, K], dW [N, K], float32) of the forward from dY (bfloat16 [M, N]).

    ``Xq``/``gamma_a``: the forward's activation codes (quantize_activations);
    ``packedT``/``mask``: pack_transposed(W, gamma); K: the weights' columns.
    """
    torch = _torch()
    for t, nm in ((dY, "dY"), (gamma, "gamma")):
        _require_cuda(t, nm)
    if dY.dtype != torch.bfloat16:
        raise ValueError("dY must be bfloat16")
    M, N = dY.shape
    lib = abi.load()
    dX = torch.empty((M, K), dtype=torch.float32, device=dY.device) if need_dx else None
    dW = torch.empty((N, K), dtype=torch.float32, device=dY.device) if need_dw else None
    if workspace is None:
        workspace = torch.empty((lib.bitlinear_backward_workspace_bytes(M, N, K),), dtype=torch.uint8,
                                device=dY.device)
    abi.check("bitlinear_backward",
              lib.bitlinear_backward(_ptr(dY), M, N, K, _ptr(packedT), _ptr(gamma), _ptr(Xq), _ptr(gamma_a),
                                     _ptr(mask), _ptr(dX), _ptr(dW), _ptr(workspace),
                                     workspace.numel() * workspace.element_size(), _stream(dY)))
    return dX, dW


# ---- the operators around BitLinear (include/bitlinear_block.h) -------------
#
# Activations saved in 8 bits are a pair (codes int8 [M, padded_k(K)], scales
# float32 [M, padded_k(K) / 64]).  Every tensor of a call lies on one GPU, which
# need not be the current one; the work goes to that GPU's current stream.
#
# The calls of a decode step last about as long as this file's own work for
# them, so it is kept short: addresses go to ctypes as they are, what is looked
# up once is kept, arrays shaped like another are made like it, and other shapes
# are passed to torch.empty as numbers (0.3 us less than as a tuple).

_BLOCK = None


class _BlockCalls:
    """What every call below needs, looked up once: torch's functions and dtypes and the C functions."""

    def __init__(self):
        torch = _torch()
        lib = abi.load()
        self.bf16, self.i32 = torch.bfloat16, torch.int32
        self.forward_workspace_bytes = lib.bitlinear_forward_workspace_bytes
        self.f32, self.i8, self.empty, self.empty_like = torch.float32, torch.int8, torch.empty, torch.empty_like
        self.plain = {torch.float32: abi.F32, torch.bfloat16: abi.BF16}
        self.on_device = torch.cuda.device
        # the current device and a stream's address without torch's objects for them, where it has that
        self.device_now = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
        self.stream_of = getattr(torch._C, "_cuda_getCurrentRawStream",
                                 lambda index: torch.cuda.current_stream(index).cuda_stream)
        for name in (*abi.BLOCK_SIGNATURES, *abi.GATED_SIGNATURES, *abi.ADAPTER_SIGNATURES):
            setattr(self, name[len("bitlinear_"):], getattr(lib, name))

    def launch(self, fn, device, *args):
        """Calls a C function on `device`'s current stream, with that device current."""
        index = device.index
        if index == self.device_now():
            status = fn(*args, self.stream_of(index))
        else:
            with self.on_device(index):
                status = fn(*args, self.stream_of(index))
        if status:
            abi.check(fn.__name__, status)


def _block():
    global _BLOCK
    if _BLOCK is None:
        _BLOCK = _BlockCalls()
    return _BLOCK


def _plain_dtype(B, dtype, name):
    d = B.plain.get(dtype)
    if d is None:
        raise ValueError(f"{name} must be float32 or bfloat16")
    return d


def _matrix(B, t, name):
    """Checks a contiguous GPU [M, K] tensor; its abi dtype, M and K."""
    if not (t.is_cuda and t.is_contiguous()):
        _require_cuda(t, name)
    shape = t.shape
    if len(shape) != 2 or t.numel() == 0:
        raise ValueError(f"{name} must be [M, K] with at least one value")
    M, K = shape
    return _plain_dtype(B, t.dtype, name), M, K


def _vector(B, t, n, device, name):
    """The address of a float32 tensor of n values on `device` (None: 0)."""
    if t is None:
        return 0
    if not (t.is_cuda and t.is_contiguous()):
        _require_cuda(t, name)
    if t.dtype != B.f32 or t.numel() != n:
        raise ValueError(f"{name} must hold {n} float32 values")
    if t.get_device() != device.index:
        raise ValueError(f"{name} is on another device")
    return t.data_ptr()


def _whole_or_saved(B, x, K, name, M=None):
    """(data address, scales address, abi dtype, M, K, device) of a [M, K] tensor or a saved pair."""
    if not isinstance(x, (tuple, list)):
        dt, m, k = _matrix(B, x, name)
        if (K is not None and k != K) or (M is not None and m != M):
            raise ValueError(f"{name} does not have the other arrays' shape")
        return x.data_ptr(), 0, dt, m, k, x.device
    codes, scales = x
    if K is None:
        raise ValueError(f"K is needed where {name} is saved in 8 bits")
    _require_cuda(codes, name + " codes")
    _require_cuda(scales, name + " scales")
    groups = (K + 63) // 64
    if codes.dtype != B.i8 or codes.dim() != 2 or codes.numel() == 0 or codes.shape[1] != 64 * groups:
        raise ValueError(f"{name} codes must be int8 [M, padded_k(K)]")
    m = codes.shape[0]
    if scales.dtype != B.f32 or scales.shape != (m, groups):
        raise ValueError(f"{name} scales must be float32 [M, padded_k(K) / 64]")
    if scales.device != codes.device:
        raise ValueError(f"{name} codes and scales are on different devices")
    if M is not None and m != M:
        raise ValueError(f"{name} does not have the other arrays' shape")
    return codes.data_ptr(), scales.data_ptr(), abi.SAVED8, m, K, codes.device


def _output(B, out, M, K, dtype, device, like=None):
    """`out`, checked, or a new [M, K] tensor (`like`: one of that shape on that device)."""
    if out is None:
        if like is not None and like.dtype == dtype:
            return B.empty_like(like)
        return B.empty(M, K, dtype=dtype, device=device)
    _require_cuda(out, "out")
    if out.shape != (M, K) or out.dtype != dtype or out.device != device:
        raise ValueError(f"out must be {dtype} [{M}, {K}] on {device}")
    return out


def _empty_saved(B, M, K, device):
    groups = (K + 63) // 64
    return (B.empty(M, 64 * groups, dtype=B.i8, device=device),
            B.empty(M, groups, dtype=B.f32, device=device))


def save_activations(X):
    """X (float32 or bfloat16 [M, K]) in 8 bits: the pair (codes, scales)."""
    B = _BLOCK or _block()
    dt, M, K = _matrix(B, X, "X")
    device = X.device
    codes, scales = saved = _empty_saved(B, M, K, device)
    B.launch(B.save_activations, device, X.data_ptr(), dt, M, K, codes.data_ptr(), scales.data_ptr())
    return saved


def restore_activations(saved, K: int, dtype=None, out=None):
    """The [M, K] values that ``saved`` stands for, as float32 (default) or bfloat16."""
    B = _BLOCK or _block()
    codes, scales, _, M, K, device = _whole_or_saved(B, tuple(saved), K, "saved")
    if dtype is None:
        dtype = B.f32 if out is None else out.dtype
    dt = _plain_dtype(B, dtype, "dtype")
    X = _output(B, out, M, K, dtype, device)
    B.launch(B.restore_activations, device, codes, scales, M, K, X.data_ptr(), dt)
    return X


def layer_norm(X, weight=None, bias=None, eps: float = 1e-5, K: int | None = None, out_dtype=None,
               return_stats: bool = False, save: bool = False, out=None):
    """Layer norm over the rows of X: float32 or bfloat16 [M, K], or a saved pair (then K is needed).

    ``weight``, ``bias``: float32 [K] or None.  Y is of ``out_dtype`` (default: X's; float32 for a saved
    pair).  Returns Y; (Y, mean, rstd) with ``return_stats``, for :func:`layer_norm_backward`; and
    (Y, mean, rstd, saved) with ``save``, X in 8 bits from the same pass.
    """
    B = _BLOCK or _block()
    x, xs, dt, M, K, device = _whole_or_saved(B, X, K, "X")
    like = None if xs else X
    if out_dtype is None:
        out_dtype = out.dtype if out is not None else B.f32 if xs else X.dtype
    ydt = _plain_dtype(B, out_dtype, "out_dtype")
    w, b = _vector(B, weight, K, device, "weight"), _vector(B, bias, K, device, "bias")
    if save and xs:
        raise ValueError("X is saved already")
    Y = _output(B, out, M, K, out_dtype, device, like)
    if not (return_stats or save):
        B.launch(B.layer_norm, device, x, xs, dt, M, K, w, b, eps, Y.data_ptr(), ydt, 0, 0, 0, 0)
        return Y
    mean = B.empty(M, dtype=B.f32, device=device)
    rstd = B.empty_like(mean)
    if not save:
        B.launch(B.layer_norm, device, x, xs, dt, M, K, w, b, eps, Y.data_ptr(), ydt, mean.data_ptr(),
                 rstd.data_ptr(), 0, 0)
        return Y, mean, rstd
    codes, scales = saved = _empty_saved(B, M, K, device)
    B.launch(B.layer_norm, device, x, xs, dt, M, K, w, b, eps, Y.data_ptr(), ydt, mean.data_ptr(),
             rstd.data_ptr(), codes.data_ptr(), scales.data_ptr())
    return Y, mean, rstd, saved


def layer_norm_backward(dY, X, mean, rstd, weight=None, out_dtype=None, need_dx: bool = True,
                        need_dw: bool = True, workspace=None):
    """Gradients (dX, dweight, dbias) of :func:`layer_norm` from dY (float32 or bfloat16 [M, K]).

    ``X``: the forward's input, whole or as it was saved; ``mean``, ``rstd``: from the forward.  dX [M, K]
    is of ``out_dtype`` (default: dY's), dweight and dbias are float32 [K]; None where not needed.
    """
    B = _BLOCK or _block()
    ddt, M, K = _matrix(B, dY, "dY")
    device = dY.device
    x, xs, dt, _, _, xdev = _whole_or_saved(B, X, K, "X", M)
    if xdev != device:
        raise ValueError("X is on another device")
    if mean is None or rstd is None:
        raise ValueError("mean and rstd of the forward are needed")
    mp, rp = _vector(B, mean, M, device, "mean"), _vector(B, rstd, M, device, "rstd")
    w = _vector(B, weight, K, device, "weight")
    if not (need_dx or need_dw):
        raise ValueError("nothing to compute")
    if out_dtype is None:
        out_dtype = dY.dtype
    odt = _plain_dtype(B, out_dtype, "out_dtype")
    dX = dw = db = None
    dxp = dwp = dbp = wsp = ws_bytes = 0
    if need_dx:
        dX = _output(B, None, M, K, out_dtype, device, dY)
        dxp = dX.data_ptr()
    if need_dw:
        dw = B.empty(K, dtype=B.f32, device=device)
        db = B.empty_like(dw)
        dwp, dbp = dw.data_ptr(), db.data_ptr()
        if workspace is None:
            ws_bytes = B.layer_norm_backward_workspace_bytes(M, K)
            if ws_bytes:
                workspace = B.empty(ws_bytes, dtype=B.i8, device=device)
                wsp = workspace.data_ptr()
        else:
            _require_cuda(workspace, "workspace")
            if workspace.device != device:
                raise ValueError("workspace is on another device")
            wsp, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    B.launch(B.layer_norm_backward, device, dY.data_ptr(), ddt, x, xs, dt, mp, rp, M, K, w, dxp, odt, dwp, dbp,
             wsp, ws_bytes)
    return dX, dw, db


def relu2(H, K: int | None = None, out_dtype=None, save: bool = False, out=None):
    """A = max(H, 0)^2 for H float32 or bfloat16 [M, K], or a saved pair (then K is needed).

    A is of ``out_dtype`` (default: H's; float32 for a saved pair).  With ``save`` returns (A, saved), H in
    8 bits from the same pass.
    """
    B = _BLOCK or _block()
    h, hs, dt, M, K, device = _whole_or_saved(B, H, K, "H")
    if out_dtype is None:
        out_dtype = out.dtype if out is not None else B.f32 if hs else H.dtype
    adt = _plain_dtype(B, out_dtype, "out_dtype")
    if save and hs:
        raise ValueError("H is saved already")
    A = _output(B, out, M, K, out_dtype, device, None if hs else H)
    if not save:
        B.launch(B.relu2, device, h, hs, dt, M, K, A.data_ptr(), adt, 0, 0)
        return A
    codes, scales = saved = _empty_saved(B, M, K, device)
    B.launch(B.relu2, device, h, hs, dt, M, K, A.data_ptr(), adt, codes.data_ptr(), scales.data_ptr())
    return A, saved


def relu2_backward(dA, H, out_dtype=None, out=None):
    """dH = dA * 2 max(H, 0) from dA (float32 or bfloat16 [M, K]) and H, whole or as it was saved.

    dH is of ``out_dtype`` (default: dA's; bfloat16 is what :func:`backward` takes).
    """
    B = _BLOCK or _block()
    adt, M, K = _matrix(B, dA, "dA")
    device = dA.device
    h, hs, dt, _, _, hdev = _whole_or_saved(B, H, K, "H", M)
    if hdev != device:
        raise ValueError("H is on another device")
    if out_dtype is None:
        out_dtype = out.dtype if out is not None else dA.dtype
    odt = _plain_dtype(B, out_dtype, "out_dtype")
    dH = _output(B, out, M, K, out_dtype, device, dA)
    B.launch(B.relu2_backward, device, dA.data_ptr(), adt, h, hs, dt, M, K, dH.data_ptr(), odt)
    return dH


# ---- the gated feed-forward block (include/bitlinear_gated.h) ----------------

_ACTS = {"relu2": abi.ACT_RELU2, "silu": abi.ACT_SILU}


def _act(act):
    a = _ACTS.get(act)
    if a is None:
        raise ValueError("act must be 'relu2' or 'silu'")
    return a


def _path(path):
    p = _PATHS.get(path)
    if p is None:
        raise ValueError("path must be 'auto', 'decode' or 'prefill'")
    return p


def _placed(t, index, name):
    """Raises unless t is a contiguous tensor on GPU `index`."""
    if t.get_device() != index or not t.is_contiguous():
        _require_cuda(t, name)
        raise ValueError(f"{name} is on another device")


def _ternary(B, w, K, N, index, name):
    """(packed address, gamma address, N) of (packed [N, packed_words(K)], gamma [1]) on GPU `index`."""
    packed, gamma = w
    if packed.get_device() != index or not packed.is_contiguous():
        _placed(packed, index, f"{name}'s packed weights")
    shape = packed.shape
    if len(shape) != 2 or shape[1] != (K + 63) // 64 * 4 or shape[0] < 1 or packed.element_size() != 4 \
            or (N is not None and shape[0] != N):
        raise ValueError(f"{name}'s packed weights must hold padded_k({K}) // 16 32-bit words for each of "
                         f"{'their' if N is None else N} rows")
    if gamma.get_device() != index or gamma.dtype != B.f32 or gamma.numel() != 1:
        _placed(gamma, index, f"{name}'s gamma")
        raise ValueError(f"{name}'s gamma must hold 1 float32 value")
    return packed.data_ptr(), gamma.data_ptr(), shape[0]


def _workspace(B, workspace, need, device):
    """(address, bytes, tensor to keep) of `workspace`, or of a new one of `need` bytes."""
    if workspace is None:
        if not need:
            return 0, 0, None
        workspace = B.empty(need, dtype=B.i8, device=device)
        return workspace.data_ptr(), need, workspace
    _require_cuda(workspace, "workspace")
    if workspace.device != device:
        raise ValueError("workspace is on another device")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


def _fits_decode(M, K, N):
    """decode_fits without the library's calls: at most 16 tokens, their codes within 65536 bytes."""
    return M <= 16 and M * ((K + 63) // 64 * 64 + 16) <= 65536 and M * N < (1 << 29)


def gated_forward(X, gate, up, K: int | None = None, act: str = "relu2", out_dtype=None, save=None,
                  path: str = "auto", out=None, workspace=None):
    """H = act(BitLinear_gate(X)) * BitLinear_up(X), act 'relu2' or 'silu'.

    X: float32 or bfloat16 [M, D], or its codes as :func:`quantize_activations` returns them (then K = D is
    needed; ``path`` and ``workspace`` do not apply).  ``gate``, ``up``: (packed [F, words(D)], gamma [1]).
    H [M, F] is of ``out_dtype`` (default float32).  With ``save`` a dtype returns (H, G, U), both projections
    in that type, for :func:`gated_backward`.
    """
    B = _BLOCK or _block()
    a, p = _act(act), _path(path)
    codes = isinstance(X, (tuple, list))
    if codes:
        Xq, ga, rs = X
        if K is None:
            raise ValueError("K is needed where X is given as codes")
        for t, nm in ((Xq, "Xq"), (rs, "rowsum")):
            _require_cuda(t, nm)
        M, device = Xq.shape[0], Xq.device
        if Xq.dtype != B.i8 or Xq.dim() != 2 or not Xq.numel() or Xq.shape[1] != (K + 63) // 64 * 64:
            raise ValueError("Xq must be int8 [M, padded_k(K)]")
        if rs.dtype != B.i32 or rs.numel() != M or rs.device != device:
            raise ValueError("rowsum must hold M int32 values on X's device")
        gap = _vector(B, ga, M, device, "gamma_a")
    else:
        dt, M, D = _matrix(B, X, "X")
        if K is not None and K != D:
            raise ValueError("K does not match X")
        K, device = D, X.device
    gp, gg, F = _ternary(B, gate, K, None, device.index, "gate")
    up_, ug, _ = _ternary(B, up, K, F, device.index, "up")
    if out_dtype is None:
        out_dtype = B.f32 if out is None else out.dtype
    hdt = _plain_dtype(B, out_dtype, "out_dtype")
    H = _output(B, out, M, F, out_dtype, device)
    G = U = None
    G_, U_, sdt = 0, 0, 0
    if save is not None:
        sdt = _plain_dtype(B, save, "save")
        G = B.empty(M, F, dtype=save, device=device)
        U = B.empty_like(G)
        G_, U_ = G.data_ptr(), U.data_ptr()
    if codes:
        B.launch(B.gated_forward_quantized, device, Xq.data_ptr(), gap, rs.data_ptr(), M, K, F, gp, gg, up_, ug, a,
                 H.data_ptr(), hdt, G_, U_, sdt)
    else:
        need = 0
        if workspace is None and not (p != abi.PATH_PREFILL and _fits_decode(M, K, F)) and p != abi.PATH_DECODE:
            need = B.forward_workspace_bytes(M, K)
        wsp, ws_bytes, keep = _workspace(B, workspace, need, device)
        B.launch(B.gated_forward, device, X.data_ptr(), dt, M, K, F, gp, gg, up_, ug, a, H.data_ptr(), hdt, G_, U_,
                 sdt, p, wsp, ws_bytes)
    return H if save is None else (H, G, U)


def gated_ffn_forward(X, gate, up, down, act: str = "relu2", path: str = "auto", return_hidden: bool = False,
                      out=None, workspace=None):
    """Y = BitLinear_down(act(BitLinear_gate(X)) * BitLinear_up(X)) for X float32 or bfloat16 [M, D].

    ``gate``, ``up`` = (packed [F, words(D)], gamma [1]), ``down`` = (packed [D_out, words(F)], gamma [1]).
    Returns Y float32 [M, D_out] (and the hidden layer float32 [M, F] if asked).
    """
    B = _BLOCK or _block()
    a, p = _act(act), _path(path)
    dt, M, D = _matrix(B, X, "X")
    device = X.device
    gp, gg, F = _ternary(B, gate, D, None, device.index, "gate")
    up_, ug, _ = _ternary(B, up, D, F, device.index, "up")
    dp, dg, Do = _ternary(B, down, F, None, device.index, "down")
    Y = _output(B, out, M, Do, B.f32, device)
    H = B.empty(M, F, dtype=B.f32, device=device) if return_hidden else None
    need = 0 if workspace is not None else B.gated_ffn_workspace_bytes(M, D, F, Do)
    wsp, ws_bytes, keep = _workspace(B, workspace, need, device)
    B.launch(B.gated_ffn_forward, device, X.data_ptr(), dt, M, D, F, Do, gp, gg, up_, ug, a, dp, dg, Y.data_ptr(),
             H.data_ptr() if return_hidden else 0, p, wsp, ws_bytes)
    return (Y, H) if return_hidden else Y


def gated_backward(dH, G, U, act: str = "relu2", out_dtype=None):
    """(dG, dU) of H = act(G) * U from dH (float32 or bfloat16 [M, F]) and the kept G and U.

    Both are of ``out_dtype`` (default bfloat16, what :func:`gated_input_backward` and :func:`backward` take).
    """
    B = _BLOCK or _block()
    a = _act(act)
    hdt, M, F = _matrix(B, dH, "dH")
    gdt, m, f = _matrix(B, G, "G")
    udt, m2, f2 = _matrix(B, U, "U")
    if (m, f) != (M, F) or (m2, f2) != (M, F) or udt != gdt:
        raise ValueError("dH, G and U must have one shape, G and U one dtype")
    device = dH.device
    if G.device != device or U.device != device:
        raise ValueError("dH, G and U are on different devices")
    if out_dtype is None:
        out_dtype = B.bf16
    odt = _plain_dtype(B, out_dtype, "out_dtype")
    dG = B.empty(M, F, dtype=out_dtype, device=device)
    dU = B.empty_like(dG)
    B.launch(B.gated_backward, device, dH.data_ptr(), hdt, G.data_ptr(), U.data_ptr(), gdt, M, F, a, dG.data_ptr(),
             dU.data_ptr(), odt)
    return dG, dU


def gated_input_backward(dG, dU, gateT, upT, K: int, out=None, workspace=None):
    """dX = gamma_gate (dG W_gate) + gamma_up (dU W_up), float32 [M, K], from bfloat16 dG, dU [M, F].

    ``gateT``, ``upT`` = (packedT [K, words(F)] as :func:`pack_transposed` returns it, gamma [1]); K: the
    projections' input width.  Their dW: :func:`backward` with dG and dU, ``need_dx=False``.
    """
    B = _BLOCK or _block()
    _, M, F = _matrix(B, dG, "dG")
    _, m, f = _matrix(B, dU, "dU")
    if dG.dtype != B.bf16 or dU.dtype != B.bf16 or (m, f) != (M, F):
        raise ValueError("dG and dU must be bfloat16 of one shape")
    device = dG.device
    if dU.device != device:
        raise ValueError("dG and dU are on different devices")
    gp, gg, _ = _ternary(B, gateT, F, K, device.index, "gateT")
    up_, ug, _ = _ternary(B, upT, F, K, device.index, "upT")
    dX = _output(B, out, M, K, B.f32, device)
    need = 0
    if workspace is None:
        copies = bool(F % 8 or dG.data_ptr() % 16 or dU.data_ptr() % 16)
        need = B.gated_input_backward_workspace_bytes(M, F, K, copies)
    wsp, ws_bytes, keep = _workspace(B, workspace, need, device)
    B.launch(B.gated_input_backward, device, dG.data_ptr(), dU.data_ptr(), M, F, K, gp, gg, up_, ug, dX.data_ptr(),
             wsp, ws_bytes)
    return dX


# ---- low-rank adapters and dropout (include/bitlinear_adapters.h) --------------
#
# Adapters are a triple (down [A, R, K], up [A, R, N], scales float32 [A]), down
# and up float32 or bfloat16; rows int32 [M] names the adapter of each token
# (outside 0 .. A - 1: none).

def _adapters(B, adapters, rows, M, K, N, device):
    """(A, R, N, addresses of down and up, their abi dtype, addresses of scales and rows), checked."""
    down, up, scales = adapters
    index = device.index
    for t, nm in ((down, "down"), (up, "up"), (rows, "rows"), (scales, "scales")):
        if t.get_device() != index or not t.is_contiguous():
            _placed(t, index, nm)
    wdt = _plain_dtype(B, down.dtype, "down")
    if up.dtype != down.dtype:
        raise ValueError("down and up must have one dtype")
    ds, us = down.shape, up.shape
    if len(ds) != 3 or len(us) != 3 or us[:2] != ds[:2] or 0 in ds or us[2] < 1:
        raise ValueError("down must be [A, R, K] and up [A, R, N]")
    A, R, k = ds
    n = us[2]
    if k != K or (N is not None and n != N):
        raise ValueError("down and up do not match the projection")
    if rows.dtype != B.i32 or rows.shape != (M,):
        raise ValueError("rows must hold M int32 values")
    if scales.dtype != B.f32 or scales.numel() != A:
        raise ValueError(f"scales must hold {A} float32 values")
    return A, R, n, down.data_ptr(), up.data_ptr(), wdt, scales.data_ptr(), rows.data_ptr()


def adapters_forward(X, adapters, rows, Y, return_low: bool = False, workspace=None):
    """Y[m] += scale[a] (X[m] down[a]^T) up[a], a = rows[m], into Y (float32 [M, N], as :func:`forward`
    returns it), which is returned.

    X: float32 or bfloat16 [M, K].  With ``return_low`` returns (Y, T), T = X down^T float32 [M, R] for
    :func:`adapters_backward`.
    """
    B = _BLOCK or _block()
    dt, M, K = _matrix(B, X, "X")
    device = X.device
    A, R, N, dn, up, wdt, sc, ids = _adapters(B, adapters, rows, M, K, None, device)
    _output(B, Y, M, N, B.f32, device)
    T = B.empty(M, R, dtype=B.f32, device=device) if return_low else None
    need = 0 if workspace is not None else B.adapters_workspace_bytes(M, K, N, R)
    wsp, ws_bytes, keep = _workspace(B, workspace, need, device)
    B.launch(B.adapters_forward, device, X.data_ptr(), dt, M, K, N, ids, A, R, dn, up, wdt, sc, Y.data_ptr(),
             T.data_ptr() if return_low else 0, wsp, ws_bytes)
    return (Y, T) if return_low else Y


def adapted_forward(X, packed, gamma, adapters, rows, K: int | None = None, path: str = "auto",
                    return_low: bool = False, out=None, workspace=None):
    """Y[m] = BitLinear(X)[m] + scale[a] (X[m] down[a]^T) up[a], a = rows[m]: a shared ternary projection
    and every token's own adapter.

    X: float32 or bfloat16 [M, K]; ``packed``, ``gamma``, ``path``: as for :func:`forward`.  Returns Y
    float32 [M, N], or (Y, T) with ``return_low`` (see :func:`adapters_forward`).
    """
    B = _BLOCK or _block()
    p = _path(path)
    dt, M, Kx = _matrix(B, X, "X")
    if K is not None and K != Kx:
        raise ValueError("K does not match X")
    K, device = Kx, X.device
    pk, gm, N = _ternary(B, (packed, gamma), K, None, device.index, "the projection")
    A, R, _, dn, up, wdt, sc, ids = _adapters(B, adapters, rows, M, K, N, device)
    Y = _output(B, out, M, N, B.f32, device)
    T = B.empty(M, R, dtype=B.f32, device=device) if return_low else None
    need = 0 if workspace is not None else B.adapted_workspace_bytes(M, K, N, R)
    wsp, ws_bytes, keep = _workspace(B, workspace, need, device)
    B.launch(B.adapted_forward, device, X.data_ptr(), dt, M, K, pk, N, gm, ids, A, R, dn, up, wdt, sc, Y.data_ptr(),
             T.data_ptr() if return_low else 0, p, wsp, ws_bytes)
    return (Y, T) if return_low else Y


def adapters_backward(dY, X, T, adapters, rows, dX=None, need_dx: bool = True, need_dw: bool = True,
                      workspace=None):
    """Gradients (dX, ddown, dup) of :func:`adapters_forward` from dY (float32 or bfloat16 [M, N]).

    ``X``, ``T``: the forward's input and its X down^T.  ``dX``: a float32 [M, K] tensor to add to (the
    frozen projection's, from :func:`backward`); else a new one, zeros for tokens without an adapter.
    ddown, dup: float32 [A, R, K] and [A, R, N].  None where not needed.
    """
    B = _BLOCK or _block()
    ddt, M, N = _matrix(B, dY, "dY")
    xdt, m, K = _matrix(B, X, "X")
    device = dY.device
    if m != M:
        raise ValueError("X and dY do not have the same rows")
    if X.device != device:
        raise ValueError("X is on another device")
    A, R, _, dn, up, wdt, sc, ids = _adapters(B, adapters, rows, M, K, N, device)
    if not (need_dx or need_dw):
        raise ValueError("nothing to compute")
    if dX is not None and not need_dx:
        raise ValueError("dX is given and not needed")
    accumulate = dX is not None
    tp = _vector(B, T, M * R, device, "T") if need_dw else 0
    if need_dw and T is None:
        raise ValueError("T of the forward is needed")
    dd = du = None
    dxp = ddp = dup_ = 0
    if need_dx:
        dX = _output(B, dX, M, K, B.f32, device)
        dxp = dX.data_ptr()
    if need_dw:
        dd = B.empty(A, R, K, dtype=B.f32, device=device)
        du = B.empty(A, R, N, dtype=B.f32, device=device)
        ddp, dup_ = dd.data_ptr(), du.data_ptr()
    need = 0 if workspace is not None else B.adapters_backward_workspace_bytes(M, K, N, A, R)
    wsp, ws_bytes, keep = _workspace(B, workspace, need, device)
    B.launch(B.adapters_backward, device, dY.data_ptr(), ddt, X.data_ptr(), xdt, tp, M, K, N, ids, A, R, dn, up, wdt,
             sc, dxp, int(accumulate), ddp, dup_, wsp, ws_bytes)
    return dX, dd, du


def dropout(X, p: float, seed: int, offset: int = 0, residual=None, out_dtype=None, out=None):
    """X with each value dropped with probability p and the others times 1 / (1 - p), plus ``residual``.

    X, ``residual``: float32 or bfloat16 of one shape.  The mask is a function of (seed, offset, index), 64
    bits each, and never stored: the backward pass is the same call on the gradient.  The result is of
    ``out_dtype`` (default: X's); ``out`` may be X or the residual itself.
    """
    B = _BLOCK or _block()
    if not (X.is_cuda and X.is_contiguous()):
        _require_cuda(X, "X")
    xdt = _plain_dtype(B, X.dtype, "X")
    n, device = X.numel(), X.device
    if n == 0:
        raise ValueError("X must hold at least one value")
    rp = rdt = 0
    if residual is not None:
        if not (residual.is_cuda and residual.is_contiguous()):
            _require_cuda(residual, "residual")
        rdt = _plain_dtype(B, residual.dtype, "residual")
        if residual.shape != X.shape or residual.get_device() != device.index:
            raise ValueError("residual must have X's shape and device")
        rp = residual.data_ptr()
    if out_dtype is None:
        out_dtype = X.dtype if out is None else out.dtype
    ydt = _plain_dtype(B, out_dtype, "out_dtype")
    if not (0.0 <= p < 1.0):
        raise ValueError("p must be at least 0 and below 1")
    if not (0 <= seed < 1 << 64 and 0 <= offset < 1 << 64):
        raise ValueError("seed and offset must be unsigned 64-bit numbers")
    if out is None:
        out = B.empty_like(X, dtype=out_dtype)
    else:
        _require_cuda(out, "out")
        if out.shape != X.shape or out.dtype != out_dtype or out.device != device:
            raise ValueError(f"out must be {out_dtype} of X's shape on {device}")
    B.launch(B.dropout, device, X.data_ptr(), xdt, rp, rdt, n, p, seed, offset, out.data_ptr(), ydt)
    return out
