"""ctypes view of libbitlinear.so (the C ABI declared in include/bitlinear.h and
include/bitlinear_block.h) and of the benchmark's probe library libbitlinear_probe.so
(include/bitlinear_probe.h).

Loading is lazy and fails loudly: there is no fallback implementation.
"""
from __future__ import annotations

import ctypes
import os

from .build import LIB_PATH, PROBE_LIB_PATH

OK = 0
ERR_NULL = -1
ERR_SHAPE = -2
ERR_DTYPE = -3
ERR_ALIGN = -4
ERR_WORKSPACE = -5
ERR_HIP = -6
ERR_ARG = -7

F32 = 0
BF16 = 1
SAVED8 = 2  # an input saved in 8 bits (bitlinear_block.h)

PATH_AUTO = 0
PATH_DECODE = 1
PATH_PREFILL = 2

_i64 = ctypes.c_int64
_int = ctypes.c_int
_f32 = ctypes.c_float
_sz = ctypes.c_size_t
_p = ctypes.c_void_p

# name -> (restype, argtypes)
SIGNATURES = {
    "bitlinear_padded_k": (_i64, [_i64]),
    "bitlinear_packed_bytes": (_sz, [_i64, _i64]),
    "bitlinear_quantize_workspace_bytes": (_sz, []),
    "bitlinear_forward_workspace_bytes": (_sz, [_i64, _i64]),
    "bitlinear_max_decode_m": (_int, []),
    "bitlinear_max_decode_codes": (_i64, []),
    "bitlinear_quantize_weights": (_int, [_p, _i64, _i64, _p, _p, _p, _sz, _p]),
    "bitlinear_quantize_activations": (_int, [_p, _int, _i64, _i64, _p, _p, _p, _p]),
    "bitlinear_forward": (_int, [_p, _int, _i64, _i64, _p, _i64, _p, _p, _p, _sz, _p]),
    "bitlinear_forward_ex": (_int, [_p, _int, _i64, _i64, _p, _i64, _p, _p, _p, _int, _p, _sz, _p]),
    "bitlinear_forward_quantized": (_int, [_p, _p, _p, _i64, _i64, _p, _i64, _p, _p, _p, _p]),
    "bitlinear_forward_batched": (_int, [_i64, _p, _int, _i64, _i64, _p, _i64, _p, _p, _p]),
    "bitlinear_ffn_workspace_bytes": (_sz, [_i64, _i64, _i64, _i64]),
    "bitlinear_ffn_forward": (_int, [_i64, _p, _int, _i64, _i64, _i64, _i64, _p, _p, _p, _p, _p, _p, _int,
                                     _p, _sz, _p]),
    "bitlinear_ste_mask_bytes": (_sz, [_i64, _i64]),
    "bitlinear_pack_transposed": (_int, [_p, _i64, _i64, _p, _p, _p, _p]),
    "bitlinear_backward_workspace_bytes": (_sz, [_i64, _i64, _i64]),
    "bitlinear_backward": (_int, [_p, _i64, _i64, _i64, _p, _p, _p, _p, _p, _p, _p, _p, _sz, _p]),
    "bitlinear_r3_padded_k": (_i64, [_i64]),
    "bitlinear_r3_packed_bytes": (_sz, [_i64, _i64]),
    "bitlinear_quantize_weights_r3": (_int, [_p, _i64, _i64, _p, _p, _p, _sz, _p]),
    "bitlinear_forward_r3": (_int, [_i64, _p, _int, _i64, _i64, _p, _i64, _p, _p, _p, _p]),
    "bitlinear_lut_workspace_bytes": (_sz, [_i64, _i64, _i64]),
    "bitlinear_forward_lut": (_int, [_i64, _p, _int, _i64, _i64, _p, _i64, _p, _p, _p, _p, _sz, _p]),
    "bitlinear_forward_noalloc": (_int, [_p, _int, _i64, _i64, _p, _i64, _p, _p, _p]),
    "bitlinear_status_string": (ctypes.c_char_p, [_int]),
}

# the operators around BitLinear (include/bitlinear_block.h, same library)
BLOCK_SIGNATURES = {
    "bitlinear_saved_groups": (_i64, [_i64]),
    "bitlinear_save_activations": (_int, [_p, _int, _i64, _i64, _p, _p, _p]),
    "bitlinear_restore_activations": (_int, [_p, _p, _i64, _i64, _p, _int, _p]),
    "bitlinear_layer_norm": (_int, [_p, _p, _int, _i64, _i64, _p, _p, _f32, _p, _int, _p, _p, _p, _p, _p]),
    "bitlinear_layer_norm_backward_workspace_bytes": (_sz, [_i64, _i64]),
    "bitlinear_layer_norm_backward": (_int, [_p, _int, _p, _p, _int, _p, _p, _i64, _i64, _p, _p, _int, _p, _p,
                                             _p, _sz, _p]),
    "bitlinear_relu2": (_int, [_p, _p, _int, _i64, _i64, _p, _int, _p, _p, _p]),
    "bitlinear_relu2_backward": (_int, [_p, _int, _p, _p, _int, _i64, _i64, _p, _int, _p]),
}

NOALLOC_SCRATCH_BYTES = 80 * 1024 * 1024  # BITLINEAR_NOALLOC_SCRATCH_BYTES

# the attainable-peak probes of libbitlinear_probe.so (not the BitLinear ABI)
PROBE_SIGNATURES = {
    "bitlinear_probe_stream": (_int, [_p, _p, _i64, _int, _p, _p]),
    "bitlinear_probe_mfma_i8": (_int, [_int, _int, _p, _p]),
    "bitlinear_probe_mfma_bf16": (_int, [_int, _int, _p, _p]),
}

_LIB = None
_PROBE_LIB = None


class BitLinearError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} failed: status {status} ({status_string(status)})")


def _open(path: str, signatures) -> ctypes.CDLL:
    if not os.path.exists(path):
        raise RuntimeError(
            f"{path} is missing: build the HIP libraries first "
            "(python -m bitlinear_absmean_ternarise_bit_amd.build)")
    # Load torch's HIP runtime first when torch is present: the library then
    # binds to that same runtime, so streams and device pointers from torch are
    # valid in its launches (a second runtime in the process would not share them).
    try:
        import torch  # noqa: F401
    except ImportError:
        pass
    lib = ctypes.CDLL(path)
    for name, (res, args) in signatures.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load the BitLinear HIP library (once).  Raises if it has not been built."""
    global _LIB
    if _LIB is None:
        _LIB = _open(path, {**SIGNATURES, **BLOCK_SIGNATURES})
    return _LIB


def load_probe(path: str = PROBE_LIB_PATH) -> ctypes.CDLL:
    """Load the benchmark's probe library (once).  Raises if it has not been built."""
    global _PROBE_LIB
    if _PROBE_LIB is None:
        _PROBE_LIB = _open(path, PROBE_SIGNATURES)
    return _PROBE_LIB


def status_string(status: int) -> str:
    return load().bitlinear_status_string(status).decode()


def check(fn: str, status: int) -> None:
    if status != OK:
        raise BitLinearError(fn, status)
