"""ctypes declarations of the libqlora C ABI (include/qlora.h)."""
from __future__ import annotations

import ctypes as C
import os

PKG = os.path.dirname(os.path.abspath(__file__))
# QLORA_LIB selects another build of the same sources (the sanitizer build, for example)
LIB_PATH = os.environ.get("QLORA_LIB") or os.path.join(PKG, "libqlora.so")

NOALLOC_SCRATCH_BYTES = 64 * 1024 * 1024   # QLORA_NOALLOC_SCRATCH_BYTES in qlora.h

STATUS = {
    0: "QLORA_OK",
    1: "QLORA_ERR_NULL",
    2: "QLORA_ERR_SHAPE",
    3: "QLORA_ERR_ALIGN",
    4: "QLORA_ERR_UNSUPPORTED",
    5: "QLORA_ERR_WORKSPACE",
    6: "QLORA_ERR_HIP",
}


class qlora_nf4(C.Structure):
    _fields_ = [
        ("rows", C.c_int64),
        ("cols", C.c_int64),
        ("double_quant", C.c_int32),
        ("codebook", C.c_int32),
        ("block_size", C.c_int32),
        ("reserved", C.c_int32),
        ("codes", C.c_void_p),
        ("absmax", C.c_void_p),
        ("c1", C.c_void_p),
        ("mu", C.c_void_p),
    ]


class qlora_heads(C.Structure):
    _fields_ = [("data", C.c_void_p), ("row_stride", C.c_int64), ("head_stride", C.c_int64), ("heads", C.c_int32),
                ("reserved", C.c_int32)]


class qlora_kv_cache(C.Structure):
    _fields_ = [("pages", C.c_int64), ("page_size", C.c_int32), ("heads", C.c_int32), ("head_dim", C.c_int32),
                ("block_size", C.c_int32), ("codebook", C.c_int32), ("reserved", C.c_int32), ("k_codes", C.c_void_p),
                ("k_scale", C.c_void_p), ("v_codes", C.c_void_p), ("v_scale", C.c_void_p)]


class qlora_kv_batch(C.Structure):
    _fields_ = [("batch", C.c_int32), ("max_pages", C.c_int32), ("start", C.c_void_p), ("length", C.c_void_p),
                ("table", C.c_void_p), ("fault", C.c_void_p)]


class qlora_kernel_time(C.Structure):
    _fields_ = [("name", C.c_char * 48), ("launches", C.c_int64), ("total_ms", C.c_double)]


_HEADS = C.c_void_p   # const qlora_heads*: a structure by reference, or its bytes

# name -> (restype, argtypes); every name is declared in include/qlora.h
SIGNATURES = {
    "qlora_status_str": (C.c_char_p, [C.c_int]),
    "qlora_version": (C.c_char_p, []),
    "qlora_nf4_codebook": (C.c_int, [C.POINTER(C.c_float), C.POINTER(C.c_float)]),
    "qlora_codebook_table": (C.c_int, [C.c_int32, C.POINTER(C.c_float), C.POINTER(C.c_float)]),
    "qlora_merge_adapter": (C.c_int, [C.POINTER(qlora_nf4), C.c_void_p, C.c_void_p, C.c_int32, C.c_float, C.c_void_p,
                                      C.c_void_p]),
    "qlora_adamw_step": (C.c_int, [C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_int64, C.c_int64,
                                   C.c_float, C.c_float, C.c_float, C.c_float, C.c_float, C.c_void_p]),
    "qlora_nf4_sizes": (C.c_int, [C.c_int64, C.c_int64, C.c_int32, C.c_int32, C.POINTER(C.c_size_t),
                                  C.POINTER(C.c_size_t), C.POINTER(C.c_size_t), C.POINTER(C.c_size_t)]),
    "qlora_quantize_workspace": (C.c_size_t, [C.c_int64, C.c_int64, C.c_int32, C.c_int32]),
    "qlora_fwd_workspace": (C.c_size_t, [C.c_int64, C.c_int64, C.c_int64, C.c_int32]),
    "qlora_bwd_workspace": (C.c_size_t, [C.c_int64, C.c_int64, C.c_int64, C.c_int32]),
    "qlora_quantize_nf4": (C.c_int, [C.c_void_p, C.c_int64, C.c_int64, C.POINTER(qlora_nf4), C.c_void_p, C.c_size_t,
                                     C.c_void_p]),
    "qlora_dequant": (C.c_int, [C.POINTER(qlora_nf4), C.c_void_p, C.c_void_p]),
    "qlora_linear_fwd": (C.c_int, [C.c_void_p, C.c_int64, C.POINTER(qlora_nf4), C.c_void_p, C.c_void_p, C.c_int32,
                                   C.c_float, C.c_void_p, C.c_void_p, C.c_void_p, C.c_size_t, C.c_void_p]),
    "qlora_linear_fwd_noalloc": (C.c_int, [C.c_void_p, C.c_int64, C.POINTER(qlora_nf4), C.c_void_p, C.c_void_p,
                                           C.c_int32, C.c_float, C.c_void_p, C.c_void_p, C.c_void_p]),
    "qlora_linear_bwd": (C.c_int, [C.c_void_p, C.c_void_p, C.c_void_p, C.c_int64, C.POINTER(qlora_nf4), C.c_void_p,
                                   C.c_void_p, C.c_int32, C.c_float, C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p,
                                   C.c_size_t, C.c_void_p]),
    "qlora_state_page_out": (C.c_int, [C.c_void_p, C.c_void_p, C.c_size_t, C.c_void_p]),
    "qlora_state_page_in": (C.c_int, [C.c_void_p, C.c_void_p, C.c_size_t, C.c_void_p]),
    "qlora_qk_norm_rope": (C.c_int, [_HEADS, _HEADS, C.c_int64, C.c_int32, C.c_void_p,
                                     C.c_void_p, C.c_float, C.c_void_p, C.c_void_p, C.c_int32, C.c_int32,
                                     _HEADS, _HEADS, C.c_void_p]),
    "qlora_qk_norm_rope_bwd_workspace": (C.c_size_t, [C.c_int64, C.c_int32, C.c_int32, C.c_int32]),
    "qlora_qk_norm_rope_bwd": (C.c_int, [_HEADS, _HEADS, _HEADS,
                                         _HEADS, C.c_int64, C.c_int32, C.c_void_p, C.c_void_p,
                                         C.c_float, C.c_void_p, C.c_void_p, C.c_int32, C.c_int32,
                                         _HEADS, _HEADS, C.c_void_p, C.c_void_p,
                                         C.c_void_p, C.c_size_t, C.c_void_p]),
    "qlora_kv_sizes": (C.c_int, [C.POINTER(qlora_kv_cache), C.POINTER(C.c_size_t), C.POINTER(C.c_size_t)]),
    "qlora_kv_write": (C.c_int, [_HEADS, _HEADS, C.c_int64, C.POINTER(qlora_kv_cache),
                                 C.POINTER(qlora_kv_batch), C.c_void_p]),
    "qlora_kv_read": (C.c_int, [C.POINTER(qlora_kv_cache), C.POINTER(qlora_kv_batch), C.c_int64,
                                _HEADS, _HEADS, C.c_void_p]),
    "qlora_kv_attn_workspace": (C.c_size_t, [C.POINTER(qlora_kv_cache), C.POINTER(qlora_kv_batch), C.c_int64,
                                             C.c_int32]),
    "qlora_kv_attn": (C.c_int, [_HEADS, C.c_int64, C.POINTER(qlora_kv_cache),
                                C.POINTER(qlora_kv_batch), C.c_float, C.c_int32, C.c_int32, _HEADS,
                                C.c_void_p, C.c_void_p, C.c_size_t, C.c_void_p]),
    "qlora_profile_enable": (C.c_int, [C.c_int32]),
    "qlora_profile_read": (C.c_int32, [C.POINTER(qlora_kernel_time), C.c_int32, C.c_int32]),
}

_lib = None


class StaleLibraryError(OSError):
    """The built library's source hash differs from the sources in the package."""


def load(build_if_missing: bool = True) -> C.CDLL:
    """Load libqlora.so from the package directory (building it first if it is absent).

    A library built from other sources than the ones beside it is refused: its version
    string carries the hash of the sources it was built from (see build.source_hash)."""
    global _lib
    if _lib is not None:
        return _lib
    from . import build as _build

    if not os.path.exists(LIB_PATH):
        if not build_if_missing:
            raise OSError(f"libqlora.so is not built ({LIB_PATH})")
        _build.build()
    lib = C.CDLL(LIB_PATH)
    lib.qlora_version.restype = C.c_char_p
    version = lib.qlora_version().decode()
    want = _build.source_hash()
    if f"src {want}" not in version:
        raise StaleLibraryError(f"{LIB_PATH} ({version}) was built from other sources than the current ones "
                                f"(src {want}); rebuild with python -m bit_nf4_quantized_11_amd.build")
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib
