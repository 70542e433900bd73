"""ctypes loader for the native library ``lib/libgptq.so``.

The library is loaded on first use and never replaced by anything else: if it
is missing or fails to load, every call raises.  There is no CPU fallback.
"""

from __future__ import annotations

import ctypes
import importlib.util
import os
import re
import threading
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "lib", "libgptq.so")
BINDING_PATH = os.path.join(PKG, "lib", "_binding.so")
HEADER = os.path.join(os.path.dirname(PKG), "include", "gptq.h")

_lock = threading.Lock()
_lib = None

c_i64 = ctypes.c_int64
c_int = ctypes.c_int
c_float = ctypes.c_float
c_void_p = ctypes.c_void_p


class GptqStats(ctypes.Structure):
    _fields_ = [
        ("damped_loss", ctypes.c_double),
        ("ms_prepare", ctypes.c_float),
        ("ms_factor", ctypes.c_float),
        ("ms_sweep", ctypes.c_float),
        ("ms_pack", ctypes.c_float),
        ("panel_width", ctypes.c_int32),
        ("outer_width", ctypes.c_int32),
    ]


_SIGNATURES = {
    "gptq_accumulate_hessian": (c_int, [c_void_p, c_int, c_i64, c_i64, c_void_p, c_void_p]),
    "gptq_quantize_layer": (c_int, [c_void_p, c_int, c_i64, c_i64, c_void_p, c_int, c_int, c_float, c_int,
                                    c_int, c_int, c_int, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                                    ctypes.POINTER(GptqStats)]),
    "gptq_factor_hessian": (c_int, [c_void_p, c_i64, c_float, c_int, c_void_p, c_void_p, c_void_p]),
    "gptq_factor_hessians": (c_int, [c_int, ctypes.POINTER(c_void_p), ctypes.POINTER(c_i64), c_float, c_int,
                                     ctypes.POINTER(c_void_p), ctypes.POINTER(c_void_p), c_void_p,
                                     ctypes.POINTER(c_int)]),
    "gptq_quantize_layer_factored": (c_int, [c_void_p, c_int, c_i64, c_i64, c_void_p, c_void_p, c_int, c_int,
                                             c_int, c_int, c_int, c_void_p, c_void_p, c_void_p, c_void_p,
                                             c_void_p, ctypes.POINTER(GptqStats)]),
    "gptq_quantize_linears": (c_int, [c_int, ctypes.POINTER(c_void_p), ctypes.POINTER(c_i64), c_float, c_int,
                                      ctypes.POINTER(c_void_p), ctypes.POINTER(c_void_p), c_int,
                                      ctypes.POINTER(c_void_p), c_int, ctypes.POINTER(c_i64), ctypes.POINTER(c_int),
                                      c_int, c_int, c_int, c_int, c_int, ctypes.POINTER(c_void_p),
                                      ctypes.POINTER(c_void_p), ctypes.POINTER(c_void_p), ctypes.POINTER(c_void_p),
                                      ctypes.POINTER(c_void_p), c_void_p, ctypes.POINTER(c_int)]),
    "gptq_export_layer": (c_int, [c_void_p, c_void_p, c_i64, c_i64, c_int, c_void_p, c_void_p, c_void_p]),
    "gptq_dequantize_weight": (c_int, [c_void_p, c_void_p, c_void_p, c_void_p, c_i64, c_i64, c_i64, c_int, c_int,
                                       c_void_p, c_void_p]),
    "gptq_quantized_linear": (c_int, [c_void_p, c_int, c_i64, c_i64, c_void_p, c_void_p, c_void_p, c_void_p,
                                      c_void_p, c_i64, c_i64, c_int, c_void_p, c_void_p]),
    "gptq_reorder_act_order": (c_int, [c_void_p, c_void_p, c_i64, c_i64, c_i64, c_int, c_void_p, c_void_p, c_void_p,
                                       c_void_p]),
    "gptq_test_wait_expiry": (c_int, [c_int, ctypes.c_uint32]),
    "gptq_rmsnorm": (c_int, [c_void_p, c_int, c_i64, c_i64, c_void_p, c_float, c_void_p, c_void_p]),
    "gptq_rope": (c_int, [c_void_p, c_int, c_i64, c_int, c_int, c_int, ctypes.c_double, c_void_p]),
    "gptq_attention": (c_int, [c_void_p, c_void_p, c_void_p, c_int, c_i64, c_int, c_int, c_int, c_void_p, c_void_p]),
    "gptq_silu_mul": (c_int, [c_void_p, c_void_p, c_int, c_i64, c_void_p, c_void_p]),
    "gptq_add": (c_int, [c_void_p, c_void_p, c_int, c_i64, c_void_p, c_void_p]),
    "gptq_rotary_frequencies": (c_int, [c_int, ctypes.c_double, c_int, ctypes.c_double, c_i64, ctypes.c_double,
                                        ctypes.c_double, ctypes.POINTER(ctypes.c_double), ctypes.POINTER(c_float)]),
    "gptq_rotary": (c_int, [c_void_p, c_void_p, c_int, c_i64, c_int, c_int, c_int, c_int, c_int, c_i64, c_i64, c_i64,
                            c_i64, c_void_p, c_void_p, c_float, c_void_p, c_void_p, c_i64, c_i64, c_i64, c_i64,
                            c_void_p]),
    "gptq_cache_write": (c_int, [c_void_p, c_void_p, c_int, c_i64, c_int, c_int, c_i64, c_i64, c_i64, c_i64, c_void_p,
                                 c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_int, c_i64, c_int, c_void_p,
                                 c_void_p]),
    "gptq_cache_read": (c_int, [c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_int, c_i64, c_int,
                                c_void_p, c_i64, c_int, c_int, c_int, c_void_p, c_void_p, c_void_p]),
    "gptq_paged_attention": (c_int, [c_void_p, c_int, c_i64, c_int, c_int, c_int, c_i64, c_i64, c_void_p, c_void_p,
                                     c_void_p, c_void_p, c_void_p, c_void_p, c_int, c_i64, c_int, c_void_p, c_i64,
                                     c_void_p, c_void_p, c_i64, c_i64, c_int, c_float, c_void_p, c_void_p]),
    "gptq_device_status": (c_int, [c_void_p, c_int]),
    "gptq_trim_workspace": (c_int, []),
    "gptq_status_string": (ctypes.c_char_p, [c_int]),
    "gptq_launch_count": (ctypes.c_uint64, []),
    "gptq_version": (c_int, []),
}


def lib():
    """The loaded native library (raises RuntimeError if it is not built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(
                    f"native GPTQ library missing at {LIB_PATH}; build it with "
                    "`python -m post_weight_quantization_layer_b200.build`")
            handle = ctypes.CDLL(LIB_PATH)
            for name, (res, args) in _SIGNATURES.items():
                fn = getattr(handle, name)
                fn.restype = res
                fn.argtypes = args
            _lib = handle
    return _lib


_binding = None


def binding():
    """The native front of the serving operators (csrc/binding.cpp), opened on the native library (raises
    RuntimeError if it is not built)."""
    global _binding
    if _binding is not None:
        return _binding
    with _lock:
        if _binding is None:
            if not os.path.exists(BINDING_PATH):
                raise RuntimeError(f"native binding missing at {BINDING_PATH}; build it with "
                                   "`python -m post_weight_quantization_layer_b200.build`")
            from .build import binding_abi, built_abi  # imports torch, whose libraries the binding links against
            if built_abi() != binding_abi():
                raise RuntimeError(f"the native binding was built for {built_abi()}, this is {binding_abi()}; build it "
                                   "again with `python -m post_weight_quantization_layer_b200.build`")
            spec = importlib.util.spec_from_file_location("_binding", BINDING_PATH)
            module = importlib.util.module_from_spec(spec)
            spec.loader.exec_module(module)
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(f"native GPTQ library missing at {LIB_PATH}")
            module.open(LIB_PATH)
            _binding = module
    return _binding


class _NoFront:
    """Stands where the front cannot be loaded: leaves every call to the wrappers."""

    rotary = cache_write = cache_read = paged_attention = staticmethod(lambda *args: None)


_front = None


def front():
    """``binding()`` for the wrappers of the serving operators, which can call the native library without it, some 10
    us slower: where it cannot be loaded, one warning and a stand-in."""
    global _front
    if _front is None:
        try:
            _front = binding()
        except (RuntimeError, ImportError) as e:
            warnings.warn(f"serving calls go through ctypes: {e}", RuntimeWarning, stacklevel=3)
            _front = _NoFront
    return _front


def declared_symbols():
    """Names of the functions declared in include/gptq.h."""
    with open(HEADER) as f:
        text = f.read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(gptq_[a-z_]+)\s*\(", text)))
