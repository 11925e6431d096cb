"""ctypes binding of libmoeq8.so (the in-tree HIP build).  No fallback: if the
library is missing or does not load, every call raises."""

from __future__ import annotations

import ctypes
import importlib.util
import os

from .build import BINDING_PATH, LIB_PATH

c_i32, c_i64, c_u32, c_u64 = ctypes.c_int32, ctypes.c_int64, ctypes.c_uint32, ctypes.c_uint64
c_vp, c_fp, c_size = ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t
c_f64 = ctypes.c_double



class KvCache(ctypes.Structure):
    """struct moeq8_kv_cache"""
    _fields_ = [("k", c_vp), ("k_scale", c_vp), ("v", c_vp), ("v_scale", c_vp),
                *((n, c_i64) for n in ("n_pages", "n_heads", "page_size", "d", "page_stride", "head_stride",
                                       "token_stride", "scale_page_stride", "scale_head_stride"))]


c_cache = ctypes.POINTER(KvCache)

# name -> (restype, argtypes); one entry per declaration in include/moeq8.h and
# include/moeq8_synth.h
SIGNATURES = {
    "moeq8_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "moeq8_abi_version": (ctypes.c_int, []),
    "q8_1_quantize_rows": (ctypes.c_int, [c_vp, c_i64, c_i64, c_i64, c_vp, c_vp]),
    "q8_0_quantize_rows": (ctypes.c_int, [c_vp, c_i64, c_i64, c_i64, c_vp, c_vp]),
    "q8_0_pack64_rows": (ctypes.c_int, [c_vp, c_i64, c_i64, c_i64, c_vp, c_i64, c_vp]),
    "q8_0_pack64_rounds": (ctypes.c_int, [c_vp, c_i64, c_i64, c_i64, c_vp, c_vp]),
    "q4_pack64_rows": (ctypes.c_int, [c_vp, c_i64, c_i64, c_i64, c_vp, c_i64, c_vp]),
    "q8_0_pack_gemm_rows": (ctypes.c_int, [c_vp, c_i64, c_i64, c_i64, c_vp, c_i64, c_vp]),
    "mmvq_q8_0": (ctypes.c_int, [c_vp, c_i64, c_i64, c_i64, c_i64, c_vp, c_i64, c_vp, c_vp]),
    "mmvq_q8_0_glu_pair": (ctypes.c_int, [c_vp, c_vp, c_i64, c_i64, c_i64, c_i64, c_vp, c_i64,
                                          c_vp, c_vp, c_vp, c_vp]),
    "swiglu_ds4": (ctypes.c_int, [c_vp, c_vp, c_i64, c_vp, c_vp]),
    "moe_grouping_bytes": (c_size, [c_i64, c_i32]),
    "moe_router_scores": (ctypes.c_int, [c_vp, c_i64, c_vp, c_vp]),
    "moe_route_topk": (ctypes.c_int, [c_vp, c_vp, c_vp, c_i64, c_i64, c_i64, c_i32, c_vp, c_vp,
                                      c_vp, c_vp]),
    "moe_grouped_mmvq": (ctypes.c_int, [c_i32, c_vp, c_vp, c_i64, c_i64, c_i64, c_i64, c_i64,
                                        c_vp, c_vp, c_i64, c_i32, c_vp, c_vp]),
    "moe_grouped_gemm": (ctypes.c_int, [c_i32, c_vp, c_vp, c_i64, c_i64, c_i64, c_i64, c_i64,
                                        c_vp, c_vp, c_i64, c_i32, c_vp, c_vp]),
    "moe_grouped_mmvq_ex": (ctypes.c_int, [c_i32, c_vp, c_vp, c_i64, c_i64, c_i64, c_i64, c_i64,
                                           c_vp, c_i64, c_vp, c_i64, c_i32, c_vp, c_vp, c_vp, c_i64,
                                           c_i64, c_i64, c_i64, c_vp, c_i64, c_vp, c_vp]),
    "moe_route_topk_quantize": (ctypes.c_int, [c_vp, c_i64, c_i64, c_vp, c_vp, c_vp, c_vp, c_i64,
                                               c_i64, c_i64, c_i32, c_vp, c_vp, c_vp, c_vp]),
    "moe_grouped_ffn_p64": (ctypes.c_int, [c_vp, c_vp, c_vp, c_i64, c_i64, c_i64, c_i64, c_i64, c_vp,
                                           c_vp, c_i64, c_i32, c_vp, c_vp, c_vp, c_vp, c_i64, c_i64,
                                           c_vp, c_vp, c_vp, c_vp]),
    "moe_grouped_ffn_p64_noalloc": (ctypes.c_int, [c_vp, c_vp, c_vp, c_i64, c_i64, c_i64, c_i64, c_i64, c_vp,
                                                   c_vp, c_i64, c_i32, c_vp, c_vp, c_vp, c_i64, c_i64,
                                                   c_vp, c_vp, c_vp]),
    "moe_combine": (ctypes.c_int, [c_vp, c_vp, c_vp, c_i64, c_i32, c_i64, c_vp, c_vp]),
    "moe_combine_shared": (ctypes.c_int, [c_vp, c_vp, c_vp, c_i64, c_i32, c_i64, c_vp, c_vp, c_vp]),
    "q8_block_encode": (ctypes.c_int, [c_vp, c_i64, c_i64, c_i64, c_vp, c_vp]),
    "q8_block_decode_sum": (ctypes.c_int, [c_vp, c_i32, c_i64, c_i64, c_i64, c_vp, c_i64, c_vp]),
    "q4_quantize_rows": (ctypes.c_int, [c_vp, c_i64, c_i64, c_i64, c_vp, c_vp]),
    "mmvq_q4": (ctypes.c_int, [c_vp, c_i64, c_i64, c_i64, c_i64, c_vp, c_i64, c_vp, c_vp]),
    "mmvq_q4_glu_pair": (ctypes.c_int, [c_vp, c_vp, c_i64, c_i64, c_i64, c_i64, c_vp, c_i64,
                                        c_vp, c_vp, c_vp, c_vp]),
    "moe_grouped_mmvq_q4": (ctypes.c_int, [c_i32, c_vp, c_vp, c_i64, c_i64, c_i64, c_i64, c_i64,
                                           c_vp, c_i64, c_vp, c_i64, c_i32, c_vp, c_vp]),
    "moe_grouping_bytes_wide": (c_size, [c_i64, c_i32]),
    "moe_route_topk_wide": (ctypes.c_int, [c_vp, c_vp, c_vp, c_i64, c_i64, c_i64, c_i32, c_vp, c_vp,
                                           c_vp]),
    "moe_group_routes": (ctypes.c_int, [c_vp, c_i64, c_i32, c_i64, c_vp, c_vp]),
    "rms_norm_q8": (ctypes.c_int, [c_vp, c_i64, c_vp, c_i64, c_vp, c_i64, c_vp, c_i32, c_i64, c_i64, c_f64,
                                   c_vp, c_i64, c_vp, c_vp, c_vp]),
    "i8_quantize_rows": (ctypes.c_int, [c_vp, c_i32, c_i64, c_i64, c_i64, c_vp, c_i64, c_vp, c_vp]),
    "gemm_i8": (ctypes.c_int, [c_vp, c_i64, c_vp, c_vp, c_i64, c_vp, c_vp, c_i64, c_i64, c_i64, c_i32, c_vp,
                               c_i64, c_vp]),
    "logits_process": (ctypes.c_int, [c_vp, c_i64, c_i32, c_i64, c_i64, c_vp, c_i64, c_vp, c_vp, c_vp, c_vp,
                                      c_vp, c_vp, c_vp, c_vp, c_i64, c_vp, c_vp, c_i64, c_vp, c_i64, c_vp]),
    "kv_cache_write_i8": (ctypes.c_int, [c_vp, c_i64, c_i64, c_vp, c_i64, c_i64, c_i32, c_i64, c_vp, c_cache, c_vp]),
    "kv_cache_read_i8": (ctypes.c_int, [c_cache, c_vp, c_i64, c_i32, c_vp, c_i64, c_i64, c_vp, c_i64, c_i64, c_vp]),
    "paged_attention_workspace_bytes": (c_size, [c_i64, c_i64, c_i64, c_i64, c_i64, c_i64]),
    "paged_attention_i8": (ctypes.c_int, [c_vp, c_i64, c_i64, c_i64, c_i32, c_i64, c_i64, c_i64, c_cache, c_vp, c_i64,
                                          c_i64, c_vp, c_i64, c_f64, c_vp, c_i64, c_i64, c_i64, c_vp, c_size, c_vp]),
    "logits_sample_workspace_bytes": (c_size, [c_i64, c_i64]),
    "logits_sample": (ctypes.c_int, [c_vp, c_i64, c_i32, c_i64, c_i64, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp,
                                     c_size, c_vp]),
    "moeq8_synth_stream_key": (c_u64, [c_u32, c_u32, c_u32, c_u32]),
    "moeq8_synth_q8_0_fill": (ctypes.c_int, [c_vp, c_i64, c_i64, c_i64, c_u32, c_u32, c_u32,
                                             c_u32, c_vp]),
    "moeq8_stream_read": (ctypes.c_int, [c_vp, c_i64, c_vp, c_vp]),
    "moeq8_stream_read_shape": (ctypes.c_int, [c_vp, c_i64, c_i64, c_vp, c_vp]),
}

_LIB = None


class MoeQ8Error(RuntimeError):
    def __init__(self, name: str, status: int):
        msg = lib().moeq8_status_string(status).decode()
        super().__init__(f"{name} failed with status {status}: {msg}")
        self.status = status


def lib_path() -> str:
    return os.environ.get("MOEQ8_LIB", LIB_PATH)


def lib():
    """Load libmoeq8.so once; raise if it is not built."""
    global _LIB
    if _LIB is None:
        path = lib_path()
        if not os.path.exists(path):
            raise RuntimeError(f"libmoeq8 is not built ({path} missing): run __graft_entry__.build() "
                               "or python -m quantized_moe_expert_q8_amd.build")
        # torch first: its HIP runtime (same soname) then serves this library too,
        # so torch's streams and allocations are valid here
        import torch  # noqa: F401
        so = ctypes.CDLL(path)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(so, name)
            fn.restype = res
            fn.argtypes = args
        _LIB = so
    return _LIB


def load_binding():
    """The compiled torch side of the operators around the expert layer."""
    if not os.path.exists(BINDING_PATH):
        raise RuntimeError(f"the torch binding is not built ({BINDING_PATH} missing): run __graft_entry__.build() "
                           "or python -m quantized_moe_expert_q8_amd.build")
    import torch  # noqa: F401  (its libraries, which the binding's symbols are in)
    spec = importlib.util.spec_from_file_location(f"{__package__}._binding", BINDING_PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def call(name: str, *args) -> int:
    st = getattr(lib(), name)(*args)
    if st != 0:
        raise MoeQ8Error(name, st)
    return st
