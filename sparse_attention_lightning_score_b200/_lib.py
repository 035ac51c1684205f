"""ctypes loader for ``libli.so`` (the C ABI declared in ``include/li.h``).

The library must have been built (``python -m sparse_attention_lightning_score_b200.build``);
there is no fallback: loading fails loudly when the shared object is missing.
"""
from __future__ import annotations

import ctypes
import os

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libli.so")

LI_OK, LI_ERR_INVALID_ARG, LI_ERR_UNSUPPORTED, LI_ERR_CUDA, LI_ERR_TIMEOUT, LI_ERR_BOUNDS = range(6)
LI_DTYPE_F32, LI_DTYPE_BF16, LI_DTYPE_E4M3, LI_DTYPE_E2M1 = 0, 1, 2, 3
LI_TOPK_MAX_LEN = 262144
LI_HS_NOALLOC_MAX_SCRATCH_FLOATS = 1048576
LI_OP_SCORE, LI_OP_TOPK, LI_OP_HS, LI_OP_DECODE_SELECT = range(4)
LI_BLOCK_TABLE_MAX_REQUESTS = 16384
LI_KV4_ROW_BYTES = 416
LI_ROPE_PLAIN, LI_ROPE_LINEAR, LI_ROPE_YARN = range(3)
LI_ROPE_INTERLEAVED, LI_ROPE_HALF = range(2)
LI_ROPE_MAX_TENSORS = 4

vp = ctypes.c_void_p
i32 = ctypes.c_int
i64 = ctypes.c_int64
sz = ctypes.c_size_t


class ScoreDesc(ctypes.Structure):
    _fields_ = [("rows", i32), ("heads", i32), ("dim", i32), ("max_len", i32), ("causal", i32),
                ("causal_offset", i32), ("q_dtype", i32), ("k_dtype", i32), ("tokens_per_request", i32)]


class AttnDesc(ctypes.Structure):
    _fields_ = [("rows", i32), ("heads", i32), ("requests", i32), ("num_pages", i32), ("page_size", i32),
                ("max_blocks", i32), ("cache_dtype", i32), ("scale", ctypes.c_float)]


class RopeTensor(ctypes.Structure):
    _fields_ = [("x", vp), ("out", vp), ("x_token_stride", i64), ("x_head_stride", i64), ("out_token_stride", i64),
                ("out_head_stride", i64), ("heads", i32), ("dim", i32), ("offset", i32), ("layout", i32),
                ("dtype", i32)]


# name -> (restype, argtypes); every symbol declared in include/li.h
SIGNATURES = {
    "li_status_string": (ctypes.c_char_p, [i32]),
    "li_get_last_error": (i32, []),
    "li_quantize_query": (i32, [vp, vp, i32, i32, i32, vp, vp, vp, vp]),
    "li_index_score": (i32, [vp, vp, vp, vp, i64, vp, vp, i64, ctypes.POINTER(ScoreDesc), vp, sz, vp]),
    "li_index_score_workspace": (sz, [ctypes.POINTER(ScoreDesc)]),
    "li_workspace_size": (sz, [i32, i32, i32, i32]),
    "li_topk": (i32, [vp, i64, vp, i32, i32, i32, i32, i32, vp, vp, vp]),
    "li_decode_select": (i32, [vp, vp, vp, vp, i64, vp, vp, i64, ctypes.POINTER(ScoreDesc), i32, vp, vp, vp, sz,
                               vp]),
    "li_decode_select_workspace": (sz, [ctypes.POINTER(ScoreDesc)]),
    "li_decode_select_score": (i32, [vp, vp, vp, vp, i64, vp, vp, i64, ctypes.POINTER(ScoreDesc), vp, sz, vp]),
    "li_decode_select_finish": (i32, [vp, i64, vp, ctypes.POINTER(ScoreDesc), i32, vp, vp, vp, sz, vp]),
    "li_decode_score_hist": (i32, [vp, vp, vp, vp, i64, vp, vp, i64, ctypes.POINTER(ScoreDesc), vp, vp]),
    "li_topk_hist": (i32, [vp, i64, vp, i32, i32, i32, vp, vp, vp, i32, vp]),
    "li_absorb_query": (i32, [vp, vp, vp, i32, i32, i32, i32, vp]),
    "li_latent_score": (i32, [vp, vp, vp, i64, vp, vp, i64, i32, i32, i32, i32, vp]),
    "li_latent_score_hist": (i32, [vp, vp, vp, i64, vp, vp, i64, i32, i32, i32, i32, vp, vp]),
    "li_absorb_query_layers": (i32, [vp, vp, vp, i32, i32, i32, i32, i32, vp]),
    "li_host_device_pointer": (i32, [vp, ctypes.POINTER(ctypes.c_void_p)]),
    "li_copy_from_host": (i32, [vp, vp, sz, vp]),
    "li_merge_shards": (i32, [vp, vp, i32, i32, i32, i64, i32, vp, vp, vp, sz, vp]),
    "li_merge_shards_workspace": (sz, [i32, i32, i32]),
    "li_latent_score_fp8": (i32, [vp, vp, vp, vp, i64, vp, vp, i64, i32, i32, i32, i32, vp, vp]),
    "li_hs_refine": (i32, [vp, i64, i64, vp, i32, i32, vp, vp, i32, i32, i32, i32, vp, vp, sz, vp]),
    "li_hs_refine_workspace": (sz, [i32, i32, i32]),
    "li_hs_refine_noalloc": (i32, [vp, i64, i64, vp, i32, i32, vp, vp, i32, i32, i32, i32, vp, vp]),
    "li_hs_refine_fp8": (i32, [vp, vp, i64, i64, vp, i32, i32, vp, vp, i32, i32, i32, i32, vp, vp, sz, vp]),
    "li_sparse_attention": (i32, [vp, vp, i64, i64, vp, i32, i32, i32, ctypes.c_float, vp, vp, sz, vp]),
    "li_sparse_attention_workspace": (sz, [i32, i32, i32]),
    "li_block_tables": (i32, [vp, vp, i32, vp, i32, i32, i32, vp, i32, vp, i32, vp, vp, vp, vp, vp, vp]),
    "li_rope_table": (i32, [i32, ctypes.c_double, i32, ctypes.c_double, i32, ctypes.c_double, ctypes.c_double, vp]),
    "li_rope": (i32, [ctypes.POINTER(RopeTensor), i32, i32, vp, vp, i32, ctypes.c_float, vp]),
    "li_kv4_write": (i32, [vp, i64, vp, i64, vp, i64, vp]),
    "li_kv4_read": (i32, [vp, i64, vp, i64, vp, vp]),
    "li_paged_sparse_attention": (i32, [vp, vp, vp, vp, vp, i32, ctypes.POINTER(AttnDesc), vp, vp, sz, vp]),
    "li_window_attention": (i32, [vp, vp, vp, vp, vp, i32, i32, i32, ctypes.POINTER(AttnDesc), vp, vp, sz, vp]),
    "li_paged_attention_workspace": (sz, [i32, i32, i32]),
    "li_graph_instantiate": (i32, [vp, i32, ctypes.POINTER(ctypes.c_void_p)]),
    "li_graph_launch": (i32, [vp, vp]),
    "li_graph_destroy": (i32, [vp]),
    "li_selftest_wait_timeout": (i32, [ctypes.c_uint64, vp]),
}

_lib = None


class LiError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} failed: {status_string(status)}")


def load() -> ctypes.CDLL:
    """Load libli.so once; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"libli.so not found at {LIB_PATH}; build it with "
                              "`python -m sparse_attention_lightning_score_b200.build`")
        lib = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            f = getattr(lib, name)
            f.restype = res
            f.argtypes = args
        _lib = lib
    return _lib


class _Binding:
    """The functions of ``_bind.so`` (csrc/bind.cpp), loaded at the first call of one; raises if it has
    not been built."""

    def __getattr__(self, name):
        try:
            from . import _bind
        except ImportError as e:
            raise ImportError("_bind.so does not load; build it with "
                              "`python -m sparse_attention_lightning_score_b200.build`") from e
        _bind.set_error(LiError)
        self.__dict__.update((n, f) for n, f in vars(_bind).items() if not n.startswith("_"))
        return self.__dict__[name]


bind = _Binding()


def status_string(status: int) -> str:
    return load().li_status_string(int(status)).decode()


def check(fn: str, status: int):
    if status != LI_OK:
        raise LiError(fn, status)
