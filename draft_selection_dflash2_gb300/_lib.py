"""Loaders of libdflash2.so (the CUDA kernels behind the C ABI; ctypes) and of
_dflash2_bind.so (compiled argument marshalling for the calls whose kernels are shortest).

There is no fallback: if the library has not been built for this machine,
loading raises immediately.
"""
import ctypes
import importlib.util
import os
import re

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libdflash2.so")
BIND_PATH = os.path.join(HERE, "_dflash2_bind.so")
HEADER = os.path.join(os.path.dirname(HERE), "include", "dflash2.h")

P = ctypes.c_void_p
I64 = ctypes.c_int64
U64 = ctypes.c_uint64
I32 = ctypes.c_int
U32P = ctypes.POINTER(ctypes.c_uint32)
F32 = ctypes.c_float
SZ = ctypes.c_size_t

# name -> (restype, argtypes); mirrors include/dflash2.h
SIGNATURES = {
    "dflash2_version": (I32, []),
    "dflash2_status_string": (ctypes.c_char_p, [I32]),
    "dflash2_create": (I32, [I32, ctypes.POINTER(P)]),
    "dflash2_destroy": (I32, [P]),
    "dflash2_num_sms": (I32, [P]),
    "dflash2_get_device_error": (I32, [P, P, U32P, I32]),
    "dflash2_topk": (I32, [P, P, I64, I64, I64, I32, P, P, P]),
    "dflash2_pair_scores_workspace": (SZ, [P, I64, I64, I64]),
    "dflash2_pair_scores": (I32, [P, P, P, P, P, P, P, P, P, I64, I64, I64, I64, P, P, P, SZ, P]),
    "dflash2_walk": (I32, [P, P, P, I64, I64, F32, U64, U64, P, P, P, P]),
    "dflash2_walk_viterbi": (I32, [P, P, P, I64, I64, P, P, P, P]),
    "dflash2_selector_eval": (I32, [P, P, P, I64, I64, P, P, P, P]),
    "dflash2_conv2tap_workspace": (SZ, [P, I64, I64, I64]),
    "dflash2_conv2tap": (I32, [P, P, P, P, P, P, P, P, I64, I64, I64, P, I32, P, SZ, P]),
    "dflash2_verify_workspace": (SZ, [P, I64, I64, I64]),
    "dflash2_verify": (I32, [P, P, I64, P, P, P, P, I64, I64, I64, F32, U64, U64, P, P, P, SZ, P]),
    "dflash2_lmhead_topk_workspace": (SZ, [P, I64, I64, I64]),
    "dflash2_lmhead_topk": (I32, [P, P, P, I64, I64, I64, P, P, P, SZ, P]),
    "dflash2_lmhead_topk_gate": (I32, [P, P, P, P, P, I64, I64, I64, P, P, P, P, SZ, P]),
    "dflash2_pair_scores_proj_workspace": (SZ, [P, I64, I64]),
    "dflash2_gemm_conv2tap_workspace": (SZ, [P, I64, I64, I64]),
    "dflash2_gemm_conv2tap": (I32, [P, P, P, P, P, P, P, P, P, I64, I64, I64, I64, P, SZ, P, I32, P]),
    "dflash2_pair_scores_proj": (I32, [P, P, P, P, P, P, P, P, I64, I64, I64, I64, P, SZ, P, P]),
    "dflash2_lmhead_topk_noalloc": (I32, [P, P, P, I64, I64, I64, P, P, P]),
    "dflash2_tree_attention_workspace": (SZ, [P, I64, I64, I64, I64, I64]),
    "dflash2_tree_attention": (I32, [P, P, I64, I64, I64, P, P, P, P, I64, I64, I64, P, I64, I64, I64, F32, P, P, P,
                                     SZ, P]),
    "dflash2_cache_commit": (I32, [P, P, P, I64, I64, I64, P, P, P, P, I64, I64, P, I64, P, P]),
    "dflash2_cache_scores": (I32, [P, P, I64, I64, I64, P, P, P, P, P, I64, I64, I64, F32, P, I64, P]),
    "dflash2_cache_evict": (I32, [P, P, I64, P, P, P, I64, I64, I64, P, P, P, I64, P]),
    "dflash2_selftest_wait_timeout": (I32, [P, U64, P, P]),
}


class KvCacheStruct(ctypes.Structure):
    """dflash2_kv_cache."""
    _fields_ = [("k", P), ("v", P), ("num_pages", I64), ("page_size", I64), ("heads", I64), ("head_dim", I64),
                ("page_stride", I64), ("token_stride", I64), ("head_stride", I64), ("block_table", P),
                ("max_pages", I64), ("table_ld", I64)]


_lib = None


def declared_functions(header: str = HEADER):
    """Function names declared in the public header."""
    text = open(header).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(dflash2_[a-z_0-9]+)\s*\(", text)))


def load():
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it first "
                "(python -c 'import __graft_entry__ as g; g.build()')")
        lib = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


_bind = None


def load_bind():
    """The compiled half of the binding, calling the loaded library's entry points."""
    global _bind
    if _bind is None:
        import torch  # (the module's symbols come from torch's libraries)
        lib = load()
        again = "build it (python -c 'import __graft_entry__ as g; g.build()')"
        if not os.path.exists(BIND_PATH):
            raise RuntimeError(f"{BIND_PATH} is missing: {again}")
        try:
            spec = importlib.util.spec_from_file_location("_dflash2_bind", BIND_PATH)
            mod = importlib.util.module_from_spec(spec)
            spec.loader.exec_module(mod)
        except ImportError as e:
            raise RuntimeError(f"{BIND_PATH} does not load with torch {torch.__version__}: {again}") from e
        if mod.torch_version != torch.__version__:
            raise RuntimeError(f"{BIND_PATH} was built for torch {mod.torch_version}, not {torch.__version__}: {again}")
        mod.init(*(ctypes.cast(getattr(lib, "dflash2_" + f), P).value
                   for f in ("tree_attention", "cache_commit", "cache_scores", "cache_evict")))
        _bind = mod
    return _bind
