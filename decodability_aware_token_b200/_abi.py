"""ctypes mirror of include/focus.h (argument marshalling only)."""
import ctypes as C
import importlib.util
import os
import struct
import sysconfig

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libfocus.so")
MARSHAL_PATH = os.path.join(os.path.dirname(LIB_PATH), "_marshal.so")
MARSHAL_STAMP = os.path.join(os.path.dirname(LIB_PATH), "_marshal.abi")  # what _marshal.so was built for (build.py)

FOCUS_OK = 0
FOCUS_ERR_INVALID_ARG = -1
FOCUS_ERR_LIMITS = -2
FOCUS_ERR_CUDA = -3
FOCUS_ERR_TIMEOUT = -4
FOCUS_ERR_DEVICE_BOUNDS = -5
FOCUS_ERR_UNSUPPORTED = -6
FOCUS_ERR_NO_MEMORY = -7

FOCUS_DEVERR_TOKEN_ID = 0x1
FOCUS_DEVERR_PAGE_ID = 0x2
FOCUS_DEVERR_PREFIX = 0x4
FOCUS_DEVERR_TIMEOUT = 0x8
FOCUS_DEVERR_FORCED_SET = 0x10
FOCUS_DEVERR_ROWS = 0x20

FOCUS_DTYPE_F32 = 0
FOCUS_DTYPE_BF16 = 1

# every symbol include/focus.h declares (checked by the CPU tests)
EXPORTED = ("focus_init", "focus_step", "focus_destroy", "focus_status_string", "focus_get_device_error",
            "focus_workspace_bytes", "focus_last_step_launches", "focus_profile_begin", "focus_profile_end",
            "focus_lm_head_conf_noalloc", "focus_commit_block", "focus_decode_block", "focus_probe_wait_timeout",
            "focus_chunk_init", "focus_chunk_destroy", "focus_chunk_workspace_bytes", "focus_chunk_get_device_error",
            "focus_chunk_plan_rows", "focus_chunk_qk_norm_rope", "focus_chunk_attention", "focus_prefill")

KERNEL_CLASSES = ("embed_norm", "qkv_finalize", "attn_score", "attn_ragged", "row_norm", "select", "decode",
                  "gemm_full_qkv", "gemm_full_o", "gemm_full_gateup", "gemm_full_down",
                  "gemm_qkv", "gemm_o", "gemm_gateup", "gemm_down", "gemm_lmhead")


class ModelCfg(C.Structure):
    _fields_ = [("n_layers", C.c_int32), ("hidden", C.c_int32), ("n_q_heads", C.c_int32), ("n_kv_heads", C.c_int32),
                ("head_dim", C.c_int32), ("ffn", C.c_int32), ("vocab", C.c_int32), ("rms_eps", C.c_float),
                ("rope_theta", C.c_float), ("dtype", C.c_int32)]


class Weights(C.Structure):
    _fields_ = [("embed", C.c_void_p), ("final_norm", C.c_void_p), ("lm_head", C.c_void_p),
                ("wqkv", C.POINTER(C.c_void_p)), ("wo", C.POINTER(C.c_void_p)), ("wgate", C.POINTER(C.c_void_p)),
                ("wup", C.POINTER(C.c_void_p)), ("wdown", C.POINTER(C.c_void_p)),
                ("attn_norm", C.POINTER(C.c_void_p)), ("mlp_norm", C.POINTER(C.c_void_p))]


class Limits(C.Structure):
    _fields_ = [("max_requests", C.c_int32), ("max_block", C.c_int32), ("max_keep", C.c_int32),
                ("max_pages_per_req", C.c_int32)]


class Batch(C.Structure):
    _fields_ = [("n_requests", C.c_int32), ("block_size", C.c_int32), ("page_size", C.c_int32),
                ("n_pages", C.c_int32), ("block_tokens", C.c_void_p), ("mask", C.c_void_p),
                ("prefix_len", C.c_void_p), ("page_table", C.c_void_p), ("kv_pool", C.c_void_p), ("ibc", C.c_void_p)]


class Params(C.Structure):
    _fields_ = [("tau", C.c_float), ("alpha", C.c_float), ("conf_threshold", C.c_float),
                ("forced_keep_frac", C.c_float), ("k_min", C.c_int32), ("k_max", C.c_int32),
                ("forced_keep_idx", C.c_void_p), ("forced_keep_count", C.c_void_p)]


class StepOut(C.Structure):
    _fields_ = [("keep_count", C.c_void_p), ("retained_idx", C.c_void_p), ("row_offsets", C.c_void_p),
                ("decoded_ids", C.c_void_p), ("conf", C.c_void_p), ("top_id", C.c_void_p),
                ("importance", C.c_void_p), ("hidden", C.c_void_p)]


class ChunkCfg(C.Structure):
    _fields_ = [("n_layers", C.c_int32), ("n_q_heads", C.c_int32), ("n_kv_heads", C.c_int32), ("head_dim", C.c_int32),
                ("dtype", C.c_int32), ("rope_theta", C.c_float)]


class ChunkLimits(C.Structure):
    _fields_ = [("max_requests", C.c_int32), ("max_pages_per_req", C.c_int32)]


class ChunkPlanArgs(C.Structure):
    _fields_ = [("n_requests", C.c_int32), ("max_rows", C.c_int32), ("page_size", C.c_int32), ("n_pages", C.c_int32),
                ("n_free", C.c_int32), ("prefix_len", C.c_void_p), ("new_len", C.c_void_p), ("page_table", C.c_void_p),
                ("free_pages", C.c_void_p), ("free_head", C.c_void_p), ("row_offsets", C.c_void_p),
                ("kv_len", C.c_void_p), ("row_req", C.c_void_p), ("row_pos", C.c_void_p), ("row_slot", C.c_void_p),
                ("free_next", C.c_void_p)]


class ChunkQkArgs(C.Structure):
    _fields_ = [("rows", C.c_int32), ("layer", C.c_int32), ("page_size", C.c_int32), ("n_pages", C.c_int32),
                ("eps", C.c_float), ("q_stride", C.c_int64), ("k_stride", C.c_int64), ("v_stride", C.c_int64),
                ("out_stride", C.c_int64), ("q", C.c_void_p), ("k", C.c_void_p), ("v", C.c_void_p),
                ("q_norm", C.c_void_p), ("k_norm", C.c_void_p), ("row_pos", C.c_void_p), ("row_slot", C.c_void_p),
                ("q_out", C.c_void_p), ("kv_pool", C.c_void_p)]


class ChunkAttnArgs(C.Structure):
    _fields_ = [("n_requests", C.c_int32), ("rows", C.c_int32), ("max_new", C.c_int32), ("page_size", C.c_int32),
                ("n_pages", C.c_int32), ("layer", C.c_int32), ("mask_block", C.c_int32), ("scale", C.c_float),
                ("q_stride", C.c_int64), ("out_stride", C.c_int64), ("q", C.c_void_p), ("kv_pool", C.c_void_p),
                ("row_offsets", C.c_void_p), ("kv_len", C.c_void_p), ("page_table", C.c_void_p), ("out", C.c_void_p)]


class PrefillArgs(C.Structure):
    _fields_ = [("plan", C.POINTER(ChunkPlanArgs)), ("tokens", C.c_void_p), ("max_new", C.c_int32),
                ("mask_block", C.c_int32), ("kv_pool", C.c_void_p), ("q_norm", C.POINTER(C.c_void_p)),
                ("k_norm", C.POINTER(C.c_void_p)), ("hidden", C.c_void_p)]


# The chunk operators' argument structs as packed bytes (native alignment): a call builds one bytes object instead of
# setting a field at a time, which costs more host time than a small kernel takes.
PLAN_PACK = struct.Struct("@5i11P")
QK_PACK = struct.Struct("@4if4q9P")
ATTN_PACK = struct.Struct("@7if2q6P")

_lib = None
_enqueue = None
_marshal = None


def load_enqueue():
    """(plan, qk, attention) of the chunk operators, called with a context, packed arguments and a stream.
    They only check and enqueue, so they keep the GIL: releasing it costs more than it gives here."""
    global _enqueue
    if _enqueue is None:
        load()
        lib = C.PyDLL(LIB_PATH)
        fns = (lib.focus_chunk_plan_rows, lib.focus_chunk_qk_norm_rope, lib.focus_chunk_attention)
        for fn in fns:
            fn.argtypes = [C.c_void_p, C.c_char_p, C.c_void_p]
            fn.restype = C.c_int
        _enqueue = fns
    return _enqueue


def marshal_abi():
    """The interfaces _marshal.so is compiled against: torch, its C++ ABI, the Python ABI."""
    import torch
    return f"torch {torch.__version__}, cxx11 abi {int(torch._C._GLIBCXX_USE_CXX11_ABI)}, {sysconfig.get_config_var('SOABI')}"


def marshal_stamp():
    """marshal_abi() at the time _marshal.so was built, None if it is not known."""
    try:
        with open(MARSHAL_STAMP) as f:
            return f.read().strip()
    except OSError:
        return None


def load_marshal():
    """The extension that reads the chunk operators' tensors in C++ (csrc/marshal.cpp) and the addresses of the three
    entry points, for it to call.  ImportError if it was not built, or was built for another torch or Python."""
    global _marshal
    if _marshal is None:
        import torch  # (its libraries have to be loaded first)
        lib = load()
        if not os.path.exists(MARSHAL_PATH):
            raise ImportError(f"{MARSHAL_PATH} is missing: build it with `python -m decodability_aware_token_b200.build`")
        if marshal_stamp() not in (None, marshal_abi()):  # (before it is loaded: it might not even link)
            raise ImportError(f"{MARSHAL_PATH} was built for {marshal_stamp()}, this is {marshal_abi()}: rebuild it with "
                              "`python -m decodability_aware_token_b200.build`")
        spec = importlib.util.spec_from_file_location(__package__ + "._marshal", MARSHAL_PATH)
        mod = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(mod)
        if mod.torch_version != torch.__version__.split("+")[0]:
            raise ImportError(f"{MARSHAL_PATH} was built for torch {mod.torch_version}: rebuild it")
        addr = [C.cast(getattr(lib, n), C.c_void_p).value
                for n in ("focus_chunk_plan_rows", "focus_chunk_qk_norm_rope", "focus_chunk_attention")]
        _marshal = mod, addr
    return _marshal


def load():
    """Load libfocus.so; raises ImportError if it was not built (there is no fallback path)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with `python -m decodability_aware_token_b200.build`")
    lib = C.CDLL(LIB_PATH)
    lib.focus_init.argtypes = [C.POINTER(ModelCfg), C.POINTER(Weights), C.POINTER(Limits), C.POINTER(C.c_void_p)]
    lib.focus_init.restype = C.c_int
    lib.focus_step.argtypes = [C.c_void_p, C.POINTER(Batch), C.POINTER(Params), C.POINTER(StepOut), C.c_void_p]
    lib.focus_step.restype = C.c_int
    lib.focus_destroy.argtypes = [C.c_void_p]
    lib.focus_destroy.restype = C.c_int
    lib.focus_status_string.argtypes = [C.c_int]
    lib.focus_status_string.restype = C.c_char_p
    lib.focus_get_device_error.argtypes = [C.c_void_p, C.POINTER(C.c_int32)]
    lib.focus_get_device_error.restype = C.c_int
    lib.focus_workspace_bytes.argtypes = [C.POINTER(ModelCfg), C.POINTER(Limits)]
    lib.focus_workspace_bytes.restype = C.c_size_t
    lib.focus_last_step_launches.argtypes = [C.c_void_p]
    lib.focus_last_step_launches.restype = C.c_int
    lib.focus_profile_begin.argtypes = [C.c_void_p, C.c_int, C.c_int]
    lib.focus_profile_begin.restype = C.c_int
    lib.focus_profile_end.argtypes = [C.c_void_p, C.POINTER(C.c_float), C.POINTER(C.c_int32)]
    lib.focus_profile_end.restype = C.c_int
    lib.focus_lm_head_conf_noalloc.argtypes = [C.c_void_p, C.c_int32, C.c_int32, C.c_void_p, C.c_void_p, C.c_int32,
                                               C.c_float, C.c_void_p, C.c_void_p, C.c_void_p]
    lib.focus_lm_head_conf_noalloc.restype = C.c_int
    lib.focus_probe_wait_timeout.argtypes = [C.c_void_p, C.c_void_p]
    lib.focus_probe_wait_timeout.restype = C.c_int
    lib.focus_commit_block.argtypes = [C.c_void_p, C.POINTER(Batch), C.c_void_p]
    lib.focus_commit_block.restype = C.c_int
    lib.focus_decode_block.argtypes = [C.c_void_p, C.POINTER(Batch), C.POINTER(Params), C.c_int32, C.POINTER(StepOut),
                                       C.POINTER(C.c_int32), C.c_void_p]
    lib.focus_decode_block.restype = C.c_int
    lib.focus_chunk_init.argtypes = [C.POINTER(ChunkCfg), C.POINTER(ChunkLimits), C.POINTER(C.c_void_p)]
    lib.focus_chunk_init.restype = C.c_int
    lib.focus_chunk_destroy.argtypes = [C.c_void_p]
    lib.focus_chunk_destroy.restype = C.c_int
    lib.focus_chunk_workspace_bytes.argtypes = [C.POINTER(ChunkCfg), C.POINTER(ChunkLimits)]
    lib.focus_chunk_workspace_bytes.restype = C.c_size_t
    lib.focus_chunk_get_device_error.argtypes = [C.c_void_p, C.POINTER(C.c_int32)]
    lib.focus_chunk_get_device_error.restype = C.c_int
    lib.focus_chunk_plan_rows.argtypes = [C.c_void_p, C.POINTER(ChunkPlanArgs), C.c_void_p]
    lib.focus_chunk_plan_rows.restype = C.c_int
    lib.focus_chunk_qk_norm_rope.argtypes = [C.c_void_p, C.POINTER(ChunkQkArgs), C.c_void_p]
    lib.focus_chunk_qk_norm_rope.restype = C.c_int
    lib.focus_chunk_attention.argtypes = [C.c_void_p, C.POINTER(ChunkAttnArgs), C.c_void_p]
    lib.focus_chunk_attention.restype = C.c_int
    lib.focus_prefill.argtypes = [C.c_void_p, C.c_void_p, C.POINTER(PrefillArgs), C.c_void_p]
    lib.focus_prefill.restype = C.c_int
    _lib = lib
    return lib
