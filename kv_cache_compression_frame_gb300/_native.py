"""ctypes view of libstatekv's C ABI (include/statekv.h).

Only argument marshalling lives here; every step of the prefill path runs in
the library's CUDA kernels.  Loading fails loudly if the library was not
built: there is no fallback implementation.
"""

from __future__ import annotations

import ctypes as C
import os
import struct

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libstatekv.so")

OK = 0
E_INVALID_ARG = -1
E_UNSUPPORTED = -2
E_CAPACITY = -3
E_OOM = -4
E_CUDA = -5
E_TIMEOUT = -6
E_DEVICE = -7

BF16 = 0
F32 = 1

KERNEL_ROPE_TABLE = 0
KERNEL_ROPE = 1
KERNEL_ATTENTION = 2
KERNEL_SELECT = 3
KERNEL_NAMES = ("rope_table", "rope", "attention", "select")

EXPORTS = (
    "statekv_status_string", "statekv_create", "statekv_destroy",
    "statekv_prefill_frame", "statekv_prefill_frame_host", "statekv_prefill_frames_host",
    "statekv_get_compressed", "statekv_get_detailed", "statekv_frame_index",
    "statekv_reset", "statekv_check_device_status", "statekv_get_scores",
    "statekv_get_rotated_query", "statekv_set_frame_index",
    "statekv_set_compressed", "statekv_profile_enable", "statekv_profile_read",
    "statekv_profile_kernels",
    "statekv_attend_scores_static", "statekv_decode", "statekv_text_tokens",
    "statekv_norm_rope", "statekv_tree_attention", "statekv_tree_attention_workspace",
    "statekv_append_accepted", "statekv_block_summaries",
    "statekv_sparse_attention",
    "statekv_set_qk_norm", "statekv_decode_tree", "statekv_accept", "statekv_decode_sparse",
    "statekv_paged_append", "statekv_paged_attention", "statekv_paged_attention_workspace",
    "statekv_attention_weights", "statekv_evict_rows", "statekv_verify_tree", "statekv_decode_prompt",
)

BLOCK = 64          # STATEKV_BLOCK


class Config(C.Structure):
    _fields_ = [
        ("num_streams", C.c_int32), ("num_layers", C.c_int32),
        ("num_q_heads", C.c_int32), ("num_kv_heads", C.c_int32),
        ("head_dim", C.c_int32), ("frame_tokens", C.c_int32),
        ("budget", C.c_int32), ("max_frames", C.c_int32),
        ("dtype", C.c_int32), ("device", C.c_int32),
        ("rope_theta", C.c_double), ("rope_alpha", C.c_double),
        ("rope_orig_ctx", C.c_int64), ("position_offset", C.c_int64),
        ("select_policy", C.c_int32),
    ]


class View(C.Structure):
    _fields_ = [("data", C.c_void_p), ("batch_stride", C.c_int64),
                ("head_stride", C.c_int64), ("token_stride", C.c_int64)]


def _struct(name: str, *groups) -> type:
    """A ctypes mirror of one of the header's argument structures."""
    fields = [(f, t) for t, names in groups for f in names.split()]
    return type(name, (C.Structure,), {"_fields_": fields})


NormRopeArgs = _struct(
    "NormRopeArgs", (View, "q k v q_out k_out v_out"),
    (C.c_void_p, "q_weight k_weight omega positions out_rows status"), (C.c_int64, "position0"),
    (C.c_int32, "position_stride position_layers batch layers q_heads kv_heads tokens head_dim "
                "out_capacity weight_rows dtype weight_dtype"), (C.c_float, "eps"))
TreeArgs = _struct(
    "TreeArgs", (View, "q out k_new v_new k_cache v_cache"),
    (C.c_void_p, "tree lengths status workspace"), (C.c_int64, "workspace_bytes"),
    (C.c_double, "scale"),
    (C.c_int32, "tree_stride length batch layers q_heads kv_heads tokens head_dim cache_rows"))
AppendArgs = _struct(
    "AppendArgs", (View, "k_new v_new k_cache v_cache"),
    (C.c_void_p, "path counts lengths new_lengths status"),
    (C.c_int32, "path_stride path_len length batch layers kv_heads tokens head_dim cache_rows dtype"))
SummaryArgs = _struct(
    "SummaryArgs", (View, "k_cache"), (C.c_void_p, "codes scales lengths status"),
    (C.c_int32, "length appended blocks batch layers kv_heads head_dim cache_rows"))

SparseArgs = _struct(
    "SparseArgs", (View, "q out k_cache v_cache"), (C.c_void_p, "codes scales lengths selected status"),
    (C.c_double, "scale"),
    (C.c_int32, "length top blocks batch layers q_heads kv_heads tokens head_dim cache_rows"))
_PAGED = "length table_stride table_pages num_pages page_rows "
PagedAppendArgs = _struct(
    "PagedAppendArgs", (View, "k_new v_new k_pages v_pages"),
    (C.c_void_p, "table lengths counts new_lengths status"),
    (C.c_int32, _PAGED + "batch layers kv_heads tokens head_dim dtype"))
PagedAttentionArgs = _struct(
    "PagedAttentionArgs", (View, "q out k_pages v_pages"),
    (C.c_void_p, "table lengths counts lse status workspace"), (C.c_int64, "workspace_bytes"),
    (C.c_double, "scale"), (C.c_int32, _PAGED + "batch layers q_heads kv_heads tokens head_dim"))
AttentionWeightsArgs = _struct(
    "AttentionWeightsArgs", (View, "q k_pages"),
    (C.c_void_p, "table lengths counts lse before out status"), (C.c_double, "scale"),
    (C.c_int32, _PAGED + "weight_rows batch layers q_heads kv_heads tokens head_dim"))
EvictArgs = _struct(
    "EvictArgs", (View, "k_pages v_pages k_out v_out"),
    (C.c_void_p, "table out_table lengths weights weights_out kept new_lengths status"),
    (C.c_int32, _PAGED + "weight_rows out_table_stride out_table_pages out_num_pages out_page_rows out_rows "
                "keep sinks recent batch layers kv_heads head_dim dtype"))
VerifyArgs = _struct(
    "VerifyArgs", (C.c_void_p, "target draft drafted tree uniforms path counts next status"),
    (C.c_int64, "target_stride target_row draft_stride draft_row"),
    (C.c_int32, "tree_stride sequences tokens vocab"))

# The same structures packed from flat values, a view as (pointer, batch, head,
# token stride): a fifth of the time it takes to fill a ctypes structure.
_V = "Pqqq"
PACK_NORM_ROPE = struct.Struct("@" + 6 * _V + "6Pq12if0q")
PACK_TREE = struct.Struct("@" + 6 * _V + "4Pqd9i0q")
PACK_APPEND = struct.Struct("@" + 4 * _V + "5P10i0q")
PACK_SUMMARY = struct.Struct("@" + _V + "4P8i0q")
PACK_SPARSE = struct.Struct("@" + 4 * _V + "5Pd10i0q")
PACK_PAGED_APPEND = struct.Struct("@" + 4 * _V + "5P11i0q")
PACK_PAGED_ATTENTION = struct.Struct("@" + 4 * _V + "6Pqd11i0q")
PACK_WEIGHTS = struct.Struct("@" + 2 * _V + "7Pd12i0q")
PACK_EVICT = struct.Struct("@" + 4 * _V + "8P19i0q")
PACK_VERIFY = struct.Struct("@9P4q4i0q")
# entry points that take such a packed structure and a stream; set by load()
PACKED = ("statekv_norm_rope", "statekv_tree_attention", "statekv_append_accepted",
          "statekv_block_summaries", "statekv_sparse_attention", "statekv_paged_append",
          "statekv_paged_attention", "statekv_attention_weights", "statekv_evict_rows", "statekv_verify_tree")
packed: dict = {}


class StateKVError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} ({status})")


_lib = None
_P = C.c_void_p
_PP = C.POINTER(C.c_void_p)


def load() -> C.CDLL:
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(
            f"{LIB_PATH} is missing: build it with "
            "`python -m kv_cache_compression_frame_gb300.build_lib`")
    lib = C.CDLL(LIB_PATH)
    h = _P
    sig = {
        "statekv_status_string": (C.c_char_p, [C.c_int]),
        "statekv_create": (C.c_int, [C.POINTER(Config), C.POINTER(h)]),
        "statekv_destroy": (C.c_int, [h]),
        "statekv_prefill_frame": (C.c_int, [h, _P, _P, _P, _P, _P]),
        "statekv_prefill_frame_host": (C.c_int, [h, _P, _P, _P, _P, _P]),
        "statekv_prefill_frames_host": (C.c_int, [h, C.c_int32, _P, _P, _P, _P, _P]),
        "statekv_get_compressed": (C.c_int, [h, C.c_int32, C.c_int32, _PP, _PP, _PP,
                                             C.POINTER(C.c_int32), C.POINTER(C.c_int32)]),
        "statekv_get_detailed": (C.c_int, [h, C.c_int32, C.c_int32, _PP, _PP,
                                           C.POINTER(C.c_int64), C.POINTER(C.c_int64)]),
        "statekv_frame_index": (C.c_int64, [h]),
        "statekv_decode": (C.c_int, [h, C.c_int32, _P, _P, _P, _P, _P]),
        "statekv_text_tokens": (C.c_int64, [h]),
        "statekv_set_qk_norm": (C.c_int, [h, _P, _P, C.c_float, _P]),
        "statekv_decode_tree": (C.c_int, [h, C.c_int32, _P, _P, _P, _P, _P, _P, _P]),
        "statekv_accept": (C.c_int, [h, C.c_int32, _P, _P]),
        "statekv_decode_prompt": (C.c_int, [h, C.c_int32, _P, _P, _P, _P, _P]),
        "statekv_decode_sparse": (C.c_int, [h, C.c_int32, C.c_int32, _P, _P, _P, _P, _P]),
        "statekv_reset": (C.c_int, [h]),
        "statekv_check_device_status": (C.c_int, [h, _P]),
        "statekv_get_scores": (C.c_int, [h, C.c_int32, C.c_int32, _PP, _PP,
                                         C.POINTER(C.c_int32), C.POINTER(C.c_int32)]),
        "statekv_get_rotated_query": (C.c_int, [h, _PP]),
        "statekv_set_frame_index": (C.c_int, [h, C.c_int64]),
        "statekv_set_compressed": (C.c_int, [h, C.c_int32, C.c_int32, _P, _P, _P,
                                             C.c_int32, _P]),
        "statekv_profile_enable": (C.c_int, [h, C.c_int]),
        "statekv_profile_kernels": (C.c_int, [h, C.c_uint32]),
        "statekv_profile_read": (C.c_int, [h, C.c_int32, C.POINTER(C.c_double),
                                           C.POINTER(C.c_int64)]),
        "statekv_attend_scores_static": (C.c_int, [_P, _P, _P, C.c_int32, C.c_int32,
                                                   C.c_int32, C.c_int32, C.c_int32,
                                                   C.c_int32, C.c_double, C.c_int32,
                                                   _P, _P, _P, _P]),
    }
    for name, args in (("statekv_norm_rope", NormRopeArgs), ("statekv_tree_attention", TreeArgs),
                       ("statekv_append_accepted", AppendArgs),
                       ("statekv_block_summaries", SummaryArgs),
                       ("statekv_sparse_attention", SparseArgs),
                       ("statekv_paged_append", PagedAppendArgs),
                       ("statekv_paged_attention", PagedAttentionArgs),
                       ("statekv_attention_weights", AttentionWeightsArgs),
                       ("statekv_evict_rows", EvictArgs), ("statekv_verify_tree", VerifyArgs)):
        sig[name] = (C.c_int, [C.POINTER(args), _P])
    for name in ("statekv_tree_attention_workspace", "statekv_paged_attention_workspace"):
        sig[name] = (C.c_int64, [C.c_int32] * 6)
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    ready = {}
    for name in PACKED:
        fn = lib[name]                  # a function object of its own
        fn.restype, fn.argtypes = C.c_int, [_P, _P]
        ready[name] = fn
    packed.update(ready)                # all at once: another thread may look meanwhile
    _lib = lib
    return lib


def status_string(status: int) -> str:
    try:
        return load().statekv_status_string(status).decode()
    except RuntimeError:
        return f"status {status}"


def check(status: int, what: str) -> None:
    if status != OK:
        raise StateKVError(status, what)
