"""StateKV streaming video prefill for GB300 (sm_103a).

A C-ABI CUDA library (libstatekv.so, include/statekv.h) with a thin Python
binding.  Build it with ``python -m kv_cache_compression_frame_gb300.build_lib``.
"""

from .statekv import StateKV, StateKVConfig  # noqa: F401
from .text_ops import (append_accepted, block_summaries, check_status, qk_norm_rope,  # noqa: F401
                       sparse_attention, tree_attention, tree_attention_workspace, tree_masks)
from .paged_ops import (attention_weights, evict_rows, paged_append, paged_attention,  # noqa: F401
                        paged_attention_workspace, verify_tree)
from ._native import StateKVError, load as load_library  # noqa: F401

__all__ = ["StateKV", "StateKVConfig", "StateKVError", "load_library", "qk_norm_rope",
           "tree_attention", "tree_attention_workspace", "tree_masks", "append_accepted",
           "block_summaries", "sparse_attention", "check_status", "paged_append", "paged_attention",
           "paged_attention_workspace", "attention_weights", "evict_rows", "verify_tree"]
