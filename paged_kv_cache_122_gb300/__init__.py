"""GB300-native paged KV-cache decode path: a C-ABI CUDA library and its binding.

The calls follow the pages' statement of the problem:

* ``paged_attention_decode(q, k_cache, v_cache, block_tables, seq_lens, scale, block_size)``
* ``reshape_and_cache(k, v, k_cache, v_cache, slot_mapping)``
* ``copy_blocks(k_cache, v_cache, src_dst_pairs)``

Next to them: ``rope_and_cache`` (rotary positions and the append in one pass) and
the 8-bit cache (``fp8``: e4m3 values with a scale per block and KV head) with its
own append, attention, gather and block copies (``*_fp8``).  ``paged_attention_tree``,
``accept_tree`` and ``keep_tokens`` verify trees of drafted tokens;
``paged_attention_cross`` attends to an encoder's states.

All work runs in the library's sm_103a kernels (``csrc/``); PyTorch supplies
device memory and streams.  ``BlockManager`` is the library's host-side C++
block manager (free list, block tables, copy-on-write) that produces the
slot mapping, copy pairs and tables of a decode step.  Importing the package does not load the library;
the first call does, and fails loudly if it has not been built.
"""
from .api import (  # noqa: F401
    LayerPointers,
    copy_blocks,
    new_workspace,
    paged_attention_decode,
    paged_attention_multi_query,
    pk_paged_attention_multi_query,
    pk_copy_blocks,
    pk_copy_blocks_layers,
    pk_decode_workspace_bytes,
    pk_gather_kv,
    pk_get_device_error,
    pk_paged_attention_decode,
    pk_reshape_and_cache,
    pk_reshape_and_cache_layers,
    pk_rope_and_cache,
    pk_selftest_decode_wait_timeout,
    pk_selftest_decode_stale_lengths,
    pk_set_decode_path,
    pk_swap_blocks,
    reshape_and_cache,
    rope_and_cache,
    swap_blocks,
)
from .fp8 import (  # noqa: F401
    copy_blocks_fp8,
    gather_kv_fp8,
    new_cache_fp8,
    paged_attention_decode_fp8,
    paged_attention_multi_query_fp8,
    pk_copy_blocks_fp8,
    pk_decode_fp8_workspace_bytes,
    pk_gather_kv_fp8,
    pk_paged_attention_decode_fp8,
    pk_paged_attention_multi_query_fp8,
    pk_rope_and_cache_fp8,
    pk_selftest_decode_fp8_stale_lengths,
    pk_selftest_decode_fp8_wait_timeout,
    pk_swap_blocks_fp8,
    rope_and_cache_fp8,
    swap_blocks_fp8,
)
from .tree import (  # noqa: F401
    accept_tree,
    keep_tokens,
    paged_attention_cross,
    paged_attention_tree,
    pk_accept_tree,
    pk_keep_tokens,
    pk_keep_tokens_layers,
    pk_paged_attention_cross,
    pk_paged_attention_tree,
    pk_selftest_cross_stale_lengths,
    pk_selftest_cross_wait_timeout,
    pk_tree_workspace_bytes,
)
from ._native import PagedKVError, load as load_library  # noqa: F401
from .block_manager import BlockManager  # noqa: F401
