"""Paged KV-cache decode attention for GB300 (sm_103a).

The computation lives in ``libpagedattn.so`` (C ABI in ``include/pagedattn.h``);
``pagedattn`` is its Python binding.
"""
from .pagedattn import (  # noqa: F401
    PA_BFLOAT16,
    PA_FLOAT16,
    PA_FLOAT32,
    PA_ERR_CAPACITY,
    BlockManager,
    PagedAttnError,
    alloc_fp8_cache,
    alloc_prefill_workspace,
    alloc_shared_prefix_workspace,
    alloc_workspace,
    bad_index_count,
    copy_blocks,
    copy_blocks_fp8,
    decode,
    decode_append,
    decode_fp8,
    decode_fp8_workspace_bytes,
    decode_no_alloc,
    decode_partition_tokens,
    decode_shared_prefix,
    decode_shared_prefix_workspace_bytes,
    decode_workspace_bytes,
    gather_cache_fp8,
    last_error,
    load_library,
    prefill,
    prefill_workspace_bytes,
    no_alloc_scratch_bytes,
    reshape_and_cache,
    reshape_and_cache_fp8,
    testing_prefill_stalled,
    wait_timeout_count,
)
