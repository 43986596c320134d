"""8-bit block-scaled paged KV cache for GB300: quantize-and-scatter store, split-K decode, attention over prompts
and drafted tokens, and the cache's pages.

The compute lives in ``libkvq.so`` (CUDA, sm_103a, built from ``csrc/``); ``kvq`` is its ctypes
binding and ``workloads`` the seeded synthetic inputs.
"""
from . import kvq  # noqa: F401
from .kvq import (Layout, KvqError, alloc_append_workspace, alloc_pages_workspace, alloc_pool,  # noqa: F401
                  alloc_prompt_workspace, alloc_tree_workspace, alloc_workspace, kvq_append, kvq_bytes_per_token, kvq_decode,
                  kvq_decode_workspace_bytes, kvq_dequant_probe, kvq_device_check, kvq_encode_probe, kvq_num_pages,
                  kvq_pages_compact, kvq_pages_copy, kvq_pages_fork, kvq_pages_resize, kvq_pool_bytes, kvq_prompt,
                  kvq_scale_bytes, kvq_store, kvq_tree, kvq_version, kvq_workspace_status)

__version__ = "0.1.0"
