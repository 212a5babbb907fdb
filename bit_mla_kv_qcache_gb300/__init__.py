"""GB300-native (sm_103a) low-bit dual-path MLA KV cache: fused writer and decode attention.

The compute path is the CUDA library libmla_qcache.so (C ABI in include/mla_qcache.h);
``binding`` marshals torch tensors into it and ``cache.QuantizedMLACache`` owns the device
buffers (pool, BF16 sink/recent buffers, workspace) of one layer, ``cache.KV4Cache`` those of a
grouped-query layer in 4 bits, also for decoding with trees of drafted tokens (start_tree, append and
attend with masks, mla_qcache_verify_sampled or _greedy, keep).
"""
from .binding import (DEV_BAD_PAGE, mla_qcache_absorb_query, mla_qcache_decode_attn_pending, mla_qcache_decode_attn_multi, mla_qcache_up_project, DEV_NONFINITE, DEV_RANGE, DEV_ROWS, DEV_SEQ_OVERFLOW, DEV_TIMEOUT, EXPORTS,
                      Config, QCacheError, bf16_workspace_bytes, decode_plan, decode_launches, lib, selftest_wait_timeout, make_config, mla_qcache_advance,
                      mla_qcache_decode_attn, mla_qcache_decode_attn_bf16, mla_qcache_row_transform,
                      KV4Config, make_kv4_config, kv4_page_bytes, kv4_workspace_bytes, mla_qcache_kv4_append, mla_qcache_kv4_attn,
                      mla_qcache_append_bf16, mla_qcache_tree_mask, mla_qcache_kv4_attn_tree, mla_qcache_verify_sampled,
                      mla_qcache_verify_greedy, mla_qcache_kv4_keep,
                      mla_qcache_write, mla_qcache_write_advance, mla_qcache_write_transformed, page_bytes, strerror, workspace_bytes)
from .cache import KV4Cache, QuantizedMLACache

__all__ = ["Config", "QCacheError", "QuantizedMLACache", "lib", "make_config", "mla_qcache_advance", "mla_qcache_decode_attn",
           "mla_qcache_decode_attn_pending",
           "mla_qcache_write", "mla_qcache_write_advance", "mla_qcache_decode_attn_bf16", "bf16_workspace_bytes",
           "mla_qcache_write_transformed", "mla_qcache_row_transform",
           "mla_qcache_absorb_query", "mla_qcache_up_project", "mla_qcache_decode_attn_multi", "decode_plan", "decode_launches",
           "selftest_wait_timeout", "KV4Cache", "KV4Config", "make_kv4_config", "kv4_page_bytes", "kv4_workspace_bytes",
           "mla_qcache_kv4_append", "mla_qcache_kv4_attn", "mla_qcache_append_bf16", "mla_qcache_tree_mask", "mla_qcache_kv4_attn_tree",
           "mla_qcache_verify_sampled", "mla_qcache_verify_greedy", "mla_qcache_kv4_keep",
           "page_bytes", "strerror", "workspace_bytes", "EXPORTS", "DEV_BAD_PAGE",
           "DEV_NONFINITE", "DEV_RANGE", "DEV_ROWS", "DEV_SEQ_OVERFLOW", "DEV_TIMEOUT"]
