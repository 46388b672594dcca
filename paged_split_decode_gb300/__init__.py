"""GB300-native paged split-K decode attention.

The computation lives in libpdecode.so (CUDA kernels for sm_103a behind the C
ABI of include/pdecode.h); this package is its thin Python binding plus the
seeded synthetic workload generator. Build the library with
``paged_split_decode_gb300.build.build()``.
"""
from .binding import (DEVERR_BLOCK_ID, DEVERR_FREE_LIST, DEVERR_QUERY_START, DEVERR_SEQ_LEN,
                      DEVERR_SLOT, DEVERR_TIMEOUT, DecodeError, build_block_tables, decode_paged,
                      decode_paged_combine, decode_paged_diff, decode_paged_scored, decode_paged_varlen,
                      diff_workspace_bytes, dims_of, evict_kv_cache, get_workspace, grid_ctas, load,
                      make_dims, release_blocks, rms_norm, scored_workspace_bytes, status_str,
                      workspace_bytes, write_kv_cache, write_kv_cache_fp4)

__all__ = ["DEVERR_BLOCK_ID", "DEVERR_FREE_LIST", "DEVERR_QUERY_START", "DEVERR_SEQ_LEN",
           "DEVERR_SLOT", "DEVERR_TIMEOUT", "DecodeError", "build_block_tables", "decode_paged",
           "decode_paged_combine", "decode_paged_diff", "decode_paged_scored", "decode_paged_varlen",
           "diff_workspace_bytes", "dims_of", "evict_kv_cache", "get_workspace", "grid_ctas", "load",
           "make_dims", "release_blocks", "rms_norm", "scored_workspace_bytes", "status_str",
           "workspace_bytes", "write_kv_cache", "write_kv_cache_fp4"]
